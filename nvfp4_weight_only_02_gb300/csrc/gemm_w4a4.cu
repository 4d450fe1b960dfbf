// gemm_w4a4.cu -- Y (M x N) = s_a s_w A W^T with both operands in 4 bits, on
// the block-scaled tensor-core instructions (tcgen05, FP32 accumulators in
// TMEM).
//
// Both operands are E2M1 codes, row-major along the contraction, with a scale
// per block of 32 (MXFP4: E8M0) or 16 (NVFP4: E4M3) in tiles of 128 rows x 4
// blocks.  The instruction multiplies the codes of 64 elements, applies both
// scales and accumulates in FP32, so nothing is dequantised on the way.
//
// A CTA takes 128 weight rows as the MMA's M side and up to 128 tokens as its
// N side, so that few tokens cost few columns; the contraction is split over
// the CTAs of a cluster when there are fewer tiles than SMs, and the shares
// are added in rank order through distributed shared memory.  Codes come by
// TMA (128-byte swizzle, zero fill outside), scale tiles by bulk copies; one
// thread copies scales to TMEM and issues the MMAs.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace nvfp4 {

using namespace sm100;

namespace {

constexpr int kWsThreads = 192;  // warps 0-3: epilogue, 4: copies, 5: MMA
constexpr int kWsRows = 128;     // weight rows per CTA
constexpr int kWsK = 256;        // elements of K per stage (128 bytes of codes a row)

struct W4A4Params {
    const uint8_t *a_scales, *w_scales;
    const float *a_ts, *w_ts;
    int M, N;
    int ksteps;   // stages over the whole K
    int ktiles;   // scale tiles along K
    int mtiles;
    int split;    // CTAs of a cluster that share a tile's K
    void *y;
    int y_fp32;
    uint32_t *ctl;
};

template <bool kNv, int NT>
struct WsShape {
    static constexpr int kTiles = kNv ? 4 : 2;                    // scale tiles per stage and operand
    static constexpr int kScaleBytes = kTiles * 512;
    static constexpr int kStageBytes = kWsRows * 128 + NT * 128 + 2 * kScaleBytes;
    // two CTAs share an SM (227 KB)
    static constexpr int kStages = 112000 / kStageBytes < 5 ? 112000 / kStageBytes : 5;
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + 256;
    static constexpr int kAccCols = NT < 64 ? 64 : NT;
    static constexpr int kSfCols = 2 * kTiles * 4;                // one stage's scales of both operands
    static constexpr int kTmemCols = kAccCols + 2 * kSfCols <= 128 ? 128 : 256;
};

__device__ __forceinline__ float ld_cluster_f32(uint32_t local, uint32_t rank)
{
    float v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
                 : "=f"(v)
                 : "r"(local), "r"(rank)
                 : "memory");
    return v;
}

template <bool kNv, int NT>
__global__ void __launch_bounds__(kWsThreads)
    w4a4_stream_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_a,
                       const W4A4Params p)
{
    using S = WsShape<kNv, NT>;
    constexpr int kStages = S::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *sW = smem, *sX = sW + kStages * kWsRows * 128;
    uint8_t *sWs = sX + kStages * NT * 128, *sXs = sWs + kStages * S::kScaleBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(sXs + kStages * S::kScaleBytes);
    uint64_t *empty = full + kStages, *acc_full = empty + kStages;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(acc_full + 1);
    float *red = reinterpret_cast<float *>(smem);  // [NT][128], once the ring is drained

    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; s++) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        mbar_fence_init();
    }
    if (warp == 5) {
        tmem_alloc(s_tmem, S::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;

    const int rank = p.split > 1 ? (int)cluster_ctarank() : 0;
    const int tile = blockIdx.x / p.split, nt = tile / p.mtiles, mt = tile % p.mtiles;
    const int ks0 = (int)((int64_t)p.ksteps * rank / p.split), ks1 = (int)((int64_t)p.ksteps * (rank + 1) / p.split);
    const int nk = ks1 - ks0;

    if (warp == 4) {
        const uint8_t *wsc = p.w_scales + (size_t)nt * p.ktiles * 512;
        const uint8_t *xsc = p.a_scales + (size_t)(mt * NT / 128) * p.ktiles * 512;
        auto scale_bytes = [&](int ks) { return (uint32_t)min(S::kTiles, p.ktiles - ks * S::kTiles) * 512u; };
        auto load_w = [&](int i, int st) {
            const int ks = ks0 + i;
            const uint32_t sb = scale_bytes(ks);
            mbar_arrive_expect_tx(&full[st], (kWsRows + NT) * 128 + 2 * sb);
            tma_load_2d(sW + st * kWsRows * 128, &tmap_w, &full[st], ks * 128, nt * kWsRows);
            bulk_g2s(sWs + st * S::kScaleBytes, wsc + (size_t)ks * S::kScaleBytes, sb, &full[st]);
        };
        auto load_x = [&](int i, int st) {
            const int ks = ks0 + i;
            tma_load_2d(sX + st * NT * 128, &tmap_a, &full[st], ks * 128, mt * NT);
            bulk_g2s(sXs + st * S::kScaleBytes, xsc + (size_t)ks * S::kScaleBytes, scale_bytes(ks), &full[st]);
        };
        // weights do not depend on the kernel before this one: they start first
        const int head = min(nk, kStages);
        for (int i = 0; i < head; i++) {
            if (elect_one())
                load_w(i, i);
            __syncwarp();
        }
        pdl_wait();
        for (int i = 0; i < head; i++) {
            if (elect_one())
                load_x(i, i);
            __syncwarp();
        }
        for (int i = head; i < nk; i++) {
            const int st = i % kStages;
            if (!mbar_wait_warp(&empty[st], (i / kStages + 1) & 1)) {
                record_status(p.ctl, NVFP4_ERR_TIMEOUT);
                break;
            }
            if (elect_one()) {
                load_w(i, st);
                load_x(i, st);
            }
            __syncwarp();
        }
    } else if (warp == 5) {
        constexpr uint32_t id0 = idesc_fp4(kWsRows, NT, kNv ? 0 : 1, 0);
        constexpr uint32_t id2 = idesc_fp4(kWsRows, NT, kNv ? 0 : 1, 2);
        for (int i = 0; i < nk; i++) {
            const int st = i % kStages;
            // the MMAs that read this half of the scale columns (two stages ago) are done, and this stage's
            // operands have landed
            if ((i >= 2 && !mbar_wait_warp(&empty[(i - 2) % kStages], ((i - 2) / kStages) & 1)) ||
                !mbar_wait_warp(&full[st], (i / kStages) & 1)) {
                record_status(p.ctl, NVFP4_ERR_TIMEOUT);
                break;
            }
            tc_fence_after();
            if (elect_one()) {
                const uint64_t wd = smem_desc_sw128(smem_addr(sW + st * kWsRows * 128));
                const uint64_t xd = smem_desc_sw128(smem_addr(sX + st * NT * 128));
                const uint64_t wsd = smem_desc_scales(smem_addr(sWs + st * S::kScaleBytes));
                const uint64_t xsd = smem_desc_scales(smem_addr(sXs + st * S::kScaleBytes));
                const uint32_t sfw = tmem + S::kAccCols + (i & 1) * S::kSfCols, sfx = sfw + S::kTiles * 4;
                const int tiles = min(S::kTiles, p.ktiles - (ks0 + i) * S::kTiles);
#pragma unroll
                for (int t = 0; t < S::kTiles; t++) {
                    if (t < tiles) {
                        tmem_cp_scales(sfw + 4 * t, wsd + 32 * t);
                        tmem_cp_scales(sfx + 4 * t, xsd + 32 * t);
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const int t = kNv ? j : j / 2;
                    if (t < tiles)
                        mma_fp4_ss<kNv>(tmem, wd + 2 * j, xd + 2 * j, !kNv && (j & 1) ? id2 : id0, sfw + 4 * t,
                                        sfx + 4 * t, (i | j) != 0);
                }
                mma_commit(&empty[st]);
            }
            __syncwarp();
        }
        if (elect_one())
            mma_commit(acc_full);
        __syncwarp();
    } else {
        if (!mbar_wait_warp(acc_full, 0)) {
            if (threadIdx.x == 0)
                record_status(p.ctl, NVFP4_ERR_TIMEOUT);
        }
        tc_fence_after();
    }
    __syncwarp();

    // one after the other: the product of two small tensor scales may underflow
    const float s_a = p.a_ts ? *p.a_ts : 1.0f, s_w = p.w_ts ? *p.w_ts : 1.0f;
    const int n = nt * kWsRows + threadIdx.x;
    auto store = [&](int col, float v) {
        const int m = mt * NT + col;
        if (m < p.M && n < p.N) {
            v = __fmul_rn(__fmul_rn(v, s_a), s_w);
            if (p.y_fp32)
                reinterpret_cast<float *>(p.y)[(size_t)m * p.N + n] = v;
            else
                reinterpret_cast<__nv_bfloat16 *>(p.y)[(size_t)m * p.N + n] = __float2bfloat16_rn(v);
        }
    };
    if (warp < 4) {
        const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
        constexpr int kChunk = NT < 32 ? NT : 32;
        for (int c = 0; c < NT; c += 32) {
            uint32_t v[32];
            tmem_ld32_start(lane_base + c, v);
            tmem_ld32_finish(v);
#pragma unroll
            for (int i = 0; i < kChunk; i++) {
                if (p.split == 1)
                    store(c + i, __uint_as_float(v[i]));
                else
                    red[(c + i) * 128 + threadIdx.x] = __uint_as_float(v[i]);
            }
        }
    }
    if (p.split > 1) {
        __syncthreads();
        cluster_sync();
        if (warp < 4) {
            const int c0 = NT * rank / p.split, c1 = NT * (rank + 1) / p.split;
            for (int c = c0; c < c1; c++) {
                const uint32_t at = smem_addr(&red[c * 128 + threadIdx.x]);
                float v = 0.0f;
                for (int r = 0; r < p.split; r++)
                    v += ld_cluster_f32(at, (uint32_t)r);
                store(c, v);
            }
        }
        __syncwarp();
        cluster_sync();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem, S::kTmemCols);
    }
}

template <bool kNv, int NT>
cudaError_t run_stream(const W4A4Args &a, cudaStream_t s, const DeviceInfo &dev)
{
    using S = WsShape<kNv, NT>;
    CUtensorMap tw, ta;
    cudaError_t e = encode_tensor_map_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w_codes, (uint64_t)a.K / 2,
                                         (uint64_t)a.N, (uint64_t)a.K / 2, 128, kWsRows, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess)
        e = encode_tensor_map_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.a_codes, (uint64_t)a.K / 2, (uint64_t)a.M,
                                 (uint64_t)a.K / 2, 128, NT, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess)
        return e;
    W4A4Params p;
    p.a_scales = a.a_scales;
    p.w_scales = a.w_scales;
    p.a_ts = a.a_ts;
    p.w_ts = a.w_ts;
    p.M = (int)a.M;
    p.N = (int)a.N;
    p.ksteps = (int)((a.K + kWsK - 1) / kWsK);
    const int64_t per_tile = kNv ? 64 : 128;
    p.ktiles = (int)((a.K + per_tile - 1) / per_tile);
    p.mtiles = (int)((a.M + NT - 1) / NT);
    p.y = a.y;
    p.y_fp32 = a.y_fp32 ? 1 : 0;
    p.ctl = a.ctl;
    const int64_t tiles = (int64_t)p.mtiles * ((a.N + kWsRows - 1) / kWsRows);
    // two CTAs per SM: split K while the tiles leave room
    p.split = (int)std::max<int64_t>(1, std::min<int64_t>({8, p.ksteps, 2 * dev.num_sms / tiles}));
    e = cudaFuncSetAttribute(w4a4_stream_kernel<kNv, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)S::kSmem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * p.split));
    cfg.blockDim = dim3(kWsThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.after_quantise ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, w4a4_stream_kernel<kNv, NT>, tw, ta, p);
}

template <bool kNv>
cudaError_t run_w4a4(const W4A4Args &a, cudaStream_t s, const DeviceInfo &dev)
{
    if (a.M <= 16)
        return run_stream<kNv, 16>(a, s, dev);
    if (a.M <= 32)
        return run_stream<kNv, 32>(a, s, dev);
    if (a.M <= 64)
        return run_stream<kNv, 64>(a, s, dev);
    if (a.M <= 128)
        return run_stream<kNv, 128>(a, s, dev);
    return launch_w4a4_tile(a, s, dev);
}

}  // namespace

cudaError_t launch_w4a4(const W4A4Args &a, cudaStream_t s, const DeviceInfo &dev)
{
    return a.nvfp4 ? run_w4a4<true>(a, s, dev) : run_w4a4<false>(a, s, dev);
}

}  // namespace nvfp4
