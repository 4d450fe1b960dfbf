// gemm_w4a4.cu -- Y (M x N) = s_a s_w A W^T with both operands in 4 bits, on
// the block-scaled tensor-core instructions (tcgen05, FP32 accumulators in
// TMEM): few tokens.
//
// Both operands are E2M1 codes, row-major along the contraction, with a scale
// per block of 32 (MXFP4: E8M0) or 16 (NVFP4: E4M3) in tiles of 128 rows x 4
// blocks.  The instruction multiplies the codes of 64 elements, applies both
// scales and accumulates in FP32, so nothing is dequantised on the way.
//
// What bounds few tokens is the weights' bytes.  A CTA takes 128 weight rows as
// the MMA's M side and the tokens as its N side, so that few tokens cost few
// columns; K is split over the CTAs of a cluster when there are fewer tiles
// than CTA places, and the shares are added in rank order through distributed
// shared memory.  Codes come by TMA (128-byte swizzle, zero fill outside),
// scale tiles by bulk copies; one thread copies scales to TMEM and issues the
// MMAs.  A few tokens are quantised by the CTAs themselves (each the part of K
// that it multiplies) while the first weights are on their way: a kernel of its
// own costs a launch and 1 to 2 us.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "mx_codec.cuh"
#include "sm100.cuh"
#include "w4a4_shape.h"

namespace nvfp4 {

using namespace sm100;

namespace {

constexpr int kWsThreads = 192;  // warps 0-3: tokens and epilogue, 4: copies, 5: MMA

struct W4A4Params {
    const uint8_t *a_scales, *w_scales;
    const float *a_ts, *w_ts;
    const void *x;  // unquantised tokens (M x K, ldx between rows)
    int64_t ldx;
    int M, N, K;
    int ksteps;   // stages over the whole K
    int ktiles;   // scale tiles along K
    int mtiles;   // tiles of tokens
    int split;    // CTAs of a cluster that share a tile's K
    int stages;
    int early;    // the weights were complete before the kernel before this one started
    void *y;
    int y_fp32;
    uint32_t *ctl;
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t local, uint32_t rank)
{
    float4 v;
    asm volatile(
        "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\tld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n\t}"
        : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
        : "r"(local), "r"(rank)
        : "memory");
    return v;
}

template <bool kNv, int NT, Tokens kTok>
__global__ void __launch_bounds__(kWsThreads, 2)
    w4a4_stream_kernel(const __grid_constant__ CUtensorMap tmap_w, const __grid_constant__ CUtensorMap tmap_a,
                       const W4A4Params p)
{
    using S = WsShape<kNv, NT, kTok>;
    const int kStages = p.stages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    __shared__ __align__(8) uint64_t full[kWsMaxStages], empty[kWsMaxStages], acc_full[1], x_full[1];
    __shared__ uint32_t s_tmem;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = p.split > 1 ? (int)cluster_ctarank() : 0;
    const int tile = blockIdx.x / p.split, nt = tile / p.mtiles, mt = tile % p.mtiles;   // weight rows, tokens
    const int ks0 = (int)((int64_t)p.ksteps * rank / p.split), ks1 = (int)((int64_t)p.ksteps * (rank + 1) / p.split);
    const int nk = ks1 - ks0;
    const int nx = S::kOwn ? (p.ksteps + p.split - 1) / p.split : kStages;  // token stages in shared memory

    uint8_t *sW = smem, *sX = sW + kStages * kWsRows * 128;
    uint8_t *sWs = sX + nx * NT * 128, *sXs = sWs + kStages * S::kScaleBytes;
    float *red = reinterpret_cast<float *>(smem);  // [NT][128], once the ring is drained

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; s++) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(x_full, 128);
        mbar_fence_init();
    }
    if (warp == 5) {
        tmem_alloc(&s_tmem, S::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;

    if (warp == 4) {
        const uint8_t *wsc = p.w_scales + (size_t)nt * p.ktiles * 512;
        const uint8_t *xsc = p.a_scales + (size_t)mt * p.ktiles * 512;   // more than one: 128 tokens each
        auto scale_bytes = [&](int ks) { return (uint32_t)min(S::kTiles, p.ktiles - ks * S::kTiles) * 512u; };
        auto load_w = [&](int i, int st) {
            const int ks = ks0 + i;
            const uint32_t sb = scale_bytes(ks);
            mbar_arrive_expect_tx(&full[st], (kWsRows + (S::kOwn ? 0 : NT)) * 128 + (S::kOwn ? 1 : 2) * sb);
            tma_load_2d(sW + st * kWsRows * 128, &tmap_w, &full[st], ks * 128, nt * kWsRows);
            bulk_g2s(sWs + st * S::kScaleBytes, wsc + (size_t)ks * S::kScaleBytes, sb, &full[st]);
        };
        auto load_x = [&](int i, int st) {
            if (S::kOwn)
                return;
            const int ks = ks0 + i;
            tma_load_2d(sX + st * NT * 128, &tmap_a, &full[st], ks * 128, mt * NT);
            bulk_g2s(sXs + st * S::kScaleBytes, xsc + (size_t)ks * S::kScaleBytes, scale_bytes(ks), &full[st]);
        };
        // Before the kernels ahead in the stream are complete, the weights may be
        // brought on their way: into shared memory where nothing that can still
        // run writes them (p.early), else into L2 only.
        const int head = min(nk, kStages);
        if (elect_one()) {
            for (int i = 0; i < head; i++) {
                if (p.early)
                    load_w(i, i);
                else
                    tma_prefetch_2d(&tmap_w, (ks0 + i) * 128, nt * kWsRows);
            }
            pdl_wait();
            pdl_launch_dependents();
            for (int i = 0; i < head; i++) {
                if (!p.early)
                    load_w(i, i);
                load_x(i, i);
            }
            int st = 0;
            uint32_t ph = 0;
            for (int i = head; i < nk; i++) {
                if (!mbar_wait(&empty[st], ph)) {
                    record_status(p.ctl, NVFP4_ERR_TIMEOUT);
                    break;
                }
                load_w(i, st);
                load_x(i, st);
                if (++st == kStages) {
                    st = 0;
                    ph ^= 1;
                }
            }
        }
    } else if (warp == 5) {
        constexpr uint32_t id0 = idesc_fp4(kWsRows, NT, kNv ? 0 : 1, 0);
        constexpr uint32_t id2 = idesc_fp4(kWsRows, NT, kNv ? 0 : 1, 2);
        if (elect_one()) {
            bool ok = !S::kOwn || mbar_wait(x_full, 0);
            int done = 0;   // stages multiplied, if a wait gives up
            int st = 0, st2 = kStages - S::kSfBufs, sf = 0;  // st2: the stage kSfBufs steps ago
            uint32_t ph = 0, ph2 = 1;
            for (int i = 0; i < nk && ok; i++) {
                // the MMAs that read these scale columns (kSfBufs stages ago) are done, which a ring of no more
                // stages implies, and this stage's operands have landed
                ok = (kStages <= S::kSfBufs || i < S::kSfBufs || mbar_wait(&empty[st2], ph2)) &&
                     mbar_wait(&full[st], ph);
                if (!ok) {
                    done = i;
                    break;
                }
                tc_fence_after();
                const int sx = S::kOwn ? i : st;
                const uint64_t wd = smem_desc_sw128(smem_addr(sW + st * kWsRows * 128));
                const uint64_t xd = smem_desc_sw128(smem_addr(sX + sx * NT * 128));
                const uint64_t wsd = smem_desc_scales(smem_addr(sWs + st * S::kScaleBytes));
                const uint64_t xsd = smem_desc_scales(smem_addr(sXs + sx * S::kScaleBytes));
                const uint32_t sfw = tmem + S::kAccCols + sf * S::kSfCols, sfx = sfw + S::kTiles * 4;
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
                if (i + 1 == nk)
                    mma_commit(acc_full);
                if (++st == kStages) {
                    st = 0;
                    ph ^= 1;
                }
                if (++sf == S::kSfBufs)
                    sf = 0;
                if (++st2 == kStages) {
                    st2 = 0;
                    ph2 ^= 1;
                }
            }
            if (!ok) {
                // the copies that the stages multiplied so far let go land before the CTA leaves, and the epilogue
                // hears of the MMAs issued: it waits for them before TMEM is given back
                record_status(p.ctl, NVFP4_ERR_TIMEOUT);
                ring_drain(full, kStages, done, min(nk, done + kStages));
                mma_commit(acc_full);
            }
        }
    } else {
        pdl_wait();
        if (S::kOwn) {
            // ---------------- this CTA's part of the tokens, quantised into the swizzled layout of a TMA copy:
            // four lanes a block of 32, eight elements each
            using T = typename std::conditional<kTok == kFp32, float, __nv_bfloat16>::type;
            const T *x = reinterpret_cast<const T *>(p.x);
            const int per = nk * (kWsK / 8), items = p.M * per;   // groups of eight elements, per token and in all
            constexpr int kU = kTok == kFp32 ? 3 : 6;             // loads in flight
            for (int i0 = threadIdx.x; i0 - (int)threadIdx.x < items; i0 += 128 * kU) {
                Raw8<T> raw[kU];
#pragma unroll
                for (int u = 0; u < kU; u++) {
                    const int i = i0 + 128 * u, m = i / per, k = ks0 * kWsK + (i - m * per) * 8;
                    raw[u].zero();
                    if (i < items && k < p.K)
                        raw[u].load(x + (int64_t)m * p.ldx + k);
                }
#pragma unroll
                for (int u = 0; u < kU; u++) {
                    const int i = i0 + 128 * u, m = i / per, g = i - m * per;
                    uint32_t a = raw[u].amax_bits();
                    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
                    a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
                    uint32_t byte;
                    const uint32_t q = raw[u].encode(a, byte);
                    if (i < items) {
                        const int ks = g / (kWsK / 8), kb = g % (kWsK / 8) * 4;   // stage, byte of its row
                        *reinterpret_cast<uint32_t *>(sX + ks * NT * 128 + m * 128 + (((kb >> 4) ^ (m & 7)) << 4) +
                                                      (kb & 15)) = q;
                        if ((lane & 3) == 0)
                            sXs[ks * S::kScaleBytes + (kb >> 6) * 512 + m * 16 + (kb >> 4 & 3)] = (uint8_t)byte;
                    }
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(x_full);
        }
        if (!mbar_wait_warp(acc_full, 0)) {
            if (threadIdx.x == 0)
                record_status(p.ctl, NVFP4_ERR_TIMEOUT);
            // longer than the issuing thread can take over its own waits
            for (int i = 0; i < 2 * nk + kStages + 4 && !mbar_wait_warp(acc_full, 0); i++) {
            }
        }
        tc_fence_after();
    }
    __syncwarp();

    // one after the other: the product of two small tensor scales may underflow
    const float s_a = p.a_ts ? *p.a_ts : 1.0f, s_w = p.w_ts ? *p.w_ts : 1.0f;
    auto store = [&](int m, int n, float v) {
        v = __fmul_rn(__fmul_rn(v, s_a), s_w);
        if (p.y_fp32)
            reinterpret_cast<float *>(p.y)[(size_t)m * p.N + n] = v;
        else
            reinterpret_cast<__nv_bfloat16 *>(p.y)[(size_t)m * p.N + n] = __float2bfloat16_rn(v);
    };
    if (warp < 4) {
        const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
        const int n = nt * kWsRows + threadIdx.x;
        constexpr int kChunk = NT < 32 ? NT : 32;
        for (int c = 0; c < NT; c += 32) {
            uint32_t v[32];
            __syncwarp();   // the stores before may have parted the warp
            tmem_ld32_start(lane_base + c, v);
            tmem_ld32_finish(v);
#pragma unroll
            for (int i = 0; i < kChunk; i++) {
                const int m = mt * NT + c + i;
                if (p.split > 1)
                    red[(c + i) * 128 + threadIdx.x] = __uint_as_float(v[i]);
                else if (m < p.M && n < p.N)
                    store(m, n, __uint_as_float(v[i]));
            }
        }
    }
    if (p.split > 1) {
        // ---------------- the tokens' columns are shared out; four weight rows a thread
        __syncthreads();
        cluster_sync();
        const int cols = min(NT, p.M - mt * NT);
        const int c0 = cols * rank / p.split, c1 = cols * (rank + 1) / p.split;
        for (int i = threadIdx.x; i < (c1 - c0) * 32; i += kWsThreads) {
            const int c = c0 + i / 32, r4 = i % 32 * 4;
            const uint32_t at = smem_addr(&red[c * 128 + r4]);
            float4 part[8];
#pragma unroll
            for (int r = 0; r < 8; r++)
                if (r < p.split)
                    part[r] = ld_cluster_f4(at, (uint32_t)r);
            float4 v = part[0];
#pragma unroll
            for (int r = 1; r < 8; r++) {
                if (r < p.split) {
                    v.x += part[r].x;
                    v.y += part[r].y;
                    v.z += part[r].z;
                    v.w += part[r].w;
                }
            }
            const float vv[4] = {v.x, v.y, v.z, v.w};
            const int n = nt * kWsRows + r4;
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (n + e < p.N)
                    store(mt * NT + c, n + e, vv[e]);
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

template <bool kNv, int NT, Tokens kTok>
cudaError_t run_stream(const W4A4Args &a, cudaStream_t s, const DeviceInfo &dev)
{
    using S = WsShape<kNv, NT, kTok>;
    CUtensorMap tw, ta;
    cudaError_t e = encode_tensor_map_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w_codes, (uint64_t)a.K / 2,
                                         (uint64_t)a.N, (uint64_t)a.K / 2, 128, kWsRows, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess)
        e = S::kOwn ? (ta = tw, cudaSuccess)
                    : encode_tensor_map_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.a_codes, (uint64_t)a.K / 2,
                                           (uint64_t)a.M, (uint64_t)a.K / 2, 128, NT, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e != cudaSuccess)
        return e;
    W4A4Params p;
    p.a_scales = a.a_scales;
    p.w_scales = a.w_scales;
    p.a_ts = a.a_ts;
    p.w_ts = a.w_ts;
    p.x = a.x;
    p.ldx = a.ldx;
    p.M = (int)a.M;
    p.N = (int)a.N;
    p.K = (int)a.K;
    p.ksteps = (int)((a.K + kWsK - 1) / kWsK);
    const int64_t per_tile = kNv ? 64 : 128;
    p.ktiles = (int)((a.K + per_tile - 1) / per_tile);
    p.mtiles = (int)((a.M + NT - 1) / NT);
    const int64_t tiles = (int64_t)p.mtiles * ((a.N + kWsRows - 1) / kWsRows);
    p.split = ws_split(tiles, a.K, dev.num_sms);
    const int nk = (p.ksteps + p.split - 1) / p.split;
    p.stages = S::stages(nk);
    p.early = a.after_quantise ? 1 : 0;
    p.y = a.y;
    p.y_fp32 = a.y_fp32 ? 1 : 0;
    p.ctl = a.ctl;
    e = allow_smem<w4a4_stream_kernel<kNv, NT, kTok>>(kWsSmem, dev);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * p.split));
    cfg.blockDim = dim3(kWsThreads);
    cfg.dynamicSmemBytes = S::smem(nk, p.stages);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, w4a4_stream_kernel<kNv, NT, kTok>, tw, ta, p);
}

template <bool kNv>
cudaError_t run_w4a4(const W4A4Args &a, cudaStream_t s, const DeviceInfo &dev)
{
    if (a.M <= 16)
        return run_stream<kNv, 16, kCodes>(a, s, dev);
    if (a.M <= 32)
        return run_stream<kNv, 32, kCodes>(a, s, dev);
    // More tokens go to the tile kernel, 256 x 256 at a time on 76 pairs of CTAs
    // (100 tokens: 11.3 us by tiles and 12.3 streamed at N = 18944, K = 3584; 64:
    // 11.4 and 10.8), unless there are few such tiles with long sums: only the
    // stream splits K (256 tokens at N = 3584, K = 18944: 27 and 16 us; 512: 27
    // and 24; at K = 3584: 8.8 and 9.4).
    const int64_t big = ((a.M + 255) / 256) * ((a.N + 255) / 256);
    const bool long_sums = big * 5 <= dev.num_sms && a.K >= 32 * kWsK && a.M <= 512;
    if (a.M <= 64)
        return run_stream<kNv, 64, kCodes>(a, s, dev);
    if (long_sums)
        return run_stream<kNv, 128, kCodes>(a, s, dev);
    return launch_w4a4_tile(a, s, dev);
}

}  // namespace

bool w4a4_takes_tokens(int64_t M, int64_t N, int64_t K, bool fp32, const DeviceInfo &dev)
{
    return ws_takes_tokens(M, N, K, fp32, dev.num_sms);
}

cudaError_t launch_w4a4(const W4A4Args &a, cudaStream_t s, const DeviceInfo &dev)
{
    if (a.x)
        return a.x_fp32 ? run_stream<false, 16, kFp32>(a, s, dev) : run_stream<false, 16, kBf16>(a, s, dev);
    return a.nvfp4 ? run_w4a4<true>(a, s, dev) : run_w4a4<false>(a, s, dev);
}

}  // namespace nvfp4
