// gemm_moe.cu -- MXFP4 products grouped by expert: rows of tokens sorted by
// expert, one weight matrix an expert, numbers of rows known on the device only.
//
//   Y_r = x_r W_e^T           for the rows r of expert e      (moe_tile, moe_stream)
//   dW_e = A_e^T X_e          over the rows of expert e       (moe_wgrad)
//
// The grouping (moe_plan.h) lists tiles of rows that belong to one expert; a
// launch is sized by the most tiles that there can be and reads the list.  The
// MMA's M side is the weights' rows, its N side the tokens, so a tile costs as
// many columns as it has rows: experts with few rows waste nothing.  In the
// quantised operands every expert's rows begin on a multiple of 128, where the
// tiled scales and the copies can start; in Y the rows are compact, so stores
// are by row and never touch a row of another expert or one behind the last.
//
// What bounds it.  Few rows: the weights' bytes (64 tokens with 4 of 60 experts of
// 2600 x 3584: 46 us, 6.5 TB/s).  Many: 8192 tokens with 8 of 128 experts of 1536 x
// 4096 take 155 us for 764 MB moved (DRAM 4.9 TB/s, tensor pipe 59 %); the experts'
// last tiles are a quarter more tiles than full ones would be, and a tile of few
// rows costs 0.23 us a stage, one of 256 rows 0.28 (gemm_w4a4_tile.cu).  Measured
// and left out: rows gathered by the product itself (mx_quant.cu), weights or Y
// marked to be evicted first (217 and 203 us for the layer, 204 without).
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "moe_plan.h"
#include "tile_store.cuh"
#include "w4a4_pair.cuh"
#include "w4a4_shape.h"

namespace nvfp4 {

namespace {

static_assert(2 * kStageOut <= kTlEpiWarps * kTlStoreBytes, "the tiles' staging");

struct MoeParams {
    const int32_t *header;
    const int4 *tiles;
    const uint8_t *x_scales, *w_scales;
    int N;
    int ksteps;    // stages over K
    int ktiles;    // scale tiles along K
    int wtiles;    // tiles of weight rows (256 a pair, 128 a CTA)
    int wrows;     // scale tiles over an expert's rows
    int split;     // streaming: CTAs of a cluster that share a tile's K
    int stages;
    int early;     // the plan and the weights were complete before the kernel before this one started its work
    void *y;
    int y_fp32;
    uint32_t *ctl;
};

// ---------------------------------------------------------------- CTA pairs
// Items (tile of rows, 256 weight rows), dealt out to the pairs in turn, the
// weight tile fastest.
template <int TR, bool kF32>
__global__ void __launch_bounds__(kTlThreads, 1) __cluster_dims__(2, 1, 1)
    moe_tile_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                    const __grid_constant__ CUtensorMap tm_sw, const __grid_constant__ CUtensorMap tm_sx,
                    const MoeParams p)
{
    using S = TlShape<false, TR>;
    constexpr int kStages = S::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *sA = smem, *sB = sA + kStages * S::kABytes, *sOut = sB + kStages * S::kBBytes;
    uint8_t *sSa = sOut + 2 * kStageOut, *sSb = sSa + kStages * S::kSaBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(sSb + kStages * S::kSbBytes);
    uint64_t *empty = full + kStages, *acc_full = empty + kStages, *acc_empty = acc_full + 2;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(acc_empty + 2);
    volatile int *s_abort = reinterpret_cast<volatile int *>(s_tmem + 1);
    volatile uint32_t *s_loaded = s_tmem + 2, *s_issued = s_tmem + 3;   // stages copied and multiplied

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int crank = (int)cluster_ctarank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; s++) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&acc_full[0], 1);
        mbar_init(&acc_full[1], 1);
        mbar_init(&acc_empty[0], 2 * kTlEpiWarps);
        mbar_init(&acc_empty[1], 2 * kTlEpiWarps);
        *s_abort = 0;
        *s_loaded = 0;
        *s_issued = 0;
        mbar_fence_init();
    }
    if (warp == kTlEpiWarps + 1)
        tmem_alloc_pair(s_tmem, S::kTmemCols);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers and TMEM before anything of the pair touches them
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    pdl_wait();
    pdl_launch_dependents();

    const int cid = (int)cluster_id_x(), ncl = (int)cluster_count_x();
    const int ntot = p.header[kMoeTiles] * p.wtiles;
    auto fail = [&]() {
        record_status(p.ctl, NVFP4_ERR_TIMEOUT);
        *s_abort = 1;
    };
    auto aborted = [&]() { return __any_sync(0xffffffffu, *s_abort); };
    // columns of a tile's MMAs
    auto width = [](int rows) { return (rows + 31) & ~31; };

    if (warp == kTlEpiWarps) {
        // ---------------- copies: this CTA's half of each operand
        if (elect_one()) {
            uint32_t it = 0;
            for (int t = cid; t < ntot && !*s_abort; t += ncl) {
                const int4 tile = p.tiles[t / p.wtiles];
                const int wt = t % p.wtiles, half = width(tile.w) / 2;
                for (int ks = 0; ks < p.ksteps; ks++, it++) {
                    const int st = it % kStages;
                    if (!mbar_wait(&empty[st], ((it / kStages) & 1) ^ 1)) {
                        fail();
                        break;
                    }
                    const uint32_t bar = cluster_addr(&full[st], 0);
                    if (crank == 0)
                        mbar_arrive_expect_tx(&full[st], 2 * S::kStageBytes);
                    tma_load_3d_pair(sA + st * S::kABytes, &tm_w, bar, ks * 128, wt * 256 + crank * 128, tile.x);
                    tma_load_2d_pair(sB + st * S::kBBytes, &tm_x, bar, ks * 128, tile.y + crank * half);
                    // behind an expert's last scale tile: the next expert's, for rows that are not stored
                    tma_load_3d_pair(sSa + st * S::kSaBytes, &tm_sw, bar, 0, ks * S::kTiles,
                                     tile.x * p.wrows + 2 * wt + crank);
                    tma_load_3d_pair(sSb + st * S::kSbBytes, &tm_sx, bar, 0, ks * S::kTiles, tile.y / kMoeBlock);
                }
            }
            // every stage released before leaving: the leader's commits must not arrive at a CTA that is gone
            for (int k = 0; k < kStages && !*s_abort; k++) {
                const uint32_t i2 = it + k;
                if (i2 >= (uint32_t)kStages && !mbar_wait(&empty[i2 % kStages], ((i2 / kStages) & 1) ^ 1))
                    fail();
            }
            *s_loaded = it;
        }
    } else if (warp == kTlEpiWarps + 1) {
        // ---------------- MMA, by one thread of the pair's leader
        if (crank == 0 && elect_one()) {
            uint32_t it = 0, lt = 0;
            for (int t = cid; t < ntot && !*s_abort; t += ncl, lt++) {
                const int rows = p.tiles[t / p.wtiles].w;
                const uint32_t id0 = idesc_fp4(256, width(rows), 1, 0), id2 = idesc_fp4(256, width(rows), 1, 2);
                // the shared columns of the accumulator before this one have been read, or without
                // shared columns the accumulator that this tile takes
                if (S::kShared ? lt >= 1 && !mbar_wait(&acc_empty[0], (lt - 1) & 1)
                               : lt >= 2 && !mbar_wait(&acc_empty[lt & 1], (lt / 2 - 1) & 1)) {
                    fail();
                    break;
                }
                tc_fence_after();
                const uint32_t acc = tmem + (lt & 1 ? S::kAcc1 : 0);
                bool ok = true;
                for (int ks = 0; ks < p.ksteps; ks++, it++) {
                    const int st = it % kStages;
                    // the MMAs that read these scale columns (kSfBufs stages ago) are done, and this stage's
                    // operands have landed
                    constexpr uint32_t kB = S::kSfBufs;
                    if ((it >= kB && !mbar_wait(&empty[(it - kB) % kStages], ((it - kB) / kStages) & 1)) ||
                        !mbar_wait(&full[st], (it / kStages) & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = smem_desc_sw128(smem_addr(sA + st * S::kABytes));
                    const uint64_t bd = smem_desc_sw128(smem_addr(sB + st * S::kBBytes));
                    const uint64_t sad = smem_desc_scales(smem_addr(sSa + st * S::kSaBytes));
                    const uint64_t sbd = smem_desc_scales(smem_addr(sSb + st * S::kSbBytes));
                    const uint32_t sfa = tmem + S::kSfCol + it % S::kSfBufs * S::kSf, sfb = sfa + S::kSfA;
#pragma unroll
                    for (int k = 0; k < S::kTiles; k++) {
                        tmem_cp_scales_pair(sfa + 4 * k, sad + k * 32);
#pragma unroll
                        for (int r = 0; r < S::kBRowTiles; r++)
                            tmem_cp_scales_pair(sfb + 4 * (k * S::kBRowTiles + r), sbd + (r * S::kTiles + k) * 32);
                    }
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        mma_fp4_pair<false>(acc, ad + 2 * j, bd + 2 * j, j & 1 ? id2 : id0, sfa + 4 * (j / 2),
                                            sfb + 4 * (j / 2) * S::kBRowTiles, (ks | j) != 0);
                    mma_commit_pair(&empty[st]);
                    if (ks + 1 == p.ksteps)
                        mma_commit_pair(&acc_full[lt & 1]);
                }
                if (!ok) {
                    fail();
                    break;
                }
            }
            *s_issued = it;
        }
    } else {
        // ---------------- epilogue: warp w has weight rows 32 (w % 4) .. + 31, one a lane, and every other 32
        // tokens, the columns that both accumulators use first
        constexpr int kChunks = TR / 32, kSharedChunks = S::kShared / 32;
        const int quad = warp & 3, half = warp >> 2;
        const uint32_t bar0 = cluster_addr(&acc_empty[0], 0), bar1 = cluster_addr(&acc_empty[1], 0);
        uint8_t *stage = sOut + half * kStageOut;
        uint32_t lt = 0;
        bool dead = false;   // after a wait that gave up: the four warps that store together stay together
        for (int t = cid; t < ntot; t += ncl, lt++) {
            const int4 tile = p.tiles[t / p.wtiles];
            const int n0 = t % p.wtiles * 256 + crank * 128;
            if (!dead && (aborted() || !mbar_wait_warp(&acc_full[lt & 1], (lt >> 1) & 1))) {
                fail();
                dead = true;
            }
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(quad * 32) << 16) + (lt & 1 ? S::kAcc1 : 0);
            // accumulator 0 ends with the shared columns, accumulator 1 begins with them
            const int first = lt & 1 ? 0 : kChunks - kSharedChunks;
            uint32_t buf[2][32];
            tile_ld_start<kF32>(acc + (first + half) % kChunks * 32, buf[0]);
#pragma unroll
            for (int i = 0; i < kChunks / 2; i++) {
                uint32_t(&v)[32] = buf[i & 1];
                __syncwarp();   // the stores before may have parted the warp
                tmem_ld32_finish(v);
                if (i + 1 < kChunks / 2)
                    tile_ld_start<kF32>(acc + (first + half + 2 * (i + 1)) % kChunks * 32, buf[(i + 1) & 1]);
                if (S::kShared ? half + 2 * i < kSharedChunks && half + 2 * i + 2 >= kSharedChunks
                               : i + 1 == kChunks / 2) {
                    // this warp's part of the shared columns (of all) is in registers
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_cluster(S::kShared || !(lt & 1) ? bar0 : bar1);
                }
                const int c0 = (first + half + 2 * i) % kChunks * 32, left = min(32, tile.w - c0);
                if (left > 0 && n0 < p.N)
                    store_rows<kF32>(v, stage, 1 + half, p.y, tile.z + c0, left, p.N, n0, quad, lane, !dead);
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (crank == 0 && warp == kTlEpiWarps + 1 && *s_abort) {
        // after a wait that gave up: copies on their way land, and MMAs issued are done, before either CTA leaves
        const uint32_t loaded = *s_loaded, issued = *s_issued;
        ring_drain(full, kStages, loaded > (uint32_t)kStages ? loaded - kStages : 0u, loaded);
        if (issued > 0)
            ring_drain(empty, kStages, issued - 1, issued);
        __syncwarp();
    }
    cluster_sync();  // neither CTA leaves while the other may still signal or read it
    if (warp == kTlEpiWarps + 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, S::kTmemCols);
    }
}

// ---------------------------------------------------------------- few rows
// A CTA takes 128 weight rows and one tile of rows (NT at most); K is split
// over the CTAs of a cluster when there are fewer tiles than CTA places, the
// shares added in rank order through distributed shared memory.  Up to 16 rows,
// a decode step's usual number, only those are copied.
constexpr int kMsFew = 16;
constexpr int kMsThreads = 192;  // warps 0-3: epilogue, 4: copies, 5: MMA

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

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            smem_addr(dst)),
        "l"((uint64_t)map), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}

template <int NT>
__global__ void __launch_bounds__(kMsThreads, 2)
    moe_stream_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                      const __grid_constant__ CUtensorMap tm_few, const MoeParams p)
{
    using S = WsShape<false, NT, kCodes>;
    const int kStages = p.stages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    __shared__ __align__(8) uint64_t full[kWsMaxStages], empty[kWsMaxStages], acc_full[1];
    __shared__ uint32_t s_tmem;

    const int warp = threadIdx.x >> 5;
    const int rank = p.split > 1 ? (int)cluster_ctarank() : 0;
    const int item = blockIdx.x / p.split, wt = item % p.wtiles;
    const int ks0 = (int)((int64_t)p.ksteps * rank / p.split), ks1 = (int)((int64_t)p.ksteps * (rank + 1) / p.split);
    const int nk = ks1 - ks0;
    // Behind the quantiser, which waited for what is before it, the list and the weights can be read at once; only the
    // rows are waited for.
    if (!p.early) {
        pdl_wait();
        pdl_launch_dependents();
    }
    if (item / p.wtiles >= p.header[kMoeTiles]) {
        if (p.early)
            pdl_wait();     // a launch of nothing but these must not end before the quantiser
        return;             // the whole cluster
    }
    const int4 tile = p.tiles[item / p.wtiles];

    uint8_t *sW = smem, *sX = sW + kStages * kWsRows * 128;
    uint8_t *sWs = sX + kStages * NT * 128, *sXs = sWs + kStages * S::kScaleBytes;
    float *red = reinterpret_cast<float *>(smem);  // [NT][128], once the ring is drained

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; s++) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(acc_full, 1);
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
        if (elect_one()) {
            const uint8_t *wsc = p.w_scales + ((size_t)tile.x * p.wrows + wt) * p.ktiles * 512;
            const uint8_t *xsc = p.x_scales + (size_t)(tile.y / kMoeBlock) * p.ktiles * 512;
            const bool few = tile.w <= kMsFew;
            auto scale_bytes = [&](int ks) { return (uint32_t)min(S::kTiles, p.ktiles - ks * S::kTiles) * 512u; };
            auto load_w = [&](int i, int st) {
                const int ks = ks0 + i;
                const uint32_t sb = scale_bytes(ks);
                mbar_arrive_expect_tx(&full[st], (kWsRows + (few ? kMsFew : NT)) * 128 + 2 * sb);
                tma_load_3d(sW + st * kWsRows * 128, &tm_w, &full[st], ks * 128, wt * kWsRows, tile.x);
                bulk_g2s(sWs + st * S::kScaleBytes, wsc + (size_t)ks * S::kScaleBytes, sb, &full[st]);
            };
            auto load_x = [&](int i, int st) {
                const int ks = ks0 + i;
                tma_load_2d(sX + st * NT * 128, few ? &tm_few : &tm_x, &full[st], ks * 128, tile.y);
                bulk_g2s(sXs + st * S::kScaleBytes, xsc + (size_t)ks * S::kScaleBytes, scale_bytes(ks), &full[st]);
            };
            const int head = min(nk, kStages);
            for (int i = 0; i < head; i++)
                load_w(i, i);
            if (p.early) {
                pdl_wait();
                pdl_launch_dependents();
            }
            for (int i = 0; i < head; i++)
                load_x(i, i);
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
        if (elect_one()) {
            const int cols = (tile.w + 15) & ~15;
            const uint32_t id0 = idesc_fp4(kWsRows, cols, 1, 0), id2 = idesc_fp4(kWsRows, cols, 1, 2);
            const uint32_t off = (uint32_t)(tile.y % kMoeBlock) / 32;   // columns of the rows' scale tile before this tile
            bool ok = true;
            int done = 0;   // stages multiplied, if a wait gives up
            int st = 0, st2 = kStages - S::kSfBufs, sf = 0;  // st2: the stage kSfBufs steps ago
            uint32_t ph = 0, ph2 = 1;
            for (int i = 0; i < nk; i++) {
                // the MMAs that read these scale columns (kSfBufs stages ago) are done, which a ring of no more
                // stages implies, and this stage's operands have landed
                ok = (kStages <= S::kSfBufs || i < S::kSfBufs || mbar_wait(&empty[st2], ph2)) &&
                     mbar_wait(&full[st], ph);
                if (!ok) {
                    done = i;
                    break;
                }
                tc_fence_after();
                const uint64_t wd = smem_desc_sw128(smem_addr(sW + st * kWsRows * 128));
                const uint64_t xd = smem_desc_sw128(smem_addr(sX + st * NT * 128));
                const uint64_t wsd = smem_desc_scales(smem_addr(sWs + st * S::kScaleBytes));
                const uint64_t xsd = smem_desc_scales(smem_addr(sXs + st * S::kScaleBytes));
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
                    if (j / 2 < tiles)
                        mma_fp4_ss<false>(tmem, wd + 2 * j, xd + 2 * j, j & 1 ? id2 : id0, sfw + 4 * (j / 2),
                                          sfx + 4 * (j / 2) + off, (i | j) != 0);
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
        if (p.early)
            pdl_wait();     // before Y is written
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

    auto store = [&](int c, int n, float v) {
        const size_t at = (size_t)(tile.z + c) * p.N + n;
        if (p.y_fp32)
            reinterpret_cast<float *>(p.y)[at] = v;
        else
            reinterpret_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16_rn(v);
    };
    if (warp < 4) {
        const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
        const int n = wt * kWsRows + threadIdx.x;
        for (int c = 0; c < tile.w; c += 32) {
            uint32_t v[32];
            __syncwarp();   // the stores before may have parted the warp
            tmem_ld32_start(lane_base + c, v);
            tmem_ld32_finish(v);
#pragma unroll
            for (int i = 0; i < 32; i++) {
                if (c + i < tile.w) {
                    if (p.split > 1)
                        red[(c + i) * 128 + threadIdx.x] = __uint_as_float(v[i]);
                    else if (n < p.N)
                        store(c + i, n, __uint_as_float(v[i]));
                }
            }
        }
    }
    if (p.split > 1) {
        // ---------------- the tile's rows are shared out; four weight rows a thread
        __syncthreads();
        cluster_sync();
        const int c0 = tile.w * rank / p.split, c1 = tile.w * (rank + 1) / p.split;
        for (int i = threadIdx.x; i < (c1 - c0) * 32; i += kMsThreads) {
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
            const int n = wt * kWsRows + r4;
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (n + e < p.N)
                    store(c, n + e, vv[e]);
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

// ---------------------------------------------------------------- weight gradient
// Items (expert, 256 x 256 of its gradient).  The contraction runs over the
// expert's blocks of 128 rows, whose padding is zeros; a stage takes two of
// them, the last one may hold one of the next expert's as well, which is not
// multiplied.  An expert without rows gets zeros.
struct WgradParams {
    const int32_t *first_block;
    int E, N, K;
    int mpairs, ntiles;
    void *dw;
    int dw_fp32;
    uint32_t *ctl;
};

__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *src, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"((uint64_t)map),
                 "r"(smem_addr(src)), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

template <int BN>
__global__ void __launch_bounds__(kTlThreads, 1) __cluster_dims__(2, 1, 1)
    moe_wgrad_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ CUtensorMap tm_sa, const __grid_constant__ CUtensorMap tm_sb,
                     const __grid_constant__ CUtensorMap tm_y, const WgradParams p)
{
    using S = TlShape<false, BN>;
    constexpr int kStages = S::kStages;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *sA = smem, *sB = sA + kStages * S::kABytes, *sOut = sB + kStages * S::kBBytes;
    uint8_t *sSa = sOut + kTlEpiWarps * kTlStoreBytes, *sSb = sSa + kStages * S::kSaBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(sSb + kStages * S::kSbBytes);
    uint64_t *empty = full + kStages, *acc_full = empty + kStages, *acc_empty = acc_full + 2;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(acc_empty + 2);
    volatile int *s_abort = reinterpret_cast<volatile int *>(s_tmem + 1);
    volatile uint32_t *s_loaded = s_tmem + 2, *s_issued = s_tmem + 3;   // stages copied and multiplied

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int crank = (int)cluster_ctarank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; s++) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&acc_full[0], 1);
        mbar_init(&acc_full[1], 1);
        mbar_init(&acc_empty[0], 2 * kTlEpiWarps);
        mbar_init(&acc_empty[1], 2 * kTlEpiWarps);
        *s_abort = 0;
        *s_loaded = 0;
        *s_issued = 0;
        mbar_fence_init();
    }
    if (warp == kTlEpiWarps + 1)
        tmem_alloc_pair(s_tmem, S::kTmemCols);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers and TMEM before anything of the pair touches them
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    pdl_wait();
    pdl_launch_dependents();

    const int cid = (int)cluster_id_x(), ncl = (int)cluster_count_x();
    const int per = p.mpairs * p.ntiles;
    const int64_t ntot = (int64_t)p.E * per;
    auto fail = [&]() {
        record_status(p.ctl, NVFP4_ERR_TIMEOUT);
        *s_abort = 1;
    };
    auto aborted = [&]() { return __any_sync(0xffffffffu, *s_abort); };

    if (warp == kTlEpiWarps) {
        if (elect_one()) {
            uint32_t it = 0;
            for (int64_t t = cid; t < ntot && !*s_abort; t += ncl) {
                const int e = (int)(t / per), i = (int)(t % per), mt = 2 * (i / p.ntiles) + crank, nt = i % p.ntiles;
                const int b0 = p.first_block[e], b1 = p.first_block[e + 1];
                for (int b = b0; b < b1; b += 2, it++) {
                    const int st = it % kStages;
                    if (!mbar_wait(&empty[st], ((it / kStages) & 1) ^ 1)) {
                        fail();
                        break;
                    }
                    const uint32_t bar = cluster_addr(&full[st], 0);
                    if (crank == 0)
                        mbar_arrive_expect_tx(&full[st], 2 * S::kStageBytes);
                    tma_load_2d_pair(sA + st * S::kABytes, &tm_a, bar, b * (kMoeBlock / 2), mt * 128);
                    tma_load_2d_pair(sB + st * S::kBBytes, &tm_b, bar, b * (kMoeBlock / 2), nt * BN + crank * (BN / 2));
                    tma_load_3d_pair(sSa + st * S::kSaBytes, &tm_sa, bar, 0, b, mt);
                    tma_load_3d_pair(sSb + st * S::kSbBytes, &tm_sb, bar, 0, b, nt * BN / 128);
                }
            }
            // every stage released before leaving: the leader's commits must not arrive at a CTA that is gone
            for (int k = 0; k < kStages && !*s_abort; k++) {
                const uint32_t i2 = it + k;
                if (i2 >= (uint32_t)kStages && !mbar_wait(&empty[i2 % kStages], ((i2 / kStages) & 1) ^ 1))
                    fail();
            }
            *s_loaded = it;
        }
    } else if (warp == kTlEpiWarps + 1) {
        if (crank == 0 && elect_one()) {
            constexpr uint32_t id0 = idesc_fp4(256, BN, 1, 0), id2 = idesc_fp4(256, BN, 1, 2);
            uint32_t it = 0, lt = 0;
            for (int64_t t = cid; t < ntot && !*s_abort; t += ncl) {
                const int e = (int)(t / per);
                const int b0 = p.first_block[e], b1 = p.first_block[e + 1];
                if (b0 == b1)
                    continue;
                if (S::kShared ? lt >= 1 && !mbar_wait(&acc_empty[0], (lt - 1) & 1)
                               : lt >= 2 && !mbar_wait(&acc_empty[lt & 1], (lt / 2 - 1) & 1)) {
                    fail();
                    break;
                }
                tc_fence_after();
                const uint32_t acc = tmem + (lt & 1 ? S::kAcc1 : 0);
                bool ok = true;
                for (int b = b0; b < b1; b += 2, it++) {
                    const int st = it % kStages;
                    constexpr uint32_t kB = S::kSfBufs;
                    if ((it >= kB && !mbar_wait(&empty[(it - kB) % kStages], ((it - kB) / kStages) & 1)) ||
                        !mbar_wait(&full[st], (it / kStages) & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = smem_desc_sw128(smem_addr(sA + st * S::kABytes));
                    const uint64_t bd = smem_desc_sw128(smem_addr(sB + st * S::kBBytes));
                    const uint64_t sad = smem_desc_scales(smem_addr(sSa + st * S::kSaBytes));
                    const uint64_t sbd = smem_desc_scales(smem_addr(sSb + st * S::kSbBytes));
                    const uint32_t sfa = tmem + S::kSfCol + it % S::kSfBufs * S::kSf, sfb = sfa + S::kSfA;
                    const int blocks = min(2, b1 - b);
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        if (k < blocks) {
                            tmem_cp_scales_pair(sfa + 4 * k, sad + k * 32);
#pragma unroll
                            for (int r = 0; r < S::kBRowTiles; r++)
                                tmem_cp_scales_pair(sfb + 4 * (k * S::kBRowTiles + r), sbd + (r * S::kTiles + k) * 32);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        if (j / 2 < blocks)
                            mma_fp4_pair<false>(acc, ad + 2 * j, bd + 2 * j, j & 1 ? id2 : id0, sfa + 4 * (j / 2),
                                                sfb + 4 * (j / 2) * S::kBRowTiles, (b - b0 + j) != 0);
                    }
                    mma_commit_pair(&empty[st]);
                    if (b + 2 >= b1)
                        mma_commit_pair(&acc_full[lt & 1]);
                }
                if (!ok) {
                    fail();
                    break;
                }
                lt++;
            }
            *s_issued = it;
        }
    } else {
        // ---------------- epilogue: warp w has lanes 32 (w % 4) .. + 31 and every other 32 columns, the columns
        // that both accumulators use first
        constexpr int kChunks = BN / 32, kSharedChunks = S::kShared / 32;
        const int quad = warp & 3, half = warp >> 2;
        const uint32_t bar0 = cluster_addr(&acc_empty[0], 0), bar1 = cluster_addr(&acc_empty[1], 0);
        uint8_t *out = sOut + warp * kTlStoreBytes;
        uint32_t lt = 0;
        for (int64_t t = cid; t < ntot && !aborted(); t += ncl) {
            const int e = (int)(t / per), i0 = (int)(t % per), mt = 2 * (i0 / p.ntiles) + crank, nt = i0 % p.ntiles;
            const bool empty_group = p.first_block[e] == p.first_block[e + 1];
            const int m0 = mt * 128 + quad * 32;
            if (!empty_group) {
                if (!mbar_wait_warp(&acc_full[lt & 1], (lt >> 1) & 1)) {
                    fail();
                    break;
                }
                tc_fence_after();
            }
            const uint32_t acc = tmem + ((uint32_t)(quad * 32) << 16) + (lt & 1 ? S::kAcc1 : 0);
            const int first = lt & 1 ? 0 : kChunks - kSharedChunks;
            uint32_t buf[2][32];
            if (!empty_group)
                tmem_ld32_start(acc + (first + half) % kChunks * 32, buf[0]);
#pragma unroll
            for (int i = 0; i < kChunks / 2; i++) {
                uint32_t(&v)[32] = buf[i & 1];
                __syncwarp();   // the stores before may have parted the warp
                if (!empty_group) {
                    tmem_ld32_finish(v);
                    if (i + 1 < kChunks / 2)
                        tmem_ld32_start(acc + (first + half + 2 * (i + 1)) % kChunks * 32, buf[(i + 1) & 1]);
                    if (S::kShared ? half + 2 * i < kSharedChunks && half + 2 * i + 2 >= kSharedChunks
                                   : i + 1 == kChunks / 2) {
                        // this warp's part of the shared columns (of all) is in registers
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0)
                            mbar_arrive_cluster(S::kShared || !(lt & 1) ? bar0 : bar1);
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 32; c++)
                        v[c] = 0u;
                }
                const int n0 = nt * BN + (first + half + 2 * i) % kChunks * 32;
                if (m0 >= p.N || n0 >= p.K)
                    continue;
                // 64 bytes a row at a time: all of the chunk in bf16, half of it in FP32
                auto stage_and_store = [&](const uint4 (&w)[4], int n) {
                    if (lane == 0)
                        bulk_wait_read<0>();   // the store before has read the staging
                    __syncwarp();
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        *reinterpret_cast<uint4 *>(out + lane * 64 + ((q ^ (lane >> 1 & 3)) * 16)) = w[q];
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_3d(&tm_y, out, n, m0, e);
                        bulk_commit();
                    }
                };
                uint4 w[4];
                if (p.dw_fp32) {
#pragma unroll
                    for (int h = 0; h < 2; h++) {
#pragma unroll
                        for (int q = 0; q < 4; q++)
                            w[q] = make_uint4(v[16 * h + 4 * q], v[16 * h + 4 * q + 1], v[16 * h + 4 * q + 2],
                                              v[16 * h + 4 * q + 3]);
                        if (n0 + 16 * h < p.K)
                            stage_and_store(w, n0 + 16 * h);
                    }
                } else {
#pragma unroll
                    for (int q = 0; q < 4; q++)
                        w[q] = make_uint4(pack2(v[8 * q], v[8 * q + 1]), pack2(v[8 * q + 2], v[8 * q + 3]),
                                          pack2(v[8 * q + 4], v[8 * q + 5]), pack2(v[8 * q + 6], v[8 * q + 7]));
                    stage_and_store(w, n0);
                }
            }
            lt += empty_group ? 0 : 1;
        }
        if (lane == 0)
            bulk_wait_read<0>();
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (crank == 0 && warp == kTlEpiWarps + 1 && *s_abort) {
        // after a wait that gave up: copies on their way land, and MMAs issued are done, before either CTA leaves
        const uint32_t loaded = *s_loaded, issued = *s_issued;
        ring_drain(full, kStages, loaded > (uint32_t)kStages ? loaded - kStages : 0u, loaded);
        if (issued > 0)
            ring_drain(empty, kStages, issued - 1, issued);
        __syncwarp();
    }
    cluster_sync();  // neither CTA leaves while the other may still signal or read it
    if (warp == kTlEpiWarps + 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, S::kTmemCols);
    }
}

// ---------------------------------------------------------------- launches
// The experts' codes: K/2 bytes x N rows x E, a box of 128 rows of one expert.
cudaError_t weight_map(CUtensorMap *map, const MoeGemmArgs &a)
{
    const uint64_t row = (uint64_t)a.K / 2;
    return encode_tensor_map_3d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w_codes, {row, (uint64_t)a.N, (uint64_t)a.E},
                                {row, row * (uint64_t)a.N}, {128, 128, 1}, CU_TENSOR_MAP_SWIZZLE_128B);
}

MoeParams params(const MoeGemmArgs &a)
{
    MoeParams p = {};
    p.header = a.header;
    p.tiles = a.tiles;
    p.x_scales = a.x_scales;
    p.w_scales = a.w_scales;
    p.N = (int)a.N;
    p.ksteps = (int)((a.K + 255) / 256);
    p.ktiles = (int)((a.K + 127) / 128);
    p.wrows = (int)((a.N + 127) / 128);
    p.split = 1;
    p.early = a.after_quantise ? 1 : 0;
    p.y = a.y;
    p.y_fp32 = a.y_fp32 ? 1 : 0;
    p.ctl = a.ctl;
    return p;
}

template <int TR, bool kF32>
cudaError_t run_moe_tile(const MoeGemmArgs &a, cudaStream_t s, const DeviceInfo &dev)
{
    using S = TlShape<false, TR>;
    const uint64_t row = (uint64_t)a.K / 2;
    MoeParams p = params(a);
    CUtensorMap tw, tx, tsw, tsx;
    cudaError_t e = weight_map(&tw, a);
    if (e == cudaSuccess)
        e = encode_tensor_map_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.x_codes, row, (uint64_t)a.padded_rows, row, 128,
                                 TR / 2, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess)
        e = encode_scale_map(&tsw, a.w_scales, (uint64_t)p.ktiles, (uint64_t)a.E * p.wrows, S::kTiles, 1);
    if (e == cudaSuccess)
        e = encode_scale_map(&tsx, a.x_scales, (uint64_t)p.ktiles, (uint64_t)a.padded_rows / 128, S::kTiles,
                             S::kBRowTiles);
    if (e == cudaSuccess)
        e = allow_smem<moe_tile_kernel<TR, kF32>>(S::kSmem, dev);
    if (e != cudaSuccess)
        return e;
    p.wtiles = (int)((a.N + 255) / 256);
    const int64_t most = a.max_tiles * p.wtiles;
    return launch_dependent(moe_tile_kernel<TR, kF32>, dim3(2 * (unsigned)std::min<int64_t>(most, dev.num_sms / 2)),
                            kTlThreads, S::kSmem, s, tw, tx, tsw, tsx, p);
}

template <int NT>
cudaError_t run_moe_stream(const MoeGemmArgs &a, cudaStream_t s, const DeviceInfo &dev)
{
    using S = WsShape<false, NT, kCodes>;
    const uint64_t row = (uint64_t)a.K / 2;
    MoeParams p = params(a);
    CUtensorMap tw, tx, tf;
    cudaError_t e = weight_map(&tw, a);
    if (e == cudaSuccess)
        e = encode_tensor_map_2d(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.x_codes, row, (uint64_t)a.padded_rows, row, 128,
                                 NT, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess)
        e = encode_tensor_map_2d(&tf, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.x_codes, row, (uint64_t)a.padded_rows, row, 128,
                                 kMsFew, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess)
        e = allow_smem<moe_stream_kernel<NT>>(kWsSmem, dev);
    if (e != cudaSuccess)
        return e;
    p.wtiles = p.wrows;
    const int64_t items = a.max_tiles * p.wtiles;
    p.split = ws_split(items, a.K, dev.num_sms);
    const int nk = (p.ksteps + p.split - 1) / p.split;
    p.stages = S::stages(nk);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items * p.split));
    cfg.blockDim = dim3(kMsThreads);
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
    return cudaLaunchKernelEx(&cfg, moe_stream_kernel<NT>, tw, tx, tf, p);
}

}  // namespace

cudaError_t launch_moe_gemm(const MoeGemmArgs &a, cudaStream_t s, const DeviceInfo &dev)
{
    switch (a.tile_rows) {
    case 64:
        return run_moe_stream<64>(a, s, dev);
    case 128:
        return a.y_fp32 ? run_moe_tile<128, true>(a, s, dev) : run_moe_tile<128, false>(a, s, dev);
    default:
        return a.y_fp32 ? run_moe_tile<256, true>(a, s, dev) : run_moe_tile<256, false>(a, s, dev);
    }
}

cudaError_t launch_moe_wgrad(const MoeWgradArgs &a, cudaStream_t s, const DeviceInfo &dev)
{
    constexpr int BN = 256;
    using S = TlShape<false, BN>;
    const uint64_t row = (uint64_t)a.padded_rows / 2, kt = (uint64_t)a.padded_rows / 128;
    const uint64_t esize = a.dw_fp32 ? 4 : 2;
    CUtensorMap ta, tb, tsa, tsb, ty;
    cudaError_t e = encode_tensor_map_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.a_codes, row, (uint64_t)a.N, row, 128, 128,
                                         CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess)
        e = encode_tensor_map_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.x_codes, row, (uint64_t)a.K, row, 128, BN / 2,
                                 CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess)
        e = encode_scale_map(&tsa, a.a_scales, kt, (uint64_t)(a.N + 127) / 128, S::kTiles, 1);
    if (e == cudaSuccess)
        e = encode_scale_map(&tsb, a.x_scales, kt, (uint64_t)(a.K + 127) / 128, S::kTiles, S::kBRowTiles);
    if (e == cudaSuccess)
        e = encode_tensor_map_3d(&ty, a.dw_fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.dw,
                                 {(uint64_t)a.K, (uint64_t)a.N, (uint64_t)a.E},
                                 {(uint64_t)a.K * esize, (uint64_t)a.K * esize * (uint64_t)a.N},
                                 {(uint32_t)(64 / esize), 32, 1}, CU_TENSOR_MAP_SWIZZLE_64B);
    if (e == cudaSuccess)
        e = allow_smem<moe_wgrad_kernel<BN>>(S::kSmem, dev);
    if (e != cudaSuccess)
        return e;
    WgradParams p;
    p.first_block = a.first_block;
    p.E = a.E;
    p.N = (int)a.N;
    p.K = (int)a.K;
    p.mpairs = (int)((a.N + 255) / 256);
    p.ntiles = (int)((a.K + BN - 1) / BN);
    p.dw = a.dw;
    p.dw_fp32 = a.dw_fp32 ? 1 : 0;
    p.ctl = a.ctl;
    const int64_t items = (int64_t)a.E * p.mpairs * p.ntiles;
    return launch_dependent(moe_wgrad_kernel<BN>, dim3(2 * (unsigned)std::min<int64_t>(items, dev.num_sms / 2)), kTlThreads,
                            S::kSmem, s, ta, tb, tsa, tsb, ty, p);
}

}  // namespace nvfp4
