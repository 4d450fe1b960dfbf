// gemm_w4a4_tile.cu -- the W4A4 product for many tokens: CTA pairs, one
// 256 x BN output tile per pair at a time.
//
// At 4 bits the tensor cores consume operands faster than a single CTA can be
// fed: a stage of 256 elements of K keeps them busy for about 512 cycles on
// a 128 x 256 tile, and such a tile would need 48 KB per stage.  The two CTAs
// of a pair therefore run one MMA (cta_group::2): each holds its 128 rows of A
// and half of the rows of B (32 KB per stage), and the instruction reads B from
// both.  The accumulator (128 lanes x BN columns in each CTA) is drained to
// registers at once when the K loop ends, so that the next tile's MMAs start
// while this one's rows are converted and stored.
//
// Scales: each CTA loads the scale tiles of its own A rows and of all B rows;
// the leader's copies to TMEM (cta_group::2) work on both CTAs' memory.
//
// What bounds it (16384 x 18944 x 3584, MXFP4: 320 us, 6.9 PFLOP/s; under load
// for longer the power limit lowers the clock from 2.07 to about 1.85 GHz and it
// takes 335 to 360).  A tile of 14 stages takes about 9500 cycles: 14 x 516 of
// MMAs (128 cycles for each 64 elements of K), 700 in which the copies of the
// next stage are late because the stores of the tile before share their way (no
// store: 8800), about 450 to hand the accumulator over, the rest in the issuing
// thread.  Measured and left out: B multicast over two pairs (a quarter less to
// read from L2, but clusters of four fill 144 of 152 SMs: 334 us), stores spread
// over the next tile's K loop (no change), no reuse of TMEM columns between the
// accumulators at 224 columns (fewer operations a byte), five stages with 32 KB
// for the stores (341 us).
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace nvfp4 {

using namespace sm100;

namespace {

constexpr int kTlEpiWarps = 8;
constexpr int kTlThreads = 32 * (kTlEpiWarps + 2);  // + copies, MMA
constexpr int kTlGroup = 8;                          // raster: pairs of row tiles per group
constexpr int kTlStoreBytes = 2048;                  // a warp's staging for TMA stores: 32 rows of 64 bytes

struct TileParams {
    const float *a_ts, *w_ts;
    int M, N;
    int ksteps;  // stages over K
    int mpairs, ntiles;
    void *y;
    int y_fp32, tma_store;
    uint32_t *ctl;
};

template <bool kNv, int BN>
struct TlShape {
    static constexpr int kTiles = kNv ? 4 : 2;                 // scale tiles per stage and 128 rows
    static constexpr int kBRowTiles = (BN + 127) / 128;         // scale tiles over B's rows
    static constexpr int kABytes = 128 * 128, kBBytes = BN / 2 * 128;
    static constexpr int kSaBytes = kTiles * 512, kSbBytes = kBRowTiles * kTiles * 512;
    static constexpr int kStageBytes = kABytes + kBBytes + kSaBytes + kSbBytes;
    static constexpr int kFixed = kTlEpiWarps * kTlStoreBytes + 512;
    static constexpr int kFit = (232448 - kFixed) / kStageBytes;
    static constexpr int kStages = kFit < 8 ? kFit : 8;
    static constexpr size_t kSmem = kFixed + (size_t)kStages * kStageBytes;
    static constexpr int kSfA = kTiles * 4, kSfB = kTiles * kBRowTiles * 4, kSf = kSfA + kSfB;
    static constexpr int kTmemCols = 512;
    // columns: accumulator 0 at 0, accumulator 1 at BN - kShared, then two stages' scales (more would take
    // columns from the accumulators: 343 us instead of 334 at 16384 x 18944 x 3584)
    static constexpr int kSfBufs = 2;
    static constexpr int kOver = 2 * BN + kSfBufs * kSf - kTmemCols;
    static constexpr int kShared = kOver > 64 ? (kOver + 31) / 32 * 32 : kOver > 0 ? 64 : 0;
    static constexpr int kAcc1 = BN - kShared, kSfCol = 2 * BN - kShared;
    static_assert(kSfCol + kSfBufs * kSf <= kTmemCols && kSfBufs < kStages && (kShared == 0 || kShared >= 64),
                  "TMEM; each half of the epilogue has a shared chunk");
};

__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}

// Loads whose bytes are counted on the pair leader's barrier.
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const CUtensorMap *map, uint32_t bar, int x, int y)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4}], [%2];" ::"r"(smem_addr(dst)),
        "l"((uint64_t)map), "r"(bar), "r"(x), "r"(y)
        : "memory");
}

__device__ __forceinline__ void tma_load_3d_pair(void *dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, "
        "%5}], [%2];" ::"r"(smem_addr(dst)),
        "l"((uint64_t)map), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *src, int x, int y)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"((uint64_t)map),
                 "r"(smem_addr(src)), "r"(x), "r"(y)
                 : "memory");
}

__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read()
{
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// Arrival on a barrier of the pair.  What it hands over is TMEM that has been
// read (tcgen05.wait::ld), so a release of this thread's memory operations at
// cluster scope is not needed; it would wait for the stores in flight (1500
// cycles between two tiles).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tmem_alloc_pair(uint32_t *dst, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

__device__ __forceinline__ void tmem_cp_scales_pair(uint32_t taddr, uint64_t desc)
{
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}

template <bool kBlock16>
__device__ __forceinline__ void mma_fp4_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t sa_tmem, uint32_t sb_tmem, uint32_t accumulate)
{
    if (kBlock16)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
                d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sa_tmem), "r"(sb_tmem)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(
                d_tmem),
            "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(sa_tmem), "r"(sb_tmem)
            : "memory");
}

// One arrival on the barrier at bar's offset in both CTAs when the MMAs (and
// scale copies) issued so far have completed.
__device__ __forceinline__ void mma_commit_pair(uint64_t *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_addr(bar)),
        "h"((uint16_t)3)
        : "memory");
}

__device__ __forceinline__ uint32_t pack2(uint32_t a, uint32_t b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(a), __uint_as_float(b));
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Raster: groups of kTlGroup row-tile pairs, the pair index fastest.
__device__ __forceinline__ void tile_at(int t, int mpairs, int ntiles, int &mp, int &nt)
{
    const int per = kTlGroup * ntiles, g = t / per, i = t % per;
    const int gm = min(kTlGroup, mpairs - g * kTlGroup);
    mp = g * kTlGroup + i % gm;
    nt = i / gm;
}

template <bool kNv, int BN>
__global__ void __launch_bounds__(kTlThreads, 1) __cluster_dims__(2, 1, 1)
    w4a4_tile_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ CUtensorMap tm_sa, const __grid_constant__ CUtensorMap tm_sb,
                     const __grid_constant__ CUtensorMap tm_y, const TileParams p)
{
    using S = TlShape<kNv, BN>;
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
    const int ntot = p.mpairs * p.ntiles;
    auto fail = [&]() {
        record_status(p.ctl, NVFP4_ERR_TIMEOUT);
        *s_abort = 1;
    };
    auto aborted = [&]() { return __any_sync(0xffffffffu, *s_abort); };

    if (warp == kTlEpiWarps) {
        // ---------------- copies: this CTA's half of each operand
        if (elect_one()) {
            uint32_t it = 0;
            for (int t = cid; t < ntot && !*s_abort; t += ncl) {
                int mp, nt;
                tile_at(t, p.mpairs, p.ntiles, mp, nt);
                const int mt = 2 * mp + crank;
                for (int ks = 0; ks < p.ksteps; ks++, it++) {
                    const int st = it % kStages;
                    if (!mbar_wait(&empty[st], ((it / kStages) & 1) ^ 1)) {
                        fail();
                        break;
                    }
                    const uint32_t bar = cluster_addr(&full[st], 0);
                    if (crank == 0)
                        mbar_arrive_expect_tx(&full[st], 2 * S::kStageBytes);
                    tma_load_2d_pair(sA + st * S::kABytes, &tm_a, bar, ks * 128, mt * 128);
                    tma_load_2d_pair(sB + st * S::kBBytes, &tm_b, bar, ks * 128, nt * BN + crank * (BN / 2));
                    tma_load_3d_pair(sSa + st * S::kSaBytes, &tm_sa, bar, 0, ks * S::kTiles, mt);
                    tma_load_3d_pair(sSb + st * S::kSbBytes, &tm_sb, bar, 0, ks * S::kTiles, nt * BN / 128);
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
        // ---------------- MMA, by one thread of the pair's leader.  What this loop takes per stage bounds
        // narrow tiles: 460 cycles, 100 less than with all lanes in it and votes.
        if (crank == 0 && elect_one()) {
            constexpr uint32_t id0 = idesc_fp4(256, BN, kNv ? 0 : 1, 0), id2 = idesc_fp4(256, BN, kNv ? 0 : 1, 2);
            uint32_t it = 0, lt = 0;
            for (int t = cid; t < ntot && !*s_abort; t += ncl, lt++) {
                int mp, nt;
                tile_at(t, p.mpairs, p.ntiles, mp, nt);
                // the shared columns of the accumulator before this one have been read, or without
                // shared columns the accumulator that this tile takes (barriers for each accumulator:
                // either side may be two tiles ahead of the other)
                if (S::kShared ? lt >= 1 && !mbar_wait(&acc_empty[0], (lt - 1) & 1)
                               : lt >= 2 && !mbar_wait(&acc_empty[lt & 1], (lt / 2 - 1) & 1)) {
                    fail();
                    break;
                }
                tc_fence_after();
                const uint32_t acc = tmem + (lt & 1 ? S::kAcc1 : 0);
                // 192 rows: every other tile begins in the middle of a scale tile, two columns on
                const uint32_t sb_off = (uint32_t)(nt * BN % 128) / 32;
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
                    for (int j = 0; j < 4; j++) {
                        const int k = kNv ? j : j / 2;
                        const uint32_t sa = sfa + 4 * k, sb = sfb + 4 * k * S::kBRowTiles + sb_off;
                        mma_fp4_pair<kNv>(acc, ad + 2 * j, bd + 2 * j, !kNv && (j & 1) ? id2 : id0, sa, sb,
                                          (ks | j) != 0);
                    }
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
        // ---------------- epilogue: warp w has lanes 32 (w % 4) .. + 31 and every other 32 columns, the columns
        // that both accumulators use first
        constexpr int kChunks = BN / 32, kSharedChunks = S::kShared / 32;
        const int quad = warp & 3, half = warp >> 2;
        const uint32_t bar0 = cluster_addr(&acc_empty[0], 0), bar1 = cluster_addr(&acc_empty[1], 0);
        uint8_t *out = sOut + warp * kTlStoreBytes;
        const float s_a = p.a_ts ? *p.a_ts : 1.0f, s_w = p.w_ts ? *p.w_ts : 1.0f;
        const bool scaled = p.a_ts || p.w_ts;
        uint32_t lt = 0;
        for (int t = cid; t < ntot && !aborted(); t += ncl, lt++) {
            int mp, nt;
            tile_at(t, p.mpairs, p.ntiles, mp, nt);
            if (!mbar_wait_warp(&acc_full[lt & 1], (lt >> 1) & 1)) {
                fail();
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(quad * 32) << 16) + (lt & 1 ? S::kAcc1 : 0);
            const int m0 = (2 * mp + crank) * 128 + quad * 32;
            // accumulator 0 ends with the shared columns, accumulator 1 begins with them
            const int first = lt & 1 ? 0 : kChunks - kSharedChunks;
            uint32_t buf[2][32];
            tmem_ld32_start(acc + (first + half) % kChunks * 32, buf[0]);
#pragma unroll
            for (int i = 0; i < kChunks / 2; i++) {
                uint32_t(&v)[32] = buf[i & 1];
                __syncwarp();   // the stores before may have parted the warp
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
                const int n0 = nt * BN + (first + half + 2 * i) % kChunks * 32;
                if (m0 >= p.M || n0 >= p.N)
                    continue;
                if (scaled) {
                    // one after the other: the product of two small tensor scales may underflow
#pragma unroll
                    for (int c = 0; c < 32; c++)
                        v[c] = __float_as_uint(__fmul_rn(__fmul_rn(__uint_as_float(v[c]), s_a), s_w));
                }
                if (p.tma_store) {
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
                            tma_store_2d(&tm_y, out, n, m0);
                            bulk_commit();
                        }
                    };
                    uint4 w[4];
                    if (p.y_fp32) {
#pragma unroll
                        for (int h = 0; h < 2; h++) {
#pragma unroll
                            for (int q = 0; q < 4; q++)
                                w[q] = make_uint4(v[16 * h + 4 * q], v[16 * h + 4 * q + 1], v[16 * h + 4 * q + 2],
                                                  v[16 * h + 4 * q + 3]);
                            if (n0 + 16 * h < p.N)
                                stage_and_store(w, n0 + 16 * h);
                        }
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; q++)
                            w[q] = make_uint4(pack2(v[8 * q], v[8 * q + 1]), pack2(v[8 * q + 2], v[8 * q + 3]),
                                              pack2(v[8 * q + 4], v[8 * q + 5]), pack2(v[8 * q + 6], v[8 * q + 7]));
                        stage_and_store(w, n0);
                    }
                } else if (m0 + lane < p.M) {
                    // rows of Y that do not start on 16-byte boundaries: a lane writes its row element by element,
                    // and the stores bound the kernel (4096 x 18945 x 3584: bf16 695 us, FP32 563; 18944: 85 and 104)
                    const size_t at = (size_t)(m0 + lane) * p.N + n0;
#pragma unroll
                    for (int c = 0; c < 32; c++) {
                        if (n0 + c < p.N) {
                            if (p.y_fp32)
                                reinterpret_cast<uint32_t *>(p.y)[at + c] = v[c];
                            else
                                reinterpret_cast<__nv_bfloat16 *>(p.y)[at + c] =
                                    __float2bfloat16_rn(__uint_as_float(v[c]));
                        }
                    }
                }
            }
        }
        if (lane == 0)
            bulk_wait_read<0>();
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (crank == 0 && warp == kTlEpiWarps + 1 && *s_abort) {
        // after a wait that gave up: copies on their way land, and MMAs issued are done, before either CTA leaves (the
        // leader's barriers count both CTAs' copies; what the other one issued beyond them is as old as its own wait)
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

template <bool kNv, int BN>
cudaError_t run_tile(const W4A4Args &a, cudaStream_t s, const DeviceInfo &dev)
{
    using S = TlShape<kNv, BN>;
    const uint64_t row = (uint64_t)a.K / 2;
    const uint64_t kt = ((uint64_t)a.K + (kNv ? 63 : 127)) / (kNv ? 64 : 128);
    CUtensorMap ta, tb, tsa, tsb, ty;
    cudaError_t e = encode_tensor_map_2d(&ta, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.a_codes, row, (uint64_t)a.M, row, 128,
                                         128, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess)
        e = encode_tensor_map_2d(&tb, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w_codes, row, (uint64_t)a.N, row, 128, BN / 2,
                                 CU_TENSOR_MAP_SWIZZLE_128B);
    if (e == cudaSuccess)
        e = encode_scale_map(&tsa, a.a_scales, kt, (uint64_t)(a.M + 127) / 128, S::kTiles, 1);
    if (e == cudaSuccess)
        e = encode_scale_map(&tsb, a.w_scales, kt, (uint64_t)(a.N + 127) / 128, S::kTiles, S::kBRowTiles);
    const int esize = a.y_fp32 ? 4 : 2;
    const bool tma_store = a.N * esize % 16 == 0;
    if (e == cudaSuccess)
        e = tma_store ? encode_tensor_map_2d(&ty, a.y_fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                                           : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                                             a.y, (uint64_t)a.N, (uint64_t)a.M, (uint64_t)a.N * esize, 64 / esize, 32,
                                             CU_TENSOR_MAP_SWIZZLE_64B)
                      : (ty = ta, cudaSuccess);
    if (e == cudaSuccess)
        e = allow_smem<w4a4_tile_kernel<kNv, BN>>(S::kSmem, dev);
    if (e != cudaSuccess)
        return e;
    TileParams p;
    p.a_ts = a.a_ts;
    p.w_ts = a.w_ts;
    p.M = (int)a.M;
    p.N = (int)a.N;
    p.ksteps = (int)((a.K + 255) / 256);
    p.mpairs = (int)((a.M + 255) / 256);
    p.ntiles = (int)((a.N + BN - 1) / BN);
    p.y = a.y;
    p.y_fp32 = a.y_fp32 ? 1 : 0;
    p.tma_store = tma_store ? 1 : 0;
    p.ctl = a.ctl;
    const int64_t tiles = (int64_t)p.mpairs * p.ntiles;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (unsigned)std::min<int64_t>(tiles, dev.num_sms / 2));
    cfg.blockDim = dim3(kTlThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, w4a4_tile_kernel<kNv, BN>, ta, tb, tsa, tsb, ty, p);
}

// Width of the tiles: the one whose waves of pairs take least.  A stage of 256
// elements of K takes 0.28 us at 256 columns and 0.23 at 192 (bound by the MMAs
// and, in NVFP4, twelve scale copies beside them), 0.23 at 128 (by the issuing
// thread), a tile about 0.7 us besides.  2048 x 3584 x 18944: 50.4 us in 112
// tiles of 256, 39.6 in 152 of 192.
template <bool kNv>
cudaError_t run_widths(const W4A4Args &a, cudaStream_t s, const DeviceInfo &dev)
{
    const int widths[3] = {256, 192, 128};
    const double per_stage[3] = {0.28, 0.23, 0.23};
    const int64_t ksteps = (a.K + 255) / 256, pairs = dev.num_sms / 2;
    int best = 0;
    double least = 0;
    for (int i = 0; i < 3; i++) {
        const int64_t tiles = ((a.M + 255) / 256) * ((a.N + widths[i] - 1) / widths[i]);
        const double t = (double)((tiles + pairs - 1) / pairs) * (ksteps * per_stage[i] + 0.7);
        if (i == 0 || t < least) {
            best = i;
            least = t;
        }
    }
    return best == 0 ? run_tile<kNv, 256>(a, s, dev) : best == 1 ? run_tile<kNv, 192>(a, s, dev)
                                                                 : run_tile<kNv, 128>(a, s, dev);
}

}  // namespace

cudaError_t launch_w4a4_tile(const W4A4Args &a, cudaStream_t s, const DeviceInfo &dev)
{
    return a.nvfp4 ? run_widths<true>(a, s, dev) : run_widths<false>(a, s, dev);
}

}  // namespace nvfp4
