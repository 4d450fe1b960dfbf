// gemm_int8.cu -- Y[m][n] = s_m s_n sum_k q[m][k] w[n][k] with 8-bit integers q
// and w and one FP32 scale for each token and output channel.
//
// This chip's 8-bit integer tensor rate is far below its 16-bit one, and the
// integers -127..127 and their products are exact in fp16 and FP32, so the
// codes are multiplied as fp16 (tcgen05, FP32 accumulators): sums are exact
// while they stay below 2^24.  Beyond, an instruction adds 16 products to a running
// sum in 2^e .. 2^(e + 1); measured, each product loses what lies below 2^(e - 25) and
// the sum is rounded to the nearest step, 2^(e - 23): 4.5 steps at most, which for
// codes of one sign comes to 3e-4 of the sum at K = 18944 and 2e-3 at 131072, less
// where K is shared out.  Uniform ones measured 2e-7 with K shared by eight CTAs and
// 3e-5 without (131072: 1.4e-5, 5e-4).  Codes of either sign stay exact there: sums
// of Gaussian rows reach 2^19 and 2^20, of uniform ones 2^22 and 2^23.
//
// The weights stay 8 bits until they are next to the tensor core.  Their rows
// are the MMA's M side, whose operand may come from TMEM: warps read a stage of
// codes from shared memory, a row a thread, make fp16 of them (byte permute into
// 1024 + u, u = w + 128, minus 1152: 5 instructions for 4 weights) and store
// them to TMEM.  Shared memory then carries each weight twice as one byte, and
// not again as two bytes written and read.  Tokens are quantised to fp16
// integers by a kernel before this one and come by TMA.
//
// What bounds it.  One token through 18944 x 3584: 15.8 us on the GPU, of which the
// weights' bytes are 10; the rest is the launch, the first stage's way and the join
// of two shares.  100 tokens through 3584 x 18944: 17 us and the quantiser's 5 (bytes
// 10, MMAs 9; 37 us with one ring for codes, tokens and converted weights).  8192
// tokens through 18944 x 3584: 622 to 660 us with the quantiser from GPU to GPU, 1.69 to
// 1.79 PFLOP/s, 87 to 93 % of the library's bf16 product in a burst and 98 to 104 % of what
// it sustains (power).
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "int8_codec.cuh"
#include "internal.h"
#include "mx_codec.cuh"
#include "tile_store.cuh"
#include "w4a4_pair.cuh"

namespace nvfp4 {

namespace {

constexpr int kI8K = 128;         // elements of K a stage
constexpr int kI8Rows = 128;      // weight rows a CTA
constexpr int kI8WBytes = kI8Rows * kI8K, kI8ACols = kI8K / 2;   // a stage's codes, and its columns as fp16 in TMEM
// Warps that convert, in groups of four (32 rows each) that take turns: a stage
// takes a group longer than the MMAs of few tokens (waits, shared memory, the
// stores' completion), so two are in work at once.
constexpr int kI8Conv = 8, kI8Groups = kI8Conv / 4;

struct Int8Params {
    const float *x_scale, *w_scale;
    const void *x;   // unquantised tokens (M x K, ldx between rows)
    int64_t ldx;
    int M, N, K;
    int ksteps;
    int mtiles, ntiles;
    int split;    // streaming: CTAs of a cluster that share a tile's K
    int early;    // the weights were complete before the kernel before this one started
    void *y;
    int y_fp32;
    uint32_t *ctl;
};

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

// D[tmem] (+)= A[tmem] B[smem]^T over 16 elements of K, f16 operands.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void mma_f16_ts_pair(uint32_t d, uint32_t a, uint64_t b_desc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// A converting warp's part of a stage: row 32 (warp % 4) + lane, from the swizzled layout of a TMA copy.
__device__ __forceinline__ void convert_rows(const uint8_t *stage, uint32_t a_tmem, int warp, int lane)
{
    const int row = (warp & 3) * 32 + lane;
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; h++) {
        uint32_t v[32];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint4 q = *reinterpret_cast<const uint4 *>(stage + row * 128 + (((4 * h + j) ^ (row & 7)) << 4));
            int8x4_to_h2x2(q.x, v[8 * j], v[8 * j + 1]);
            int8x4_to_h2x2(q.y, v[8 * j + 2], v[8 * j + 3]);
            int8x4_to_h2x2(q.z, v[8 * j + 4], v[8 * j + 5]);
            int8x4_to_h2x2(q.w, v[8 * j + 6], v[8 * j + 7]);
        }
        tmem_st32(a_tmem + ((uint32_t)((warp & 3) * 32) << 16) + h * 32, v);
    }
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t local, uint32_t rank)
{
    float v;
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
                 : "=f"(v)
                 : "r"(local), "r"(rank)
                 : "memory");
    return v;
}

// v s w, where v s must not overflow by itself: sums are 2^31 in magnitude at most, so
// above 2^96 the token's scale comes last.
constexpr float kI8Wide = 0x1p96f;
__device__ __forceinline__ float scaled(float v, float s, float w)
{
    const bool wide = fabsf(s) > kI8Wide;
    return __fmul_rn(__fmul_rn(v, wide ? w : s), wide ? s : w);
}

// ---------------------------------------------------------------- few tokens
// A CTA takes 128 weight rows and NT tokens; K is split over the CTAs of a
// cluster when there are fewer tiles than CTA places, the shares added in rank
// order through distributed shared memory.  Codes, tokens and converted weights
// have rings of their own: codes are let go when they are converted, tokens and
// TMEM columns when they are multiplied.  Very few tokens are quantised by the
// CTAs themselves (each needs the whole rows for their maxima, and writes the
// part of K that it multiplies) while the first weights are on their way: a
// kernel of its own costs a launch and 1 to 2 us.
constexpr int kIsThreads = 32 * (kI8Conv + 3);  // + copies of weights, of tokens, MMA
enum Int8Tokens { kInts, kRawBf16, kRawFp32 };

template <int NT, Int8Tokens kTok>
struct IsShape {
    static constexpr bool kOwn = kTok != kInts;
    static constexpr int kCtas = NT <= 64 ? 2 : 1;        // on an SM
    static constexpr int kXBytes = NT * kI8K * 2;
    static constexpr int kTmemCols = 512 / kCtas;
    static constexpr int kAccCols = NT < 32 ? 32 : NT;
    static constexpr int kW = kOwn ? 3 : NT == 16 ? 5 : NT == 32 ? 4 : NT == 64 ? 3 : 5;   // stages of codes,
    static constexpr int kX = kOwn ? 15 : NT == 16 ? 5 : NT == 32 ? 4 : NT == 64 ? 3 : 4;  // of tokens (own: all of a CTA's)
    static constexpr int kA = NT <= 64 ? 3 : 5;                                            // of converted weights
    static constexpr int kRing = kW * kI8WBytes + kX * kXBytes;
    // CTAs that fit an SM's shared memory never want more than its TMEM columns together (w4a4_shape.h)
    static constexpr int kLeast = kTmemCols / 128 * 46 * 1024;
    static constexpr size_t kSmem = 1024 + (kRing > kLeast ? kRing : kLeast);
    static_assert(kW >= kA && kA >= kI8Groups, "see the converting warps' waits");
    static_assert(kAccCols + kA * kI8ACols <= kTmemCols && NT * 512 <= kRing && (kSmem + 1536) * kCtas <= 228 * 1024, "fits");
};

template <int NT, Int8Tokens kTok>
__global__ void __launch_bounds__(kIsThreads, IsShape<NT, kTok>::kCtas)
    int8_stream_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, const Int8Params p)
{
    using S = IsShape<NT, kTok>;
    constexpr int kW = S::kW, kX = S::kX, kA = S::kA;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *sW = smem, *sX = sW + kW * kI8WBytes;
    float *red = reinterpret_cast<float *>(smem);   // [NT][128], once the rings are drained
    __shared__ __align__(8) uint64_t w_full[kW], w_empty[kW], x_full[kX], x_empty[kX], a_full[kA], a_empty[kA], acc_full[1];
    __shared__ uint32_t s_tmem;
    __shared__ float s_scale[S::kOwn ? NT : 1];
    __shared__ uint32_t s_max[S::kOwn ? kI8Conv : 1];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = p.split > 1 ? (int)cluster_ctarank() : 0;
    const int tile = blockIdx.x / p.split, nt = tile / p.mtiles, mt = tile % p.mtiles;
    const int ks0 = (int)((int64_t)p.ksteps * rank / p.split), ks1 = (int)((int64_t)p.ksteps * (rank + 1) / p.split);
    const int nk = ks1 - ks0, cols = min(NT, p.M - mt * NT);   // stages; tokens of this tile
    if (threadIdx.x == 0) {
        for (int s = 0; s < kW; s++) {
            mbar_init(&w_full[s], 1);
            mbar_init(&w_empty[s], 4);
        }
        for (int s = 0; s < kX; s++) {
            mbar_init(&x_full[s], S::kOwn ? 32 * kI8Conv : 1);
            mbar_init(&x_empty[s], 1);
        }
        for (int s = 0; s < kA; s++) {
            mbar_init(&a_full[s], 4);
            mbar_init(&a_empty[s], 1);
        }
        mbar_init(acc_full, 1);
        mbar_fence_init();
    }
    if (warp == kI8Conv + 2) {
        tmem_alloc(&s_tmem, S::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem, a_ring = tmem + S::kAccCols;

    if (warp == kI8Conv) {
        // ---------------- copies of the weights' codes
        auto load = [&](int i) {
            mbar_arrive_expect_tx(&w_full[i % kW], kI8WBytes);
            tma_load_2d(sW + i % kW * kI8WBytes, &tm_w, &w_full[i % kW], (ks0 + i) * kI8K, nt * kI8Rows);
        };
        if (elect_one()) {
            // Before the kernels ahead in the stream are complete, the weights may be brought on their way: into
            // shared memory where nothing that can still run writes them (p.early), else into L2 only.
            const int head = min(nk, kW);
            for (int i = 0; i < head; i++) {
                if (p.early)
                    load(i);
                else
                    tma_prefetch_2d(&tm_w, (ks0 + i) * kI8K, nt * kI8Rows);
            }
            pdl_wait();
            pdl_launch_dependents();
            for (int i = p.early ? head : 0; i < nk; i++) {
                if (i >= kW && !mbar_wait(&w_empty[i % kW], (i / kW - 1) & 1)) {
                    record_status(p.ctl, NVFP4_ERR_TIMEOUT);
                    break;
                }
                load(i);
            }
        }
    } else if (warp == kI8Conv + 1) {
        // ---------------- copies of the tokens
        if (!S::kOwn && elect_one()) {
            pdl_wait();
            for (int i = 0; i < nk; i++) {
                const int st = i % kX;
                if (i >= kX && !mbar_wait(&x_empty[st], (i / kX - 1) & 1)) {
                    record_status(p.ctl, NVFP4_ERR_TIMEOUT);
                    break;
                }
                mbar_arrive_expect_tx(&x_full[st], S::kXBytes);
                tma_load_2d(sX + st * S::kXBytes, &tm_x, &x_full[st], (ks0 + i) * kI8K, mt * NT);
                tma_load_2d(sX + st * S::kXBytes + NT * 128, &tm_x, &x_full[st], (ks0 + i) * kI8K + 64, mt * NT);
            }
        }
    } else if (warp == kI8Conv + 2) {
        // ---------------- MMA
        if (elect_one()) {
            const uint32_t id = idesc_f16(kI8Rows, (cols + 15) & ~15, 0);
            bool ok = !S::kOwn || mbar_wait(&x_full[0], 0);
            int i = 0;
            for (; i < nk && ok; i++) {
                const int st = i % kX, sa = i % kA;
                ok = (S::kOwn || mbar_wait(&x_full[st], (i / kX) & 1)) && mbar_wait(&a_full[sa], (i / kA) & 1);
                if (!ok)
                    break;
                tc_fence_after();
                const uint64_t xd = smem_desc_sw128(smem_addr(sX + st * S::kXBytes));
#pragma unroll
                for (int j = 0; j < kI8K / 16; j++)
                    mma_f16_ts(tmem, a_ring + sa * kI8ACols + j * 8, xd + (j / 4) * (NT * 128 / 16) + (j % 4) * 2, id,
                               (i | j) != 0);
                if (!S::kOwn)
                    mma_commit(&x_empty[st]);
                mma_commit(&a_empty[sa]);
                if (i + 1 == nk)
                    mma_commit(acc_full);
            }
            if (!ok) {
                // copies on their way land before the CTA leaves, and the epilogue hears of the MMAs issued
                record_status(p.ctl, NVFP4_ERR_TIMEOUT);
                if (!S::kOwn)
                    ring_drain(x_full, kX, i, min(nk, i + kX));
                ring_drain(w_full, kW, i, min(nk, i + kA + kW));
                mma_commit(acc_full);
            }
        }
    } else {
        if constexpr (S::kOwn) {
            // ---------------- this CTA's part of the tokens, as integers in the swizzled layout of a TMA copy
            pdl_wait();
            using T = std::conditional_t<kTok == kRawFp32, float, __nv_bfloat16>;
            const int k0 = ks0 * kI8K / 8, n8 = p.K / 8;
            for (int m = 0; m < p.M; m++) {
                const T *src = reinterpret_cast<const T *>(p.x) + (int64_t)m * p.ldx;
                uint32_t a = 0;
#pragma unroll 4
                for (int i = threadIdx.x; i < n8; i += 32 * kI8Conv) {
                    Raw8<T> r;
                    r.load(src + i * 8);
                    a = max(a, r.amax_bits());
                }
                a = __reduce_max_sync(0xffffffffu, a);
                named_sync(1, 32 * kI8Conv);    // the token before has been read
                if (lane == 0)
                    s_max[warp] = a;
                named_sync(1, 32 * kI8Conv);
                a = __reduce_max_sync(0xffffffffu, s_max[lane & (kI8Conv - 1)]);
                const Int8Row row(a);
                if (threadIdx.x == 0)
                    s_scale[m] = row.scale();
                for (int i = threadIdx.x; i < nk * (kI8K / 8); i += 32 * kI8Conv) {
                    uint4 h = make_uint4(0u, 0u, 0u, 0u);
                    if (k0 + i < n8) {
                        Raw8<T> r;
                        r.load(src + (k0 + i) * 8);
                        h = row.halves(r);
                    }
                    const int st = i / (kI8K / 8), g = i % (kI8K / 8);   // stage; eight elements of it
                    *reinterpret_cast<uint4 *>(sX + st * S::kXBytes + (g >> 3) * (NT * 128) + m * 128 +
                                               (((g & 7) ^ (m & 7)) << 4)) = h;
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(&x_full[0]);
            // near ties part a warp; what follows needs all of its lanes together
            __syncwarp();
        }
        // ---------------- weights to fp16
        for (int i = warp / 4; i < nk; i += kI8Groups) {
            const int sw = i % kW, sa = i % kA;
            // In this order: the other group may have had this barrier's use before, and a wait for a use passes while
            // the one before it has not even completed.  The MMAs kA stages ago are behind that one (kW >= kA).
            if ((i >= kA && !mbar_wait_warp(&a_empty[sa], (i / kA - 1) & 1)) || !mbar_wait_warp(&w_full[sw], (i / kW) & 1))
                break;
            tc_fence_after();
            convert_rows(sW + sw * kI8WBytes, a_ring + sa * kI8ACols, warp, lane);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&w_empty[sw]);
                mbar_arrive(&a_full[sa]);
            }
        }
        pdl_wait();
        if (!mbar_wait_warp(acc_full, 0)) {
            if (threadIdx.x == 0)
                record_status(p.ctl, NVFP4_ERR_TIMEOUT);
            // longer than the issuing thread can take over its own waits
            for (int i = 0; i < 3 * nk + kX + kW + kA + 4 && !mbar_wait_warp(acc_full, 0); i++) {
            }
        }
        tc_fence_after();
    }
    __syncwarp();
    auto store = [&](int m, int n, float v) {
        v = scaled(v, S::kOwn ? s_scale[m] : p.x_scale[m], p.w_scale[n]);
        if (p.y_fp32)
            reinterpret_cast<float *>(p.y)[(size_t)m * p.N + n] = v;
        else
            reinterpret_cast<__nv_bfloat16 *>(p.y)[(size_t)m * p.N + n] = __float2bfloat16_rn(v);
    };
    if (warp < kI8Conv) {
        // every other 32 tokens
        const int quad = warp & 3, r = quad * 32 + lane, n = nt * kI8Rows + r;
        for (int c = (warp >> 2) * 32; c < cols; c += 64) {
            uint32_t v[32];
            __syncwarp();   // the stores before may have parted the warp
            tmem_ld32_start(tmem + ((uint32_t)(quad * 32) << 16) + c, v);
            tmem_ld32_finish(v);
#pragma unroll
            for (int i = 0; i < 32; i++) {
                if (c + i < cols) {
                    if (p.split > 1)
                        red[(c + i) * 128 + r] = __uint_as_float(v[i]);
                    else if (n < p.N)
                        store(mt * NT + c + i, n, __uint_as_float(v[i]));
                }
            }
        }
    }
    if (p.split > 1) {
        // ---------------- the tokens are shared out
        __syncwarp();
        __syncthreads();
        cluster_sync();
        const int c0 = cols * 128 * rank / p.split, c1 = cols * 128 * (rank + 1) / p.split;
        for (int i = c0 + threadIdx.x; i < c1; i += kIsThreads) {
            const int c = i / 128, n = nt * kI8Rows + i % 128;
            const uint32_t at = smem_addr(&red[i]);
            float part[8];
#pragma unroll
            for (int q = 0; q < 8; q++)
                if (q < p.split)
                    part[q] = ld_cluster_f32(at, (uint32_t)q);
            float v = part[0];
#pragma unroll
            for (int q = 1; q < 8; q++)
                if (q < p.split)
                    v += part[q];
            if (n < p.N)
                store(mt * NT + c, n, v);
        }
        __syncwarp();
        cluster_sync();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kI8Conv + 2) {
        tc_fence_after();
        tmem_dealloc(tmem, S::kTmemCols);
    }
}

// ---------------------------------------------------------------- many tokens
// CTA pairs, 256 weight rows x BN tokens at a time, persistent.  Both CTAs
// convert their 128 weight rows into their own TMEM; the leader's MMAs read
// both, and half of the tokens from each CTA's shared memory.  Up to 192 tokens
// there are two accumulators beside the converted weights' columns, so that a
// tile's results are scaled and stored while the next tile is multiplied.
constexpr int kItEpi = 4;
constexpr int kItThreads = 32 * (kI8Conv + kItEpi + 2);   // converting, epilogue, copies, MMA
constexpr int kItGroup = 8;   // raster: token tiles per group

template <int BN>
struct ItShape {
    static constexpr int kXBytes = BN / 2 * kI8K * 2, kStageBytes = kI8WBytes + kXBytes;
    static constexpr int kFit = (232448 - 512 - kStageOut) / kStageBytes, kStages = kFit < 6 ? kFit : 6;
    static constexpr size_t kSmem = 512 + (size_t)kStages * kStageBytes + kStageOut;
    static constexpr int kAcc = BN <= 192 ? 2 : 1;               // accumulators
    static constexpr int kFree = (512 - kAcc * BN) / kI8ACols, kA = kFree < 4 ? kFree : 4;   // stages of converted weights
    static_assert(kA % kI8Groups == 0 && kStages >= kA, "see the converting warps' waits");
};

template <int BN, bool kF32>
__global__ void __launch_bounds__(kItThreads, 1) __cluster_dims__(2, 1, 1)
    int8_tile_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x, const Int8Params p)
{
    using S = ItShape<BN>;
    constexpr int kStages = S::kStages, kA = S::kA, kAcc = S::kAcc;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *sW = smem, *sX = sW + kStages * kI8WBytes, *sOut = sX + kStages * S::kXBytes;
    uint64_t *full_w = reinterpret_cast<uint64_t *>(sOut + kStageOut), *full_x = full_w + kStages;
    uint64_t *done = full_x + kStages, *a_full = done + kStages, *a_empty = a_full + kA;
    uint64_t *acc_full = a_empty + kA, *acc_empty = acc_full + kAcc;
    uint32_t *s_tmem = reinterpret_cast<uint32_t *>(acc_empty + kAcc);
    volatile int *s_abort = reinterpret_cast<volatile int *>(s_tmem + 1);
    volatile uint32_t *s_loaded = s_tmem + 2, *s_issued = s_tmem + 3;   // stages copied and multiplied

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int crank = (int)cluster_ctarank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; s++) {
            mbar_init(&full_w[s], 1);
            mbar_init(&full_x[s], 1);
            mbar_init(&done[s], 1);
        }
        for (int s = 0; s < kA; s++) {
            mbar_init(&a_full[s], 2 * 4);
            mbar_init(&a_empty[s], 1);
        }
        for (int s = 0; s < kAcc; s++) {
            mbar_init(&acc_full[s], 1);
            mbar_init(&acc_empty[s], 2 * kItEpi);
        }
        *s_abort = 0;
        *s_loaded = 0;
        *s_issued = 0;
        mbar_fence_init();
    }
    if (warp == kI8Conv + kItEpi + 1)
        tmem_alloc_pair(s_tmem, 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers and TMEM before anything of the pair touches them
    tc_fence_after();
    const uint32_t tmem = *s_tmem, a_ring = tmem + kAcc * BN;
    pdl_wait();
    pdl_launch_dependents();

    const int cid = (int)cluster_id_x(), ncl = (int)cluster_count_x();
    const int ntot = p.mtiles * p.ntiles;
    auto fail = [&]() {
        record_status(p.ctl, NVFP4_ERR_TIMEOUT);
        *s_abort = 1;
    };
    auto aborted = [&]() { return __any_sync(0xffffffffu, *s_abort); };
    // groups of kItGroup token tiles, the token tile fastest: the pairs that run together share weights and tokens in L2
    auto tile_at = [&](int t, int &mt, int &nt) {
        const int per = kItGroup * p.ntiles, g = t / per, i = t % per, gm = min(kItGroup, p.mtiles - g * kItGroup);
        mt = g * kItGroup + i % gm;
        nt = i / gm;
    };
    // columns of a tile's MMAs
    auto width = [&](int mt) { return (min(BN, p.M - mt * BN) + 31) & ~31; };

    if (warp == kI8Conv + kItEpi) {
        // ---------------- copies: this CTA's weight rows, and half of the tokens for the leader's barrier
        if (elect_one()) {
            uint32_t it = 0;
            for (int t = cid; t < ntot && !*s_abort; t += ncl) {
                int mt, nt;
                tile_at(t, mt, nt);
                const int m0 = mt * BN + crank * (width(mt) / 2), n0 = nt * 256 + crank * 128;
                for (int ks = 0; ks < p.ksteps; ks++, it++) {
                    const int st = it % kStages;
                    if (!mbar_wait(&done[st], ((it / kStages) & 1) ^ 1)) {
                        fail();
                        break;
                    }
                    mbar_arrive_expect_tx(&full_w[st], kI8WBytes);
                    tma_load_2d(sW + st * kI8WBytes, &tm_w, &full_w[st], ks * kI8K, n0);
                    const uint32_t bar = cluster_addr(&full_x[st], 0);
                    if (crank == 0)
                        mbar_arrive_expect_tx(&full_x[st], 2 * S::kXBytes);
                    tma_load_2d_pair(sX + st * S::kXBytes, &tm_x, bar, ks * kI8K, m0);
                    tma_load_2d_pair(sX + st * S::kXBytes + S::kXBytes / 2, &tm_x, bar, ks * kI8K + 64, m0);
                }
            }
            // every stage released before leaving: the leader's commits must not arrive at a CTA that is gone
            for (int k = 0; k < kStages && !*s_abort; k++) {
                const uint32_t i2 = it + k;
                if (i2 >= (uint32_t)kStages && !mbar_wait(&done[i2 % kStages], ((i2 / kStages) & 1) ^ 1))
                    fail();
            }
            *s_loaded = it;
        }
    } else if (warp == kI8Conv + kItEpi + 1) {
        // ---------------- MMA, by one thread of the pair's leader
        if (crank == 0 && elect_one()) {
            uint32_t it = 0, lt = 0;
            for (int t = cid; t < ntot && !*s_abort; t += ncl, lt++) {
                int mt, nt;
                tile_at(t, mt, nt);
                const uint32_t id = idesc_f16(256, width(mt), 0);
                if (lt >= kAcc && !mbar_wait(&acc_empty[lt % kAcc], (lt / kAcc - 1) & 1)) {
                    fail();
                    break;
                }
                tc_fence_after();
                const uint32_t acc = tmem + lt % kAcc * BN;
                bool ok = true;
                for (int ks = 0; ks < p.ksteps; ks++, it++) {
                    const int st = it % kStages, sa = it % kA;
                    if (!mbar_wait(&full_x[st], (it / kStages) & 1) || !mbar_wait(&a_full[sa], (it / kA) & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t xd = smem_desc_sw128(smem_addr(sX + st * S::kXBytes));
#pragma unroll
                    for (int j = 0; j < kI8K / 16; j++)
                        mma_f16_ts_pair(acc, a_ring + sa * kI8ACols + j * 8, xd + (j / 4) * (S::kXBytes / 2 / 16) + (j % 4) * 2,
                                        id, (ks | j) != 0);
                    mma_commit_pair(&a_empty[sa]);
                    mma_commit_pair(&done[st]);
                    if (ks + 1 == p.ksteps)
                        mma_commit_pair(&acc_full[lt % kAcc]);
                }
                if (!ok) {
                    fail();
                    break;
                }
            }
            *s_issued = it;
        }
    } else if (warp < kI8Conv) {
        // ---------------- weights to fp16, stage by stage, also while a tile's accumulator is being read
        uint32_t it = (uint32_t)warp / 4;
        const uint32_t total = (uint32_t)((ntot - cid + ncl - 1) / ncl) * (uint32_t)p.ksteps;
        for (; it < total; it += kI8Groups) {
            const int st = it % kStages, sa = it % kA;
            // In this order, as in the streaming kernel: the MMAs kA stages ago are behind the use of full_w before this one.
            // (A group has every use of the columns that it has one of.)
            if ((it >= kA && !mbar_wait_warp(&a_empty[sa], (it / kA - 1) & 1)) ||
                !mbar_wait_warp(&full_w[st], (it / kStages) & 1)) {
                fail();
                break;
            }
            if (aborted())
                break;
            tc_fence_after();
            convert_rows(sW + st * kI8WBytes, a_ring + sa * kI8ACols, warp, lane);
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_cluster(cluster_addr(&a_full[sa], 0));   // hands over TMEM that is written (wait::st)
        }
    } else {
        // ---------------- epilogue: a warp has 32 weight rows
        const int quad = warp & 3;
        uint32_t lt = 0;
        bool dead = false;   // after a wait that gave up: the four warps that store together stay together
        for (int t = cid; t < ntot; t += ncl, lt++) {
            int mt, nt;
            tile_at(t, mt, nt);
            const int n0 = nt * 256 + crank * 128, rows = min(BN, p.M - mt * BN);
            // scales of the outputs that the thread's registers hold: its lane's, or in the fragments' layout four
            float sw[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int n = n0 + quad * 32 + (kF32 ? lane : 8 * i + lane / 4);
                sw[i] = n < p.N ? p.w_scale[n] : 0.0f;
            }
            if (!dead && (aborted() || !mbar_wait_warp(&acc_full[lt % kAcc], (lt / kAcc) & 1))) {
                fail();
                dead = true;
            }
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(quad * 32) << 16) + lt % kAcc * BN;
            uint32_t buf[2][32];
            tile_ld_start<kF32>(acc, buf[0]);
#pragma unroll
            for (int c = 0; c < BN / 32; c++) {
                uint32_t(&v)[32] = buf[c & 1];
                __syncwarp();   // the stores before may have parted the warp
                tmem_ld32_finish(v);
                if (c + 1 < BN / 32) {
                    tile_ld_start<kF32>(acc + (c + 1) * 32, buf[(c + 1) & 1]);
                } else {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_cluster(cluster_addr(&acc_empty[lt % kAcc], 0));
                }
                const int left = min(32, rows - c * 32), m = mt * BN + c * 32;
                if (left <= 0 || n0 >= p.N)
                    continue;
                const float sx = lane < left ? p.x_scale[m + lane] : 0.0f;
                // register i: row i, or row 8 (i / 4 % 4) + 2 (lane % 4) + i % 2 of output 16 (i / 16) + 8 (i / 2 % 2)
                auto row_scale = [&](int i) {
                    return __shfl_sync(0xffffffffu, sx, kF32 ? i : 8 * (i / 4 % 4) + 2 * (lane & 3) + i % 2);
                };
                auto out_scale = [&](int i) { return sw[kF32 ? 0 : 2 * (i / 16) + i / 2 % 2]; };
                if (__any_sync(0xffffffffu, fabsf(sx) > kI8Wide)) {
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        v[i] = __float_as_uint(scaled(__uint_as_float(v[i]), row_scale(i), out_scale(i)));
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i++)
                        v[i] = __float_as_uint(__fmul_rn(__fmul_rn(__uint_as_float(v[i]), row_scale(i)), out_scale(i)));
                }
                store_rows<kF32>(v, sOut, 1, p.y, m, left, p.N, n0, quad, lane, !dead);
            }
        }
    }

    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == kI8Conv + kItEpi + 1 && *s_abort) {
        // after a wait that gave up: copies on their way land, and MMAs issued are done, before either CTA leaves
        const uint32_t loaded = *s_loaded, issued = *s_issued, from = loaded > (uint32_t)kStages ? loaded - kStages : 0u;
        ring_drain(full_w, kStages, from, loaded);
        if (crank == 0) {
            ring_drain(full_x, kStages, from, loaded);
            if (issued > 0)
                ring_drain(done, kStages, issued - 1, issued);
        }
        __syncwarp();
    }
    cluster_sync();  // neither CTA leaves while the other may still signal or read it
    if (warp == kI8Conv + kItEpi + 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ---------------------------------------------------------------- launches
cudaError_t maps(CUtensorMap *tw, CUtensorMap *tx, const Int8GemmArgs &a, uint32_t tokens)
{
    const cudaError_t e = encode_tensor_map_2d(tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.w, (uint64_t)a.K, (uint64_t)a.N,
                                               (uint64_t)a.K, kI8K, kI8Rows, CU_TENSOR_MAP_SWIZZLE_128B);
    return e != cudaSuccess || !tx ? e
                                   : encode_tensor_map_2d(tx, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a.x, (uint64_t)a.K,
                                                          (uint64_t)a.M, (uint64_t)a.K * 2, 64, tokens, CU_TENSOR_MAP_SWIZZLE_128B);
}

Int8Params params(const Int8GemmArgs &a)
{
    Int8Params p = {};
    p.x_scale = a.x_scale;
    p.w_scale = a.w_scale;
    p.M = (int)a.M;
    p.N = (int)a.N;
    p.K = (int)a.K;
    p.x = a.x;
    p.ldx = a.ldx;
    p.ksteps = (int)((a.K + kI8K - 1) / kI8K);
    p.split = 1;
    p.y = a.y;
    p.y_fp32 = a.y_fp32 ? 1 : 0;
    p.ctl = a.ctl;
    return p;
}

// CTAs of a cluster that share a tile's K.
int stream_split(int64_t tiles, int64_t K, int places)
{
    return (int)std::max<int64_t>(1, std::min<int64_t>({8, (K + kI8K - 1) / kI8K, places / tiles}));
}

template <int NT, Int8Tokens kTok = kInts>
cudaError_t run_int8_stream(const Int8GemmArgs &a, cudaStream_t s, const DeviceInfo &dev)
{
    using S = IsShape<NT, kTok>;
    CUtensorMap tw, tx;
    cudaError_t e = maps(&tw, S::kOwn ? nullptr : &tx, a, NT);
    if (e == cudaSuccess)
        e = allow_smem<int8_stream_kernel<NT, kTok>>(S::kSmem, dev);
    if (e != cudaSuccess)
        return e;
    if (S::kOwn)
        tx = tw;
    Int8Params p = params(a);
    p.early = S::kOwn ? 0 : 1;
    p.mtiles = (int)((a.M + NT - 1) / NT);
    const int64_t tiles = (int64_t)p.mtiles * ((a.N + kI8Rows - 1) / kI8Rows);
    p.split = stream_split(tiles, a.K, S::kCtas * dev.num_sms);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(tiles * p.split));
    cfg.blockDim = dim3(kIsThreads);
    cfg.dynamicSmemBytes = S::kSmem;
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
    return cudaLaunchKernelEx(&cfg, int8_stream_kernel<NT, kTok>, tw, tx, p);
}

template <int BN, bool kF32>
cudaError_t run_int8_tile(const Int8GemmArgs &a, cudaStream_t s, const DeviceInfo &dev)
{
    using S = ItShape<BN>;
    CUtensorMap tw, tx;
    cudaError_t e = maps(&tw, &tx, a, BN / 2);
    if (e == cudaSuccess)
        e = allow_smem<int8_tile_kernel<BN, kF32>>(S::kSmem, dev);
    if (e != cudaSuccess)
        return e;
    Int8Params p = params(a);
    p.mtiles = (int)((a.M + BN - 1) / BN);
    p.ntiles = (int)((a.N + 255) / 256);
    const int64_t tiles = (int64_t)p.mtiles * p.ntiles;
    return launch_dependent(int8_tile_kernel<BN, kF32>, dim3(2 * (unsigned)std::min<int64_t>(tiles, dev.num_sms / 2)),
                            kItThreads, S::kSmem, s, tw, tx, p);
}

// Tokens a tile: the width whose waves of pairs take least.  A stage of 128
// elements of K takes 0.66 us at 256 tokens, 0.53 at 192 and 0.355 at 128 (near the
// power limit), and 2.5 us pass between tiles of 256.  With the quantiser, us at 256
// / 192 / 128: 8192 x 18944 x 3584 685 / 628 / 621; 1024 94 / 99 / 86; 200 x 27648 x
// 5120 62 / 71 / 52; 700 x 3584 x 18944 103 / 94 / 110; 4096 340 / 441 / 365; 2048 x 3584
// x 3584 54 / 58 / 42.
template <bool kF32>
cudaError_t run_widths(const Int8GemmArgs &a, cudaStream_t s, const DeviceInfo &dev)
{
    const int widths[3] = {256, 192, 128};
    const double stage[3] = {0.66, 0.53, 0.355}, apart[3] = {2.5, 0.3, 0.3};
    const int64_t ksteps = (a.K + kI8K - 1) / kI8K, pairs = dev.num_sms / 2;
    int best = 0;
    double least = 0;
    for (int i = 0; i < 3; i++) {
        const int64_t tiles = ((a.M + widths[i] - 1) / widths[i]) * ((a.N + 255) / 256);
        const double t = (double)((tiles + pairs - 1) / pairs) * (ksteps * stage[i] + apart[i]);
        if (i == 0 || t < least) {
            best = i;
            least = t;
        }
    }
    return best == 0 ? run_int8_tile<256, kF32>(a, s, dev) : best == 1 ? run_int8_tile<192, kF32>(a, s, dev)
                                                                       : run_int8_tile<128, kF32>(a, s, dev);
}

}  // namespace

// Whether the tokens are quantised in the product's kernel, not by a kernel of their own.  Every CTA reads the whole
// rows for their maxima, so few elements only; what it multiplies has to fit beside three stages of weights.
bool int8_takes_tokens(int64_t M, int64_t N, int64_t K, const DeviceInfo &dev)
{
    const int64_t tiles = (N + kI8Rows - 1) / kI8Rows, ksteps = (K + kI8K - 1) / kI8K;
    const int split = stream_split(tiles, K, 2 * dev.num_sms);
    return M <= 16 && M * K <= 16384 && (ksteps + split - 1) / split <= IsShape<16, kRawBf16>::kX && tiles * split <= 2 * dev.num_sms;
}

cudaError_t launch_int8_gemm(const Int8GemmArgs &a, cudaStream_t s, const DeviceInfo &dev)
{
    if (a.raw)
        return a.raw_fp32 ? run_int8_stream<16, kRawFp32>(a, s, dev) : run_int8_stream<16, kRawBf16>(a, s, dev);
    if (a.M <= 16)
        return run_int8_stream<16>(a, s, dev);
    if (a.M <= 32)
        return run_int8_stream<32>(a, s, dev);
    if (a.M <= 64)
        return run_int8_stream<64>(a, s, dev);
    // More than 128 tokens go to the tile kernel, unless there are few tiles: only the stream splits K (with the quantiser,
    // stream / tiles: 200 x 3584 x 18944 42.6 / 58.4 us, 512 x 1000 x 4096 15.0 / 19.6; without a split 300 x 3584 x 18944
    // 65.2 / 58.4, 512 x 3584 x 3584 19.9 / 21.1; up to 128 tokens 100 x 18944 x 3584 21.7 / 24.1).  Its tokens bound it:
    // each CTA of 128 weight rows copies them all, 55 of the 64 bytes a cycle that an SM gets.
    const int64_t tiles = ((a.M + 127) / 128) * ((a.N + kI8Rows - 1) / kI8Rows);
    if (a.M <= 128 || (a.M <= 512 && 2 * tiles <= dev.num_sms))
        return run_int8_stream<128>(a, s, dev);
    return a.y_fp32 ? run_widths<true>(a, s, dev) : run_widths<false>(a, s, dev);
}

}  // namespace nvfp4
