// distill.cu -- distillation from a teacher's top logits: loss and gradient.
//
// Mathematics, per row with student logits z (V values), temperature tau and
// teacher entries (i_j, t_j): q = softmax(z / tau),
//   renormalised: p = softmax_j(t / tau),
//                 loss = w tau^2 sum_j p_j (log p_j - log q_{i_j});
//   with a rest class: p_j = exp(t_j), p_r = max(0, 1 - sum p_j),
//                 q_r = sum of q over the entries the teacher did not name,
//                 loss = w tau^2 [sum_j p_j (log p_j - log q_{i_j})
//                                 + p_r (log p_r - log q_r)];
//   gradient, with P = sum_j p_j (+ p_r) and c = g w tau:
//                 dz_v = c (q_v P - p_v)              v named,
//                 dz_v = c q_v (P - p_r / q_r)        v not named.
//
// The floor is one read of z and one write of dz.  A softmax gradient needs
// the row twice (its statistics first), so a row is held in the shared memory
// of a cluster of up to 8 CTAs: bulk copies bring each CTA its slice of the
// vocabulary, the CTAs exchange (max, sum) through distributed shared memory
// once, and the gradient is written from the copy on chip.  The sum over the
// entries not named is formed without them (their slots are set to -inf
// after their logits have been fetched), never as 1 - sum: with a confident
// student the difference would have no correct digit.  All statistics are
// FP32; sums have a fixed order, so results do not depend on scheduling.
//
// A bounded wait that gives up makes the row NaN, since a call without a
// workspace has no status word to record it in.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace nvfp4 {

using namespace sm100;

namespace {

constexpr int kDsThreads = 256, kDsWarps = kDsThreads / 32;

// 2^x; results below 2^-126 are flushed to 0, which a sum of values in (0, 1]
// whose largest is 1 cannot notice.
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log2 of a sum (error below 2^-22; of 0: -inf).
__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two FP32 operations in one instruction.
__device__ __forceinline__ uint64_t pair2(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 split2(uint64_t v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xFF800000u); }
__device__ __forceinline__ float quiet_nan() { return __uint_as_float(0x7FC00000u); }

// A maximum m of logits and the sum s of 2^((z - m) k2), k2 = log2(e) / tau.
// The difference is taken before the scaling where z is so large that z k2
// may leave FP32's range: a row whose logits are all the type's lowest value is
// uniform, not a row of infinities.
struct MaxSum {
    float m, s;
};

__device__ __forceinline__ float finite_or_zero(float m) { return m == neg_inf() ? 0.0f : m; }

// s of a MaxSum with its maximum moved to m (which is not below v.m)
__device__ __forceinline__ float sum_at(MaxSum v, float m, float k2)
{
    return v.s * ex2((v.m - finite_or_zero(m)) * k2);
}

__device__ __forceinline__ MaxSum merge(MaxSum a, MaxSum b, float k2)
{
    const float m = fmaxf(a.m, b.m);
    return {m, sum_at(a, m, k2) + sum_at(b, m, k2)};
}

__device__ __forceinline__ float warp_max(float v)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One value per warp -> all of them to every thread, combined in warp order.
__device__ __forceinline__ float over_warps_max(const float4 *s_w)
{
    const float4 a = s_w[0], b = s_w[1];
    return fmaxf(fmaxf(fmaxf(a.x, a.y), fmaxf(a.z, a.w)), fmaxf(fmaxf(b.x, b.y), fmaxf(b.z, b.w)));
}

__device__ __forceinline__ float over_warps_sum(const float4 *s_w)
{
    const float4 a = s_w[0], b = s_w[1];
    return ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
}

__device__ __forceinline__ void st_cluster_f4(uint32_t local, uint32_t rank, float4 v)
{
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
                 "st.shared::cluster.v4.f32 [a], {%2, %3, %4, %5};\n\t}" ::"r"(local),
                 "r"(rank), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

// Both by whole warps: lanes that took different ways before come together first.
__device__ __forceinline__ void cluster_arrive()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait()
{
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename T>
struct Vec;  // 16 bytes of logits
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(uint4 u, float (&v)[8])
    {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[8])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void unpack(uint4 u, float (&v)[4])
    {
        v[0] = __uint_as_float(u.x);
        v[1] = __uint_as_float(u.y);
        v[2] = __uint_as_float(u.z);
        v[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&v)[4])
    {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
    static __device__ __forceinline__ float get(float v) { return v; }
    static __device__ __forceinline__ float put(float v) { return v; }
};

// Logits below this magnitude times k2 are below 2^12: the rounding of such a
// product, 2^-13 at most, is corrected for (Running) or lost in bf16 (GradScale).
__device__ __forceinline__ float limit_for(float k2) { return fminf(0x1p12f / k2, 0x1p120f); }

// A thread's sum over 16 bytes of logits at a time: one fused operation and one
// exponential per element.  Any element's value m will do as the reference of
// the sum, since FP32 keeps its relative precision far above and below 1: the
// first finite vector gives it, and a sum that grows past 2^60 moves it up.  So
// no maximum is formed element by element.  A sum that overflowed in one step,
// or a row's reference near the limits or beyond, sends the row to scan_any (no
// ordinary row goes there).
struct Running {
    float m;           // reference; -limit: none yet
    uint64_t nb2, s2;  // minus the reference times k2, twice; two sums of 2^(z k2 - m k2)

    __device__ __forceinline__ Running(float limit, float k2) : m(-limit), nb2(pair2(limit * k2, limit * k2)), s2(0ull)
    {
    }
    template <int NE>
    __device__ __forceinline__ void add(const float (&v)[NE], float k2, float limit)
    {
        if (m == -limit) {
            float first = v[0];
#pragma unroll
            for (int e = 1; e < NE; e++)
                first = fmaxf(first, v[e]);
            if (!(first > m)) {
                // nothing above -limit: no addend unless the whole row is like that; a NaN stays one
#pragma unroll
                for (int e = 0; e < NE; e++)
                    if (v[e] != v[e])
                        s2 = pair2(v[e], 0.0f);
                return;
            }
            m = first;
            nb2 = pair2(-m * k2, -m * k2);
        }
        const uint64_t kk = pair2(k2, k2);
        uint64_t part = 0ull;
#pragma unroll
        for (int e = 0; e < NE; e += 2) {
            const float2 x = split2(fma2(pair2(v[e], v[e + 1]), kk, nb2));
            part = add2(part, pair2(ex2(x.x), ex2(x.y)));
        }
        s2 = add2(s2, part);
        const float2 s = split2(s2);
        if (s.x + s.y > 0x1p60f) {
            const float nb = split2(nb2).x, up = nb - 60.0f, f = ex2(up - nb);
            m = -up / k2;
            nb2 = pair2(up, up);
            s2 = pair2(s.x * f, s.y * f);
        }
    }
    // The sum is that of 2^(z k2 + nb); nb + m k2, the rounding of nb, goes into it.
    __device__ __forceinline__ MaxSum result(float k2) const
    {
        const float2 s = split2(s2);
        const float sum = (s.x + s.y) * ex2(-fmaf(m, k2, split2(nb2).x));
        return {sum == __uint_as_float(0x7F800000u) ? sum : m, sum};
    }
};

// Whether a block's references and sums, from Running, stand for its row: what
// was passed over below -limit has to be nothing beside it (2^-128).
__device__ __forceinline__ bool usable(float m, float limit) { return fabsf(m) < limit * (1.0f - 0x1p-5f); }

// (max, sum) of the elements get(j), any magnitudes: every difference before
// the scaling.
template <typename F>
__device__ __forceinline__ MaxSum scan_any(int begin, int end, int stride, float k2, F get)
{
    MaxSum r = {neg_inf(), 0.0f};
    for (int i = begin; i < end; i += stride) {
        const float v = get(i);
        if (v > r.m) {
            r.s *= ex2((r.m - v) * k2);
            r.m = v;
        }
        r.s += ex2((v - finite_or_zero(r.m)) * k2);
    }
    return r;
}

// Share of `part` in a whole with maximum `base` and sum `sum`, and its natural
// logarithm: of the share itself where FP32 holds it (a difference of logarithms
// of sums would lose the digits of a share near 1).
__device__ __forceinline__ float share_of(MaxSum part, float base, float sum, float k2)
{
    return part.s * ex2((part.m - base) * k2) * __frcp_rn(sum);
}
__device__ __forceinline__ float log_share(float share, MaxSum part, float base, float sum, float inv_tau)
{
    return share > 0x1p-100f ? logf(share) : (part.m - base) * inv_tau + logf(part.s) - logf(sum);
}

// The gradient of the entries that are not named, cu 2^((z - bu) k2) / sum: c
// q_v P, or with a rest class c (P q_r - p_r) u_v with u the softmax over them
// alone, so that a q_r below FP32's range costs nothing.  A bf16 gradient takes
// |cu| / sum into the exponent (one rounding of an argument of at most a few
// hundred: 2^-16 relative, and 2^-13 at 2^12, far below bf16's 2^-9) and its sign
// into the conversion; an FP32 one takes the difference first, which keeps the argument's
// rounding small where the gradient is large.
template <typename T>
struct GradScale {
    static constexpr bool kFold = sizeof(T) == 2;
    float cu, bu, lu, k2, off;
    bool plain, negative;

    __device__ __forceinline__ GradScale(const DistillArgs &a, float c, MaxSum all, MaxSum total, float mass,
                                         float rest_p, float rest_q, float k2_)
        : k2(k2_)
    {
        // a rest without any mass (all.s = 0) has no gradient
        const bool none = a.tail && all.s == 0.0f && total.s != 0.0f;
        const float sum = a.tail ? (none ? 1.0f : all.s) : total.s;
        bu = finite_or_zero(a.tail ? all.m : total.m);
        cu = a.tail ? c * (mass * rest_q - rest_p) : c * mass;
        plain = fabsf(bu) < limit_for(k2);
        negative = cu < 0.0f;
        if (kFold)
            lu = lg2(sum) - lg2(fabsf(cu));
        else
            cu *= __frcp_rn(sum);
        off = kFold && plain ? fmaf(bu, k2, lu) : 0.0f;
    }
    template <bool kPlain, bool kNeg>
    __device__ __forceinline__ uint4 apply(float (&v)[Vec<T>::N]) const
    {
        const uint64_t kk = pair2(k2, k2), no = pair2(-off, -off), nb = pair2(-bu, -bu);
#pragma unroll
        for (int e = 0; e < Vec<T>::N; e += 2) {
            float2 x;
            if (!kFold)
                x = split2(mul2(add2(pair2(v[e], v[e + 1]), nb), kk));
            else if (kPlain)
                x = split2(fma2(pair2(v[e], v[e + 1]), kk, no));
            else
                x = make_float2((v[e] - bu) * k2 - lu, (v[e + 1] - bu) * k2 - lu);
            v[e] = ex2(x.x);
            v[e + 1] = ex2(x.y);
            if (!kFold) {
                x = split2(mul2(pair2(v[e], v[e + 1]), pair2(cu, cu)));
                v[e] = x.x;
                v[e + 1] = x.y;
            } else if (kNeg) {
                v[e] = -v[e];
                v[e + 1] = -v[e + 1];
            }
        }
        return Vec<T>::pack(v);
    }
    // f(plain, negative): the variant of apply, chosen once a row
    template <typename F>
    __device__ __forceinline__ void choose(bool fast, F f) const
    {
        if (fast && plain && kFold && negative)
            f(std::true_type(), std::true_type());
        else if (fast && plain)
            f(std::true_type(), std::false_type());
        else if (kFold && negative)
            f(std::false_type(), std::true_type());
        else
            f(std::false_type(), std::false_type());
    }
};

__device__ __forceinline__ int64_t entry_index(const DistillArgs &a, int64_t at)
{
    return a.idx64 ? reinterpret_cast<const int64_t *>(a.idx)[at]
                   : (int64_t)reinterpret_cast<const int32_t *>(a.idx)[at];
}

__device__ __forceinline__ float entry_value(const DistillArgs &a, int64_t at)
{
    return a.val_fp32 ? reinterpret_cast<const float *>(a.val)[at]
                      : __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(a.val)[at]);
}

// After a wait for a copy that gave up: reported where there is a status word,
// and waited for once more, so that the CTA does not leave with it on its way.
// (A call: few rows take microseconds, in which more code shows.)
__device__ __noinline__ void copy_gave_up(uint32_t *ctl, uint64_t *bar)
{
    if (ctl)
        record_status(ctl, NVFP4_ERR_TIMEOUT);
    mbar_wait(bar, 0);
}

// One row per cluster of C CTAs; CTA `rank` takes logits [rank L, rank L + L).
// kEntries: teacher entries a thread holds.
template <typename T, bool kGrad, int kEntries>
__global__ void __launch_bounds__(kDsThreads)
    distill_kernel(const __grid_constant__ DistillArgs a, int C, int64_t L)
{
    constexpr int NE = Vec<T>::N;
    extern __shared__ __align__(16) uint8_t s_raw[];
    __shared__ __align__(16) float4 s_m[3][kDsWarps / 4], s_s[4][kDsWarps / 4], s_f[kDsWarps / 4];
    __shared__ __align__(16) float4 s_x[8];   // each CTA's (max, sum) of the unnamed and of the named logits
    __shared__ __align__(16) float4 s_l[8];   // each CTA's share of the loss (rank 0's copy is used)
    __shared__ __align__(8) uint64_t s_bar;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = C > 1 ? (int)cluster_ctarank() : 0;
    const int64_t row = blockIdx.x / C;
    const float w = a.weight ? a.weight[row] : 1.0f;
    const int64_t v0 = rank * L;
    const int64_t len64 = a.V - v0;
    const int len = (int)(len64 < 0 ? 0 : len64 < L ? len64 : L);

    // the slice sits at the address modulo 16 that it has in global memory
    const T *zs = reinterpret_cast<const T *>(a.z) + row * a.ldz + v0;
    const int sh = (int)(((uintptr_t)zs & 15u) / sizeof(T));
    T *s_z = reinterpret_cast<T *>(s_raw);     // element i of the slice at s_z[sh + i]
    const int nvec = len > 0 ? (sh + len + NE - 1) / NE : 0;
    T *dzs = kGrad ? reinterpret_cast<T *>(a.dz) + row * a.lddz + v0 : nullptr;
    const int shd = kGrad ? (int)(((uintptr_t)dzs & 15u) / sizeof(T)) : 0;

    // 16 bytes of dz at elements i0 .. i0 + NE - 1 of the slice, those that exist
    auto store = [&](int i0, uint4 u) {
        if (sh == shd && i0 >= 0 && i0 + NE <= len) {
            __stcs(reinterpret_cast<uint4 *>(dzs + i0), u);   // nobody reads it here
        } else {
            const T *v = reinterpret_cast<const T *>(&u);
#pragma unroll
            for (int e = 0; e < NE; e++)
                if (i0 + e >= 0 && i0 + e < len)
                    dzs[i0 + e] = v[e];
        }
    };
    auto store_zeros = [&]() {
        for (int j = tid; j < nvec; j += kDsThreads)
            store(j * NE - sh, make_uint4(0u, 0u, 0u, 0u));
        if (a.loss && rank == 0 && tid == 0)
            a.loss[row] = 0.0f;
    };
    if (w == 0.0f) {  // the logits are not looked at; a NaN weight counts as a weight
        if (kGrad)
            store_zeros();
        else if (rank == 0 && tid == 0)
            a.loss[row] = 0.0f;
        return;       // the whole cluster: nobody has touched a peer
    }

    if (tid == 0) {
        mbar_init(&s_bar, 1);
        mbar_fence_init();
        if (len > 0) {
            const uint8_t *src = reinterpret_cast<const uint8_t *>(zs - sh);
            const uint32_t bytes = (uint32_t)(((int64_t)(sh + len) * (int)sizeof(T)) & ~15);
            mbar_arrive_expect_tx(&s_bar, bytes);
            for (uint32_t o = 0; o < bytes; o += 32768)
                bulk_g2s(s_raw + o, src + o, min(32768u, bytes - o), &s_bar);
        }
    }
    // the last partial 16 bytes of the slice are not copied: one thread an element
    const int cut = (sh + len) & ~(NE - 1);
    T last = Vec<T>::put(neg_inf());
    if (tid < NE && cut + tid >= sh && cut + tid < sh + len)
        last = zs[cut + tid - sh];

    // ---- the teacher's entries: every CTA reads them all
    int idx[kEntries];      // in the vocabulary; -1: unused
    float lp[kEntries];     // teacher value, later log p_j (base e); -inf for an unused slot
    int seen = 0;           // entries that count: used ones (rest class), or ones with mass (renormalised)
    const float inv_tau = a.inv_tau, k2 = inv_tau * kLog2e;
    MaxSum t = {a.tail ? 0.0f : neg_inf(), 0.0f};
#pragma unroll
    for (int e = 0; e < kEntries; e++) {
        const int j = tid + e * kDsThreads;
        idx[e] = -1;
        lp[e] = neg_inf();
        if (j < a.k) {
            const int64_t at = row * a.k + j;
            const int64_t i = entry_index(a, at);
            const float tv = entry_value(a, at);
            if (i >= a.V) {
                if (a.ctl && rank == 0)
                    record_status(a.ctl, NVFP4_ERR_INDEX);
            } else if (i >= 0) {
                idx[e] = (int)i;
                lp[e] = tv;
                seen += a.tail || tv != neg_inf();
                // with a rest class only the plain sum of exp(t_j) is wanted: base 0
                t = a.tail ? MaxSum{0.0f, t.s + expf(tv)} : merge(t, MaxSum{tv, 1.0f}, k2);
            }
        }
    }
    __syncthreads();       // the barrier is initialised
    if (C > 1)
        cluster_arrive();  // matched below: every CTA of the cluster runs before anyone writes to it
    const bool landed = len <= 0 || (!a.give_up && mbar_wait(&s_bar, 0));
    if (!landed)
        copy_gave_up(a.ctl, &s_bar);

    // elements of the first and last 16 bytes outside the slice: -inf
    if (tid < NE && len > 0) {
        if (tid < sh)
            s_z[tid] = Vec<T>::put(neg_inf());
        if (cut + tid >= sh)
            s_z[cut + tid] = last;
    }
    __syncthreads();

    // ---- logits of this CTA's named entries, then (rest class) their slots out of the sum
    float zn[kEntries];
    MaxSum named = {neg_inf(), 0.0f};
#pragma unroll
    for (int e = 0; e < kEntries; e++) {
        const int64_t i = idx[e] - v0;
        zn[e] = 0.0f;
        if (idx[e] < 0 || i < 0 || i >= len) {
            idx[e] = -1;
        } else {
            zn[e] = Vec<T>::get(s_z[sh + i]);
            if (a.tail)
                named = merge(named, MaxSum{zn[e], zn[e] == neg_inf() ? 0.0f : 1.0f}, k2);
        }
    }
    if (a.tail) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kEntries; e++)
            if (idx[e] >= 0)
                s_z[sh + idx[e] - v0] = Vec<T>::put(neg_inf());
        __syncthreads();
    }

    // ---- one pass: running maximum and sum
    const float limit = limit_for(k2);
    Running run(limit, k2);
    for (int j = tid; j < nvec; j += kDsThreads) {
        float v[NE];
        Vec<T>::unpack(*reinterpret_cast<const uint4 *>(s_raw + (size_t)j * 16), v);
        run.add(v, k2, limit);
    }
    MaxSum all = run.result(k2);

    // ---- over the block: maxima first, then sums at the common maximum, in a fixed order
    {
        const float m1 = a.tail ? warp_max(named.m) : warp_max(t.m);
        float ma, mb;
        for (int again = 0;; again++) {
            const float m0 = warp_max(all.m);
            if (lane == 0) {
                reinterpret_cast<float *>(s_m[0])[warp] = m0;
                reinterpret_cast<float *>(s_m[1])[warp] = m1;
            }
            __syncthreads();
            ma = over_warps_max(s_m[0]);
            mb = over_warps_max(s_m[1]);
            if (again || usable(ma, limit))
                break;
            __syncthreads();   // every thread has read s_m
            all = scan_any(tid, len, kDsThreads, k2, [&](int i) { return Vec<T>::get(s_z[sh + i]); });
        }
        // a sum of NaN makes the row's loss and gradient NaN, in every CTA
        all = {ma, warp_sum(landed ? sum_at(all, ma, k2) : quiet_nan())};
        if (a.tail)
            named = {mb, warp_sum(sum_at(named, mb, k2))};
        else
            t = {mb, sum_at(t, mb, k2)};
        const float st = warp_sum(t.s), sn = warp_sum((float)seen);
        if (lane == 0) {
            reinterpret_cast<float *>(s_s[0])[warp] = all.s;
            reinterpret_cast<float *>(s_s[1])[warp] = named.s;
            reinterpret_cast<float *>(s_s[2])[warp] = st;
            reinterpret_cast<float *>(s_s[3])[warp] = sn;
        }
        __syncthreads();
        all.s = over_warps_sum(s_s[0]);
        if (a.tail)
            named.s = over_warps_sum(s_s[1]);
        t.s = over_warps_sum(s_s[2]);
        seen = (int)over_warps_sum(s_s[3]);   // at most 1024: exact
    }
    if (C > 1) {
        cluster_wait();
        if (tid < C)
            st_cluster_f4(smem_addr(&s_x[rank]), (uint32_t)tid, make_float4(all.m, all.s, named.m, named.s));
        cluster_arrive();
    }

    // ---- the teacher's distribution
    // log p_j = lp - log_s; p_j itself not from that: the difference's rounding
    // would count in a gradient where teacher and student nearly agree
    float mass = 1.0f, rest_p = 0.0f, log_s = 0.0f, inv_s = 1.0f;
    if (a.tail) {
        // a NaN sum stays a NaN; a teacher that names the whole vocabulary leaves no rest
        rest_p = t.s > 1.0f || seen >= a.V ? 0.0f : 1.0f - t.s;
        mass = t.s + rest_p;
    } else {
        const float base = finite_or_zero(t.m);
        log_s = logf(t.s);
        inv_s = __frcp_rn(t.s);
#pragma unroll
        for (int e = 0; e < kEntries; e++)
            lp[e] = (lp[e] - base) * inv_tau;
    }

    if (C > 1) {
        cluster_wait();
        float ma = neg_inf(), mn = neg_inf();
        for (int i = 0; i < C; i++) {
            ma = fmaxf(ma, s_x[i].x);
            mn = fmaxf(mn, s_x[i].z);
        }
        float sa = 0.0f, sn = 0.0f;
        for (int i = 0; i < C; i++) {
            sa += sum_at(MaxSum{s_x[i].x, s_x[i].y}, ma, k2);
            if (a.tail)
                sn += sum_at(MaxSum{s_x[i].z, s_x[i].w}, mn, k2);
        }
        all = {ma, sa};
        if (a.tail)
            named = {mn, sn};
    }
    if (seen == 0) {
        // no teacher entry: loss 0 and gradient 0, whatever the logits hold
        if (kGrad)
            store_zeros();
        else if (rank == 0 && tid == 0)
            a.loss[row] = 0.0f;
        return;
    }
    // q_v = 2^((z_v - total.m) k2) / total.s; a row of nothing but -inf has
    // total.s = 0 and gives NaN
    const MaxSum total = a.tail ? merge(all, named, k2) : all;
    const float base = finite_or_zero(total.m);
    const float rest_q = share_of(all, base, total.s, k2);   // q_r, of the entries that are not named

    // ---- this CTA's share of the loss, sent to rank 0 while the gradient is written
    if (a.loss) {
        float l = 0.0f;
        const float log_total = logf(total.s);
#pragma unroll
        for (int e = 0; e < kEntries; e++) {
            if (idx[e] >= 0) {
                const float p = expf(lp[e]) * inv_s;
                if (p != 0.0f)
                    l += p * (lp[e] - log_s - ((zn[e] - base) * inv_tau - log_total));
            }
        }
        l = warp_sum(l);
        if (lane == 0)
            reinterpret_cast<float *>(s_f)[warp] = l;
        __syncthreads();
        if (tid == 0) {
            const float sum = over_warps_sum(s_f);
            if (C > 1)
                st_cluster_f4(smem_addr(&s_l[rank]), 0u, make_float4(sum, 0.0f, 0.0f, 0.0f));
            else
                s_l[0].x = sum;
        }
    }
    if (C > 1)
        cluster_arrive();

    if (kGrad) {
        const float g = a.grad_loss ? a.grad_loss[a.grad_rows ? row : 0] : 1.0f;
        const float c = g * w * a.tau;
        const GradScale<T> scale(a, c, all, total, mass, rest_p, rest_q, k2);
        scale.choose(true, [&](auto plain, auto neg) {
            for (int j = tid; j < nvec; j += kDsThreads) {
                float v[NE];
                Vec<T>::unpack(*reinterpret_cast<const uint4 *>(s_raw + (size_t)j * 16), v);
                store(j * NE - sh, scale.template apply<decltype(plain)::value, decltype(neg)::value>(v));
            }
        });
        __syncthreads();   // the named entries are written over what the pass above stored
        const float inv_total = __frcp_rn(total.s);
#pragma unroll
        for (int e = 0; e < kEntries; e++)
            if (idx[e] >= 0)
                dzs[idx[e] - v0] = Vec<T>::put(c * (mass * (expf((zn[e] - base) * inv_tau) * inv_total) -
                                                    expf(lp[e]) * inv_s));
    }
    if (C > 1)
        cluster_wait();
    if (a.loss && rank == 0 && tid == 0) {
        float l = 0.0f;
        for (int i = 0; i < C; i++)
            l += s_l[i].x;
        if (a.tail && rest_p != 0.0f)
            l += rest_p * (logf(rest_p) - log_share(rest_q, all, base, total.s, inv_tau));
        a.loss[row] = l * w * a.tau * a.tau;
    }
}

// ---------------------------------------------------------------- many long rows
// Two CTAs per SM, persistent over the rows, a row each.  A cluster per row
// spends more on starting clusters and waiting for the slowest CTA than on the
// logits (4096 rows of 131072 bf16 logits: 500 us, 63 % of the copy bandwidth);
// here a row's chunks pass through a ring in shared memory twice (382 us,
// 83 %).  The chunks that the ring still holds after the first pass are used
// from there, the ones before them come again, most of them from L2; the
// gradient of aligned rows is stored to be evicted first, so that it does not
// push them out (with plain stores 407 us).  One warp copies, the others are
// consumers.  One CTA of 1024 threads per SM was slower (475 us against 424 at
// the time): its reductions and the turn from one pass to the other leave the
// SM without work, which the other CTA fills here.
// What bounds it is DRAM: of 1024 rows a quarter of what is read again (16 % of
// the logits; 43 % with plain stores) misses L2, and with that it moves 6.1 TB/s
// at 4096 rows, 89 % of the copy rate.  Issue (about 50 instructions per 8
// logits and pass) takes 64 % of the slots.
constexpr int kDtThreads = 512, kDtPerSm = 2, kDtWarps = kDtThreads / 32 - 1, kDtConsumers = 32 * kDtWarps;
constexpr int kDtEach = 4;                       // 16-byte vectors of a chunk that a consumer takes
constexpr int kDtVecs = kDtEach * kDtConsumers;
constexpr int kDtChunk = kDtVecs * 16;           // 30720 bytes
constexpr int kDtMaxSlots = 3;
constexpr int kDtSmem = 113 * 1024 - 1200;       // dynamic shared memory of one of two CTAs

__device__ __forceinline__ void bulk_g2s_hint(void *dst, const void *src, uint32_t bytes, uint64_t *bar, uint64_t pol)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
        "[%0], [%1], %2, [%3], %4;" ::"r"(smem_addr(dst)),
        "l"(src), "r"(bytes), "r"(smem_addr(bar)), "l"(pol)
        : "memory");
}

// One value per consumer warp -> combined in a fixed order, for every thread
// (called by whole warps).
__device__ __forceinline__ float over_consumers_max(const float *s_w, int lane) { return warp_max(s_w[lane]); }
__device__ __forceinline__ float over_consumers_sum(const float *s_w, int lane) { return warp_sum(s_w[lane]); }

template <typename T, bool kGrad>
__global__ void __launch_bounds__(kDtThreads, kDtPerSm)
    distill_stream_kernel(const __grid_constant__ DistillArgs a, const int slots)
{
    constexpr int NE = Vec<T>::N;
    extern __shared__ __align__(16) uint8_t s_ring[];  // slots chunks, then one bit per logit (rest class)
    __shared__ float s_m[2][32], s_s[4][32], s_f[32];
    __shared__ __align__(8) uint64_t full[kDtMaxSlots], empty[kDtMaxSlots];
    uint32_t *s_bits = reinterpret_cast<uint32_t *>(s_ring + slots * kDtChunk);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < slots; i++) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], kDtWarps);
        }
        mbar_fence_init();
    }
    if (a.tail) {
        const int words = (int)((a.V + NE + 31) / 32);
        for (int i = tid; i < words; i += kDtThreads)
            s_bits[i] = 0u;
    }
    if (tid < 32) {  // values of each reduction that no warp writes
        s_m[0][tid] = s_m[1][tid] = neg_inf();
        for (int i = 0; i < 4; i++)
            s_s[i][tid] = 0.0f;
        s_f[tid] = 0.0f;
    }
    __syncthreads();

    // chunks of a row, and the first one that the ring still holds after the first pass
    const T *z = reinterpret_cast<const T *>(a.z);
    auto shift = [&](int64_t row) { return (int)(((uintptr_t)(z + row * a.ldz) & 15u) / sizeof(T)); };
    auto vectors = [&](int sh) { return (int)((sh + a.V + NE - 1) / NE); };
    uint32_t load = 0;  // copies so far, in the order both sides agree on: copy i uses slot i % slots

    if (warp == kDtWarps) {
        if (lane == 0) {
            const uint64_t drop = l2_policy_evict_first();
            bool ok = true;
            for (int64_t row = blockIdx.x; row < a.T && ok; row += gridDim.x) {
                if (a.weight && a.weight[row] == 0.0f)
                    continue;
                const int sh = shift(row), n = (vectors(sh) + kDtVecs - 1) / kDtVecs;
                const int kept = kGrad ? max(0, n - slots) : n;
                const uint8_t *src = reinterpret_cast<const uint8_t *>(z + row * a.ldz - sh);
                const int64_t total = (int64_t)((sh + a.V) * (int64_t)sizeof(T)) & ~15LL;
                for (int i = 0; i < n + (kGrad ? kept : 0) && ok; i++, load++) {
                    const int c = i < n ? i : i - n, slot = load % slots;
                    if (load >= (uint32_t)slots && (a.give_up || !mbar_wait(&empty[slot], (load / slots - 1) & 1))) {
                        if (a.ctl)
                            record_status(a.ctl, NVFP4_ERR_TIMEOUT);
                        ok = false;
                        break;
                    }
                    const int64_t at = (int64_t)c * kDtChunk;
                    const uint32_t bytes = (uint32_t)max((int64_t)0, min((int64_t)kDtChunk, total - at));
                    mbar_arrive_expect_tx(&full[slot], bytes);
                    if (bytes) {
                        // chunks that will be read once more stay in L2
                        if (c < kept && i < n && kGrad)
                            bulk_g2s(s_ring + slot * kDtChunk, src + at, bytes, &full[slot]);
                        else
                            bulk_g2s_hint(s_ring + slot * kDtChunk, src + at, bytes, &full[slot], drop);
                    }
                }
            }
            // consumers that gave up wait no more, but the CTA does not leave with copies on their way
            for (uint32_t i = load > (uint32_t)slots ? load - slots : 0u; i < load; i++)
                mbar_wait(&full[i % slots], (i / slots) & 1);
        }
        return;
    }

    const float inv_tau = a.inv_tau, k2 = inv_tau * kLog2e, limit = limit_for(k2);
    const int V = (int)a.V;
    int slot = 0;             // of the next copy
    uint32_t phase = 0;       // and its barrier's parity
    // A thread whose wait gave up waits no more, and as lane 0 frees no slot any more, so that no slot is filled before
    // its last copy has landed: the producer and the other warps give up in turn, and the rows from there on are NaN.
    bool ok = !a.give_up;
    auto next = [&]() {
        if (++slot == slots) {
            slot = 0;
            phase ^= 1;
        }
    };
    auto release = [&](int at) {
        __syncwarp();
        if (lane == 0 && ok)
            mbar_arrive(&empty[at]);
    };
    // A row's weight, this thread's teacher entry and the student's logit there
    // are three dependent reads: they are issued a row ahead, the logit after
    // the first pass.
    struct Entry {
        float w = 0.0f, lp = neg_inf(), zn = 0.0f;
        int idx = -1;
    };
    auto entry_of = [&](int64_t row) {
        Entry e;
        if (row < a.T) {
            e.w = a.weight ? a.weight[row] : 1.0f;
            if (tid < a.k) {
                const int64_t at = row * a.k + tid, i = entry_index(a, at);
                e.lp = entry_value(a, at);
                if (i >= a.V && e.w != 0.0f && a.ctl)
                    record_status(a.ctl, NVFP4_ERR_INDEX);
                e.idx = i >= 0 && i < a.V ? (int)i : -1;
            }
        }
        return e;
    };
    auto logit_of = [&](Entry &e, int64_t row) {
        if (e.idx >= 0 && e.w != 0.0f)
            e.zn = Vec<T>::get(z[row * a.ldz + e.idx]);
        else
            e.lp = neg_inf();
    };
    Entry ahead = entry_of(blockIdx.x);
    logit_of(ahead, blockIdx.x);
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
        const Entry now = ahead;
        ahead = entry_of(row + gridDim.x);
        const float w = now.w;
        const int sh = shift(row), nvec = vectors(sh), n = (nvec + kDtVecs - 1) / kDtVecs;
        const T *zr = z + row * a.ldz;
        T *dzr = kGrad ? reinterpret_cast<T *>(a.dz) + row * a.lddz : nullptr;
        const bool aligned = kGrad && sh == (int)(((uintptr_t)dzr & 15u) / sizeof(T));
        // vectors [j0, j1) lie in the row; one before and one after may do so in part
        // (no copy covers the latter) and are done apart, by consumers 0 and 32
        const int j0 = sh ? 1 : 0, j1 = (sh + V) / NE;
        const int odd = tid == 0 && sh ? 0 : tid == 32 && nvec > j1 && nvec - 1 >= j0 ? nvec - 1 : -1;
        auto store_each = [&](int j, uint4 u) {
            const T *v = reinterpret_cast<const T *>(&u);
#pragma unroll
            for (int e = 0; e < NE; e++) {
                const int i = j * NE - sh + e;
                if (i >= 0 && i < V)
                    dzr[i] = v[e];
            }
        };
        auto store = [&](int j, uint4 u) {
            if (aligned && j >= j0 && j < j1)
                *reinterpret_cast<uint4 *>(dzr + j * NE - sh) = u;
            else
                store_each(j, u);
        };
        if (w == 0.0f) {  // the logits are not looked at
            if (kGrad)
                for (int j = tid; j < nvec; j += kDtConsumers)
                    store(j, make_uint4(0u, 0u, 0u, 0u));
            if (a.loss && tid == 0)
                a.loss[row] = 0.0f;
            logit_of(ahead, row + gridDim.x);
            continue;
        }

        const int idx = now.idx;
        const float zn = now.zn;
        float lp = now.lp;
        if (a.tail && idx >= 0)
            atomicOr(&s_bits[(sh + idx) >> 5], 1u << ((sh + idx) & 31));
        if (a.tail)
            named_sync(1, kDtConsumers);

        // vector j element by element: -inf outside the row
        auto odd_vector = [&](int j, float (&v)[NE]) {
#pragma unroll
            for (int e = 0; e < NE; e++) {
                const int i = j * NE - sh + e;
                v[e] = i < 0 || i >= V ? neg_inf() : Vec<T>::get(zr[i]);
            }
        };

        // without the named entries (rest class)
        auto leave_out = [&](int j, float (&v)[NE]) {
            const uint32_t bits = s_bits[(j * NE) >> 5] >> ((j * NE) & 31) & ((1u << NE) - 1u);
            if (bits) {
#pragma unroll
                for (int e = 0; e < NE; e++)
                    if (bits >> e & 1)
                        v[e] = neg_inf();
            }
        };

        // ---- first pass: running maximum and sum
        const int kept = kGrad ? max(0, n - slots) : n;   // chunks released after this pass
        Running run(limit, k2);
        int slot2 = 0;                                     // where the chunks that stay begin
        for (int c = 0; c < n; c++, next()) {
            if (c == kept)
                slot2 = slot;
            ok = ok && mbar_wait(&full[slot], phase);
            const uint8_t *at = s_ring + slot * kDtChunk;
            // a chunk wholly inside the row needs no checks
            auto sum_chunk = [&](auto inside) {
#pragma unroll
                for (int u = 0; u < kDtEach; u++) {
                    const int local = tid + u * kDtConsumers, j = c * kDtVecs + local;
                    if (decltype(inside)::value || (j >= j0 && j < j1)) {
                        float v[NE];
                        Vec<T>::unpack(*reinterpret_cast<const uint4 *>(at + local * 16), v);
                        if (a.tail)
                            leave_out(j, v);
                        run.add(v, k2, limit);
                    }
                }
            };
            if (c * kDtVecs >= j0 && (c + 1) * kDtVecs <= j1)
                sum_chunk(std::true_type());
            else
                sum_chunk(std::false_type());
            if (c < kept)
                release(slot);
        }
        if (odd >= 0) {
            float v[NE];
            odd_vector(odd, v);
            if (a.tail)
                leave_out(odd, v);
            run.add(v, k2, limit);
        }
        MaxSum all = run.result(k2);

        logit_of(ahead, row + gridDim.x);

        // ---- over the consumers: maxima first, then sums at the common maximum, in a fixed order
        const bool mine = idx >= 0;
        MaxSum named = {neg_inf(), 0.0f}, t = {neg_inf(), 0.0f};
        if (mine) {
            if (a.tail) {
                named = {zn, zn == neg_inf() ? 0.0f : 1.0f};
                t.s = expf(lp);  // only the plain sum is wanted
            } else {
                t = {lp, 1.0f};
            }
        }
        {
            const bool teach = warp * 32 < a.k;   // this warp holds entries
            const float m1 = teach ? warp_max(a.tail ? named.m : t.m) : neg_inf();
            float ma, mb;
            for (int again = 0;; again++) {
                const float m0 = warp_max(all.m);
                if (lane == 0) {
                    s_m[0][warp] = m0;
                    s_m[1][warp] = m1;
                }
                named_sync(1, kDtConsumers);
                ma = over_consumers_max(s_m[0], lane);
                mb = over_consumers_max(s_m[1], lane);
                if (again || usable(ma, limit))
                    break;
                named_sync(1, kDtConsumers);   // every thread has read s_m
                all = scan_any(tid, V, kDtConsumers, k2, [&](int i) {
                    return a.tail && (s_bits[(sh + i) >> 5] >> ((sh + i) & 31) & 1) ? neg_inf() : Vec<T>::get(zr[i]);
                });
            }
            const float sa = warp_sum(ok ? sum_at(all, ma, k2) : quiet_nan());
            float sn = 0.0f, st = 0.0f, cnt = 0.0f;
            if (teach) {
                sn = warp_sum(sum_at(named, mb, k2));
                st = warp_sum(a.tail ? t.s : sum_at(t, mb, k2));
                cnt = warp_sum(mine && (a.tail || lp != neg_inf()) ? 1.0f : 0.0f);
            }
            if (lane == 0) {
                s_s[0][warp] = sa;
                s_s[1][warp] = sn;
                s_s[2][warp] = st;
                s_s[3][warp] = cnt;
            }
            named_sync(1, kDtConsumers);
            if (a.tail && mine)
                s_bits[(sh + idx) >> 5] = 0u;   // every thread is done with the bits
            all = {ma, over_consumers_sum(s_s[0], lane)};
            if (a.tail)
                named = {mb, over_consumers_sum(s_s[1], lane)};
            t = {mb, over_consumers_sum(s_s[2], lane)};
        }
        const int seen = (int)over_consumers_sum(s_s[3], lane);   // at most 480: exact
        float mass = 1.0f, rest_p = 0.0f;
        if (a.tail) {
            // a NaN sum stays a NaN; a teacher that names the whole vocabulary leaves no rest
            rest_p = t.s > 1.0f || seen >= a.V ? 0.0f : 1.0f - t.s;
            mass = t.s + rest_p;
        } else {
            lp = (lp - finite_or_zero(t.m)) * inv_tau;
        }
        // q_v = 2^((z_v - base) k2) / total.s; a row of nothing but -inf gives NaN
        const MaxSum total = a.tail ? merge(all, named, k2) : all;
        const float base = finite_or_zero(total.m), rest_q = share_of(all, base, total.s, k2);
        float p = 0.0f;
        if (warp * 32 < a.k) {   // the others' s_f stays 0
            // p_j not from its logarithm, whose rounding would count where teacher and student nearly agree
            p = mine ? expf(lp) * (a.tail ? 1.0f : __frcp_rn(t.s)) : 0.0f;
            lp -= a.tail ? 0.0f : logf(t.s);
            if (a.loss) {
                float l = warp_sum(p != 0.0f ? p * (lp - ((zn - base) * inv_tau - logf(total.s))) : 0.0f);
                if (a.tail && warp == 0 && rest_p != 0.0f)
                    l += rest_p * (logf(rest_p) - log_share(rest_q, all, base, total.s, inv_tau));
                if (lane == 0)
                    s_f[warp] = seen ? l * w * a.tau * a.tau : 0.0f;
            }
        }

        // ---- second pass: the chunks in the ring, then the earlier ones again
        if (kGrad) {
            const float g = a.grad_loss ? a.grad_loss[a.grad_rows ? row : 0] : 1.0f;
            const float c0 = g * w * a.tau;
            const float dz_named = c0 * (mass * (expf((zn - base) * inv_tau) * __frcp_rn(total.s)) - p);
            const GradScale<T> scale(a, c0, all, total, mass, rest_p, rest_q, k2);
            // fast: whole vectors to 16-byte boundaries
            auto pass = [&](auto fast, auto neg) {
                constexpr bool kFast = decltype(fast)::value, kNeg = decltype(neg)::value;
                if (odd >= 0) {
                    float v[NE];
                    odd_vector(odd, v);
                    store_each(odd, seen ? scale.template apply<kFast, kNeg>(v) : make_uint4(0u, 0u, 0u, 0u));
                }
                for (int i = 0; i < n; i++) {
                    const bool stays = i < n - kept;
                    const int c = stays ? kept + i : i - (n - kept), at = stays ? slot2 : slot;
                    if (!stays)
                        ok = ok && mbar_wait(&full[slot], phase);
                    const uint8_t *src = s_ring + at * kDtChunk + tid * 16;
                    const int j = c * kDtVecs + tid;
                    if (!ok) {
                        const uint32_t nan = seen ? (sizeof(T) == 2 ? 0x7FC07FC0u : 0x7FC00000u) : 0u;
#pragma unroll 1
                        for (int u = 0; u < kDtEach; u++)
                            if (j + u * kDtConsumers >= j0 && j + u * kDtConsumers < j1)
                                store_each(j + u * kDtConsumers, make_uint4(nan, nan, nan, nan));
                    } else if (kFast && c * kDtVecs >= j0 && (c + 1) * kDtVecs <= j1) {
                        uint4 *dst = reinterpret_cast<uint4 *>(dzr + (int64_t)j * NE - sh);
                        // by two: all four need more than the 64 registers of two CTAs, and their spills
                        // cost 475 us instead of 402 at 4096 x 131072 (by two, 4 bytes are spilt in bf16)
#pragma unroll 2
                        for (int u = 0; u < kDtEach; u++) {
                            float v[NE];
                            Vec<T>::unpack(*reinterpret_cast<const uint4 *>(src + u * kDtConsumers * 16), v);
                            __stcs(dst + u * kDtConsumers, scale.template apply<kFast, kNeg>(v));
                        }
                    } else {
#pragma unroll 1
                        for (int u = 0; u < kDtEach; u++) {
                            const int ju = j + u * kDtConsumers;
                            if (ju >= j0 && ju < j1) {
                                float v[NE];
                                Vec<T>::unpack(*reinterpret_cast<const uint4 *>(src + u * kDtConsumers * 16), v);
                                const uint4 g4 = scale.template apply<kFast, kNeg>(v);
                                // without a teacher entry the gradient is 0, whatever the logits hold
                                if (kFast)
                                    __stcs(reinterpret_cast<uint4 *>(dzr + (int64_t)ju * NE - sh), g4);
                                else
                                    store_each(ju, seen ? g4 : make_uint4(0u, 0u, 0u, 0u));
                            }
                        }
                    }
                    release(at);
                    if (!stays)
                        next();
                    else if (++slot2 == slots)
                        slot2 = 0;
                }
            };
            scale.choose(aligned && seen != 0, pass);
            named_sync(1, kDtConsumers);  // the named entries are written over what the pass above stored
            if (mine && seen)
                dzr[idx] = Vec<T>::put(dz_named);
        } else {
            named_sync(1, kDtConsumers);
        }
        if (a.loss && warp == 0) {
            const float l = over_consumers_sum(s_f, lane);
            if (lane == 0)
                a.loss[row] = l;
        }
    }
    if (!ok && a.ctl && lane == 0)
        record_status(a.ctl, NVFP4_ERR_TIMEOUT);
}

// Shared memory of the stream kernel for V logits of `size` bytes: ring slots
// beside the bits of a rest class.
int stream_slots(const DistillArgs &a, size_t size)
{
    const int64_t bits = a.tail ? (a.V + (int64_t)(16 / size) + 31) / 32 * 4 : 0;
    return (int)std::min<int64_t>(kDtMaxSlots, (kDtSmem - bits) / kDtChunk);
}

template <typename T, bool kGrad>
cudaError_t run_distill_stream(const DistillArgs &a, int slots, cudaStream_t s, const DeviceInfo &dev)
{
    const size_t bits = a.tail ? (size_t)(a.V + (int64_t)(16 / sizeof(T)) + 31) / 32 * 4 : 0;
    const size_t smem = (size_t)slots * kDtChunk + bits;
    cudaError_t e = allow_smem<distill_stream_kernel<T, kGrad>>(kDtSmem, dev);
    if (e != cudaSuccess)
        return e;
    const unsigned grid = (unsigned)std::min<int64_t>(a.T, kDtPerSm * dev.num_sms);
    distill_stream_kernel<T, kGrad><<<grid, kDtThreads, smem, s>>>(a, slots);
    return cudaGetLastError();
}

template <typename T, bool kGrad, int kEntries>
cudaError_t run_distill(const DistillArgs &a, cudaStream_t s, const DeviceInfo &dev)
{
    // Cluster size: the smallest power of two whose slices are at most 72 KB,
    // so that three CTAs share an SM and one's copies run beside another's
    // arithmetic; with fewer rows than SMs the row is spread over more CTAs as
    // long as a slice is longer than 8 KB.
    const int64_t row_bytes = a.V * (int64_t)sizeof(T);
    int C = 1;
    while (C < 8 && (row_bytes > C * 73728LL || (a.T * C * 2 <= dev.num_sms && row_bytes > C * 8192LL)))
        C *= 2;
    constexpr int NE = Vec<T>::N;
    const int64_t L = ((a.V + C - 1) / C + NE - 1) / NE * NE;
    const size_t smem = (size_t)L * sizeof(T) + 32;
    cudaError_t e = allow_smem<distill_kernel<T, kGrad, kEntries>>(kDistillMaxSlice + 32, dev);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.T * C));
    cfg.blockDim = dim3(kDsThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, distill_kernel<T, kGrad, kEntries>, a, C, L);
}

// Clusters or the stream: bf16, loss and gradient, clusters / stream in us, rows
// of 131072 logits: 96 rows 16.0 / 19.4, 152 rows 27.0 / 21.7, 304 rows 44.3 /
// 35.6, 2432 rows 283 / 256 (all with plain stores); 2432 rows of 64 KB 54.3 /
// 79.5, of 96 KB 103.4 / 105.7.  The loss alone, 304 rows: 8 KB 4.0 / 5.0, 64 KB
// 5.7 / 7.2, 128 KB 16.3 / 10.4.  FP32 rows of 512 KB, with a gradient: 160 rows
// 49.5 / 45.4, 608 rows 146 / 138, 2432 rows 529 / 541; of 594 KB: 54.1 / 51.3,
// 159 / 161, 581 / 631; the loss alone, 608 rows of 512 KB 96.2 / 51.4, 2432 of
// 594 KB 368 / 208.  So the stream takes rows above 96 KB when there is one for
// every SM, as far as its threads hold the teacher's entries and its ring has
// two chunks; where thousands of rows above 512 KB want a gradient it loses 2 to
// 8 %, since L2 then holds little of what is read again.
//
// Within clusters, one entry a thread for up to 256 of them, else four: most
// teachers keep fewer than 256, and the other three's registers and branches
// cost every thread.
template <typename T, bool kGrad>
cudaError_t run_distill_k(const DistillArgs &a, cudaStream_t s, const DeviceInfo &dev)
{
    static_assert(kDistillMaxK == 4 * kDsThreads, "entries per thread");
    const int slots = stream_slots(a, sizeof(T));
    if (a.V * (int64_t)sizeof(T) > 98304 && a.T >= dev.num_sms && a.k <= kDtConsumers && slots >= 2)
        return run_distill_stream<T, kGrad>(a, slots, s, dev);
    return a.k <= kDsThreads ? run_distill<T, kGrad, 1>(a, s, dev) : run_distill<T, kGrad, 4>(a, s, dev);
}

}  // namespace

cudaError_t launch_distill(const DistillArgs &a, cudaStream_t s, const DeviceInfo &dev)
{
    if (a.dz)
        return a.z_fp32 ? run_distill_k<float, true>(a, s, dev) : run_distill_k<__nv_bfloat16, true>(a, s, dev);
    return a.z_fp32 ? run_distill_k<float, false>(a, s, dev) : run_distill_k<__nv_bfloat16, false>(a, s, dev);
}

}  // namespace nvfp4
