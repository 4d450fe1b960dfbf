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
#include "common.cuh"
#include "internal.h"
#include "sm100.cuh"

namespace nvfp4 {

using namespace sm100;

namespace {

constexpr int kDsThreads = 256, kDsWarps = kDsThreads / 32;
constexpr int kDsEntries = kDistillMaxK / kDsThreads;  // teacher entries a thread holds
constexpr float kLog2e = 1.4426950408889634f;

// 2^x; results below 2^-126 are flushed to 0, which a sum of values in (0, 1]
// whose largest is 1 cannot notice.
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xFF800000u); }

// Running maximum m of logits and sum s of 2^((z - m) k2), k2 = log2(e) / tau.
// The difference is taken before the scaling: a row whose logits are all the
// type's lowest value is uniform, not a row of infinities.
struct MaxSum {
    float m, s;
};

__device__ __forceinline__ float finite_or_zero(float m) { return m == neg_inf() ? 0.0f : m; }

__device__ __forceinline__ MaxSum merge(MaxSum a, MaxSum b, float k2)
{
    const float m = fmaxf(a.m, b.m), base = finite_or_zero(m);
    return {m, a.s * ex2((a.m - base) * k2) + b.s * ex2((b.m - base) * k2)};
}

__device__ __forceinline__ MaxSum warp_merge(MaxSum v, float k2)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        MaxSum u;
        u.m = __shfl_xor_sync(0xffffffffu, v.m, o);
        u.s = __shfl_xor_sync(0xffffffffu, v.s, o);
        v = merge(v, u, k2);
    }
    return v;
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Every thread gets the block's merged value (the warps' in order).
__device__ __forceinline__ MaxSum block_merge(MaxSum v, float k2, MaxSum *s_w, int warp, int lane)
{
    v = warp_merge(v, k2);
    if (lane == 0)
        s_w[warp] = v;
    __syncthreads();
    MaxSum r = s_w[0];
#pragma unroll
    for (int i = 1; i < kDsWarps; i++)
        r = merge(r, s_w[i], k2);
    return r;
}

__device__ __forceinline__ void st_cluster_f4(uint32_t local, uint32_t rank, float4 v)
{
    asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
                 "st.shared::cluster.v4.f32 [a], {%2, %3, %4, %5};\n\t}" ::"r"(local),
                 "r"(rank), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

__device__ __forceinline__ void cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait()
{
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

// One row per cluster of C CTAs; CTA `rank` takes logits [rank L, rank L + L).
template <typename T, bool kGrad>
__global__ void __launch_bounds__(kDsThreads)
    distill_kernel(const __grid_constant__ DistillArgs a, int C, int64_t L)
{
    constexpr int NE = Vec<T>::N;
    extern __shared__ __align__(16) uint8_t s_raw[];
    __shared__ MaxSum s_w[3][kDsWarps];
    __shared__ float s_f[kDsWarps];
    __shared__ __align__(16) float4 s_x[8];   // each CTA's (max, sum) of the unnamed and of the named logits
    __shared__ __align__(16) float4 s_l[8];   // each CTA's share of the loss (rank 0's copy is used)
    __shared__ int s_seen;
    __shared__ __align__(8) uint64_t s_bar;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = C > 1 ? (int)cluster_ctarank() : 0;
    const int64_t row = blockIdx.x / C;
    const float w = a.weight ? a.weight[row] : 1.0f;
    const int64_t v0 = rank * L;
    const int64_t len64 = a.V - v0;
    const int len = (int)(len64 < 0 ? 0 : len64 < L ? len64 : L);

    // the slice sits at the address modulo 16 that it has in global memory
    const T *zrow = reinterpret_cast<const T *>(a.z) + row * a.ldz;
    const T *zs = zrow + v0;
    const int sh = (int)(((uintptr_t)zs & 15u) / sizeof(T));
    T *s_z = reinterpret_cast<T *>(s_raw);     // element i of the slice at s_z[sh + i]

    if (tid == 0) {
        mbar_init(&s_bar, 1);
        mbar_fence_init();
        s_seen = 0;
    }
    __syncthreads();
    if (C > 1)
        cluster_arrive();  // matched below: every CTA of the cluster runs before anyone writes to it

    const bool on = w != 0.0f;  // a NaN weight counts as a weight
    if (on && tid == 0 && len > 0) {
        const uint8_t *src = reinterpret_cast<const uint8_t *>(zs - sh);
        const uint32_t bytes = (uint32_t)(((int64_t)(sh + len) * (int)sizeof(T)) & ~15);
        mbar_arrive_expect_tx(&s_bar, bytes);
        for (uint32_t o = 0; o < bytes; o += 32768)
            bulk_g2s(s_raw + o, src + o, min(32768u, bytes - o), &s_bar);
    }

    // ---- the teacher's entries: four a thread, every CTA reads them all
    int idx[kDsEntries];    // in the vocabulary; -1: unused
    float lp[kDsEntries];   // log p_j (base e), -inf for an unused slot
    int seen = 0;           // entries that count: used ones (rest class), or ones with mass (renormalised)
    const float inv_tau = a.inv_tau, k2 = inv_tau * kLog2e;
    MaxSum t = {neg_inf(), 0.0f};
#pragma unroll
    for (int e = 0; e < kDsEntries; e++) {
        const int j = tid + e * kDsThreads;
        idx[e] = -1;
        lp[e] = neg_inf();
        if (on && j < a.k) {
            const int64_t at = row * a.k + j;
            const int64_t i = a.idx64 ? reinterpret_cast<const int64_t *>(a.idx)[at]
                                      : (int64_t)reinterpret_cast<const int32_t *>(a.idx)[at];
            if (i >= a.V) {
                if (a.ctl && rank == 0)
                    record_status(a.ctl, NVFP4_ERR_INDEX);
            } else if (i >= 0) {
                idx[e] = (int)i;
            }
            if (idx[e] >= 0) {
                const float tv = a.val_fp32 ? reinterpret_cast<const float *>(a.val)[at]
                                            : __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(a.val)[at]);
                lp[e] = tv;
                seen += a.tail || tv != neg_inf();
                // with a rest class only the plain sum of exp(t_j) is wanted: base 0
                t = merge(t, a.tail ? MaxSum{0.0f, ex2(tv * kLog2e)} : MaxSum{tv, 1.0f}, k2);
            }
        }
    }
    if (seen)
        atomicAdd(&s_seen, seen);
    t = block_merge(t, k2, s_w[0], warp, lane);   // also orders s_seen
    const bool live = on && s_seen != 0;
    float mass = 1.0f, rest_p = 0.0f;
    if (a.tail) {
        const float sum = t.m == neg_inf() ? 0.0f : t.s;
        // a NaN sum stays a NaN; a teacher that names the whole vocabulary leaves no rest
        rest_p = sum > 1.0f || s_seen >= a.V ? 0.0f : 1.0f - sum;
        mass = sum + rest_p;
    } else {
        const float base = finite_or_zero(t.m), log_s = logf(t.s);
#pragma unroll
        for (int e = 0; e < kDsEntries; e++)
            lp[e] = (lp[e] - base) * inv_tau - log_s;
    }

    T *dzs = kGrad ? reinterpret_cast<T *>(a.dz) + row * a.lddz + v0 : nullptr;
    const int shd = kGrad ? (int)(((uintptr_t)dzs & 15u) / sizeof(T)) : 0;
    const int nvec = len > 0 ? (sh + len + NE - 1) / NE : 0;

    bool ok = true;
    if (on && len > 0) {
        ok = mbar_wait(&s_bar, 0);   // also for rows that turn out empty: the copy lands in this CTA's memory
        if (!ok && a.ctl)
            record_status(a.ctl, NVFP4_ERR_TIMEOUT);
    }
    if (!live) {
        // weight 0 or no teacher entry: loss 0 and gradient 0, whatever the logits hold
        if (kGrad) {
            for (int j = tid; j < nvec; j += kDsThreads) {
                const int i0 = j * NE - sh;
                if (sh == shd && i0 >= 0 && i0 + NE <= len) {
                    *reinterpret_cast<uint4 *>(dzs + i0) = make_uint4(0u, 0u, 0u, 0u);
                } else {
#pragma unroll
                    for (int e = 0; e < NE; e++)
                        if (i0 + e >= 0 && i0 + e < len)
                            dzs[i0 + e] = Vec<T>::put(0.0f);
                }
            }
        }
        if (a.loss && rank == 0 && tid == 0)
            a.loss[row] = 0.0f;
        if (C > 1)
            cluster_wait();
        return;
    }

    // elements of the first and last 16 bytes outside the slice: -inf; the
    // last partial 16 bytes were not copied
    if (tid < 2 * NE && len > 0) {
        const int i = tid < NE ? tid - sh : (((sh + len) & ~(NE - 1)) + tid - NE) - sh;
        if (tid < NE ? i < 0 : true) {
            const bool in = i >= 0 && i < len;
            s_z[sh + i] = in ? zs[i] : Vec<T>::put(neg_inf());
        }
    }
    __syncthreads();

    // ---- logits of this CTA's named entries, then (rest class) their slots out of the sum
    float zn[kDsEntries];
    MaxSum named = {neg_inf(), 0.0f};
#pragma unroll
    for (int e = 0; e < kDsEntries; e++) {
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
        for (int e = 0; e < kDsEntries; e++)
            if (idx[e] >= 0)
                s_z[sh + idx[e] - v0] = Vec<T>::put(neg_inf());
        __syncthreads();
    }

    // ---- one pass: running maximum and sum
    MaxSum all = {neg_inf(), 0.0f};
    for (int j = tid; j < nvec; j += kDsThreads) {
        float v[NE];
        Vec<T>::unpack(*reinterpret_cast<const uint4 *>(s_raw + (size_t)j * 16), v);
        float m = v[0];
#pragma unroll
        for (int e = 1; e < NE; e++)
            m = fmaxf(m, v[e]);
        if (m > all.m) {
            all.s *= ex2((all.m - m) * k2);
            all.m = m;
        }
        const float base = finite_or_zero(all.m);
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < NE; e++)
            s += ex2((v[e] - base) * k2);
        all.s += s;
    }
    all = block_merge(all, k2, s_w[1], warp, lane);
    if (a.tail)
        named = block_merge(named, k2, s_w[2], warp, lane);
    if (C > 1) {
        cluster_wait();
        if (tid < C)
            st_cluster_f4(smem_addr(&s_x[rank]), (uint32_t)tid, make_float4(all.m, all.s, named.m, named.s));
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        all = {s_x[0].x, s_x[0].y};
        named = {s_x[0].z, s_x[0].w};
        for (int i = 1; i < C; i++) {
            all = merge(all, MaxSum{s_x[i].x, s_x[i].y}, k2);
            if (a.tail)
                named = merge(named, MaxSum{s_x[i].z, s_x[i].w}, k2);
        }
    }
    // log2 q_v = (z_v - total.m) k2 - log2_total; a row of nothing but -inf has
    // total.s = 0 and gives NaN
    const MaxSum total = a.tail ? merge(all, named, k2) : all;
    const float base = finite_or_zero(total.m), log2_total = log2f(total.s);
    constexpr float kLn2 = 0.6931471805599453f;
    // log2 of q_r, the share of the entries that are not named
    const float log2_rest = (all.m - base) * k2 + log2f(all.s) - log2_total;

    // ---- this CTA's share of the loss, sent to rank 0 while the gradient is written
    if (a.loss) {
        float l = 0.0f;
#pragma unroll
        for (int e = 0; e < kDsEntries; e++) {
            if (idx[e] >= 0) {
                const float p = ex2(lp[e] * kLog2e);
                if (p != 0.0f)
                    l += p * (lp[e] - ((zn[e] - base) * inv_tau - log2_total * kLn2));
            }
        }
        l = warp_sum(l);
        if (lane == 0)
            s_f[warp] = l;
        __syncthreads();
        if (tid == 0) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kDsWarps; i++)
                sum += s_f[i];
            if (C > 1)
                st_cluster_f4(smem_addr(&s_l[rank]), 0u, make_float4(sum, 0.0f, 0.0f, 0.0f));
            else
                s_l[0].x = sum;
        }
    }
    __syncwarp();
    if (C > 1)
        cluster_arrive();

    if (kGrad) {
        const float g = a.grad_loss ? a.grad_loss[a.grad_rows ? row : 0] : 1.0f;
        const float c = g * w * a.tau;
        // Entries not named: c q_v P, or with a rest class c (P q_r - p_r) u_v with
        // u the softmax over them alone, so that a q_r below FP32's range costs
        // nothing.  A rest without any mass (all.s = 0) has no gradient.
        const bool none = a.tail && all.s == 0.0f && total.s != 0.0f;
        const float bu = a.tail ? finite_or_zero(all.m) : base;
        const float lu = a.tail ? (none ? 0.0f : log2f(all.s)) : log2_total;
        const float cu = a.tail ? c * (mass * ex2(log2_rest) - rest_p) : c * mass;
        for (int j = tid; j < nvec; j += kDsThreads) {
            float v[NE];
            Vec<T>::unpack(*reinterpret_cast<const uint4 *>(s_raw + (size_t)j * 16), v);
#pragma unroll
            for (int e = 0; e < NE; e++)
                v[e] = cu * ex2((v[e] - bu) * k2 - lu);
            const int i0 = j * NE - sh;
            if (sh == shd && i0 >= 0 && i0 + NE <= len) {
                *reinterpret_cast<uint4 *>(dzs + i0) = Vec<T>::pack(v);
            } else {
#pragma unroll
                for (int e = 0; e < NE; e++)
                    if (i0 + e >= 0 && i0 + e < len)
                        dzs[i0 + e] = Vec<T>::put(v[e]);
            }
        }
        __syncthreads();   // the named entries are written over what the pass above stored
#pragma unroll
        for (int e = 0; e < kDsEntries; e++)
            if (idx[e] >= 0)
                dzs[idx[e] - v0] = Vec<T>::put(c * (mass * ex2((zn[e] - base) * k2 - log2_total) - ex2(lp[e] * kLog2e)));
    }
    if (C > 1)
        cluster_wait();
    if (a.loss && rank == 0 && tid == 0) {
        float l = 0.0f;
        for (int i = 0; i < C; i++)
            l += s_l[i].x;
        if (a.tail && rest_p != 0.0f)
            l += rest_p * (logf(rest_p) - log2_rest * kLn2);
        a.loss[row] = l * w * a.tau * a.tau;
    }
}

template <typename T, bool kGrad>
cudaError_t run_distill(const DistillArgs &a, cudaStream_t s, const DeviceInfo &dev)
{
    // Cluster size: the smallest power of two whose slices are at most 40 KB,
    // so that four or more CTAs share an SM and one's copies run beside
    // another's arithmetic; with fewer rows than SMs the row is spread over
    // more CTAs, down to slices of 4 KB.
    const int64_t row_bytes = a.V * (int64_t)sizeof(T);
    int C = 1;
    while (C < 8 && (row_bytes > C * 40960LL || (a.T * C * 2 <= dev.num_sms && row_bytes > C * 8192LL)))
        C *= 2;
    constexpr int NE = Vec<T>::N;
    const int64_t L = ((a.V + C - 1) / C + NE - 1) / NE * NE;
    const size_t smem = (size_t)L * sizeof(T) + 32;
    cudaError_t e = cudaFuncSetAttribute(distill_kernel<T, kGrad>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)kDistillMaxSlice + 32);
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
    return cudaLaunchKernelEx(&cfg, distill_kernel<T, kGrad>, a, C, L);
}

}  // namespace

cudaError_t launch_distill(const DistillArgs &a, cudaStream_t s, const DeviceInfo &dev)
{
    if (a.dz)
        return a.z_fp32 ? run_distill<float, true>(a, s, dev) : run_distill<__nv_bfloat16, true>(a, s, dev);
    return a.z_fp32 ? run_distill<float, false>(a, s, dev) : run_distill<__nv_bfloat16, false>(a, s, dev);
}

}  // namespace nvfp4
