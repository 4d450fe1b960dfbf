// int8_quant.cu -- rows of 8-bit integers with one scale a row.
//
// Mathematics.  With a the largest magnitude of a row, s = a / 127 (FP32) and
// q = the integer next to 127 x / a, ties to even.  127 x / a of bf16 or FP32
// numbers is a tie, or at least 2^-33 of itself away from one, so the decision
// in FP32 stands unless the quotient comes within 1e-4 of a tie; those few are
// divided in 64 bits, where the division is exact at ties.  A row of zeros has
// s = 0 and codes 0, a row with an infinity or a NaN s = NaN and codes 0.
//
// What bounds it: the bytes, read once: a CTA holds its row in registers (rows
// above 32768 elements are read twice, the second time from L2).
#include "common.cuh"
#include "internal.h"
#include "mx_codec.cuh"

namespace nvfp4 {

namespace {

constexpr int kIqThreads = 512, kIqHold = 8;   // groups of eight elements a thread holds

__device__ __forceinline__ float int8_round(float v, float inv, float amax)
{
    const float f = v * inv, r = rintf(f);
    // also taken where the reciprocal leaves FP32's range
    if (!(fabsf(f - r) < 0.4999f))
        return (float)rint((double)v * 127.0 / (double)amax);
    return r;
}

// kHalf: the integers as fp16 (exact), what the product's copies bring; else int8.
template <typename T, bool kHalf>
__global__ void __launch_bounds__(kIqThreads)
    int8_quantize_kernel(const T *__restrict__ x, int64_t ld, int64_t cols, void *__restrict__ out, float *__restrict__ scale)
{
    __shared__ uint32_t s_max[kIqThreads / 32];
    const int64_t row = blockIdx.x, n8 = cols / 8;
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    const T *src = x + row * ld;
    Raw8<T> held[kIqHold];
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < kIqHold; u++) {
        const int64_t i = tid + (int64_t)u * kIqThreads;
        held[u].zero();
        if (i < n8)
            held[u].load(src + i * 8);
    }
#pragma unroll
    for (int u = 0; u < kIqHold; u++)
        m = max(m, held[u].amax_bits());
    for (int64_t i = tid + (int64_t)kIqHold * kIqThreads; i < n8; i += kIqThreads) {
        Raw8<T> r;
        r.load(src + i * 8);
        m = max(m, r.amax_bits());
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((tid & 31) == 0)
        s_max[tid >> 5] = m;
    __syncthreads();
    m = s_max[tid & (kIqThreads / 32 - 1)];
    m = __reduce_max_sync(0xffffffffu, m);
    const bool bad = m >= 0x7F800000u;
    const float amax = __uint_as_float(m), inv = 127.0f / amax;
    if (tid == 0)
        scale[row] = bad ? __uint_as_float(0x7FC00000u) : __fdiv_rn(amax, 127.0f);
    auto put = [&](const Raw8<T> &r, int64_t i) {
        float v[8];
        r.floats(v);
#pragma unroll
        for (int e = 0; e < 8; e++)
            v[e] = bad || m == 0 ? 0.0f : int8_round(v[e], inv, amax);
        if (kHalf) {
            uint32_t h[4];
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const __half2 p = __floats2half2_rn(v[2 * e], v[2 * e + 1]);
                h[e] = *reinterpret_cast<const uint32_t *>(&p);
            }
            reinterpret_cast<uint4 *>(out)[row * n8 + i] = make_uint4(h[0], h[1], h[2], h[3]);
        } else {
            uint32_t w[2] = {0u, 0u};
#pragma unroll
            for (int e = 0; e < 8; e++)
                w[e / 4] |= ((uint32_t)(int)v[e] & 255u) << (8 * (e % 4));
            reinterpret_cast<uint2 *>(out)[row * n8 + i] = make_uint2(w[0], w[1]);
        }
    };
#pragma unroll
    for (int u = 0; u < kIqHold; u++) {
        const int64_t i = tid + (int64_t)u * kIqThreads;
        if (i < n8)
            put(held[u], i);
    }
    for (int64_t i = tid + (int64_t)kIqHold * kIqThreads; i < n8; i += kIqThreads) {
        Raw8<T> r;
        r.load(src + i * 8);
        put(r, i);
    }
}

// int8 -> fp16, 16 values a thread.
__global__ void __launch_bounds__(256) int8_widen_kernel(const uint8_t *__restrict__ in, int64_t n16, uint4 *__restrict__ out)
{
    pdl_wait();
    pdl_launch_dependents();
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n16)
        return;
    const uint4 q = ld_once_u4(in + i * 16);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 4; e++)
        int8x4_to_h2x2(w[e], h[2 * e], h[2 * e + 1]);
    out[2 * i] = make_uint4(h[0], h[1], h[2], h[3]);
    out[2 * i + 1] = make_uint4(h[4], h[5], h[6], h[7]);
}

}  // namespace

cudaError_t launch_int8_quantize(const Int8QuantArgs &a, cudaStream_t s)
{
    const dim3 grid((unsigned)a.rows);
    if (a.x_fp32)
        return a.half ? launch_dependent(int8_quantize_kernel<float, true>, grid, kIqThreads, 0, s, (const float *)a.x, a.ld,
                                         a.cols, a.out, a.scale)
                      : launch_dependent(int8_quantize_kernel<float, false>, grid, kIqThreads, 0, s, (const float *)a.x, a.ld,
                                         a.cols, a.out, a.scale);
    using B = __nv_bfloat16;
    return a.half ? launch_dependent(int8_quantize_kernel<B, true>, grid, kIqThreads, 0, s, (const B *)a.x, a.ld, a.cols,
                                     a.out, a.scale)
                  : launch_dependent(int8_quantize_kernel<B, false>, grid, kIqThreads, 0, s, (const B *)a.x, a.ld, a.cols,
                                     a.out, a.scale);
}

cudaError_t launch_int8_widen(const int8_t *in, int64_t n, void *out, cudaStream_t s)
{
    return launch_dependent(int8_widen_kernel, dim3((unsigned)((n / 16 + 255) / 256)), 256, 0, s, (const uint8_t *)in,
                            n / 16, (uint4 *)out);
}

}  // namespace nvfp4
