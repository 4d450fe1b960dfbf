// int8_quant.cu -- rows of 8-bit integers with one scale a row (int8_codec.cuh has
// the mathematics).
//
// What bounds it: the bytes, read once: a CTA holds its row in registers (what
// lies beyond 20480 elements is read twice, the second time from L2).
#include "common.cuh"
#include "int8_codec.cuh"
#include "internal.h"
#include "mx_codec.cuh"

namespace nvfp4 {

namespace {

constexpr int kIqMax = 512;   // threads of a CTA at most

// kHalf: the integers as fp16 (exact), what the product's copies bring; else int8.  kHold: groups of eight elements that
// a thread holds.
template <typename T, bool kHalf, int kHold>
__global__ void __launch_bounds__(kIqMax)
    int8_quantize_kernel(const T *__restrict__ x, int64_t ld, int64_t cols, void *__restrict__ out, float *__restrict__ scale)
{
    __shared__ uint32_t s_max[kIqMax / 32];
    const int64_t row = blockIdx.x, n8 = cols / 8;
    const int tid = threadIdx.x, threads = blockDim.x;
    pdl_wait();
    pdl_launch_dependents();
    const T *src = x + row * ld;
    Raw8<T> held[kHold];
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < kHold; u++) {
        const int64_t i = tid + (int64_t)u * threads;
        held[u].zero();
        if (i < n8)
            held[u].load(src + i * 8);
    }
#pragma unroll
    for (int u = 0; u < kHold; u++)
        m = max(m, held[u].amax_bits());
    for (int64_t i = tid + (int64_t)kHold * threads; i < n8; i += threads) {
        Raw8<T> r;
        r.load(src + i * 8);
        m = max(m, r.amax_bits());
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if ((tid & 31) == 0)
        s_max[tid >> 5] = m;
    __syncthreads();
    m = (tid & 31) < threads / 32 ? s_max[tid & 31] : 0u;
    m = __reduce_max_sync(0xffffffffu, m);
    const Int8Row q(m);
    if (tid == 0)
        scale[row] = q.scale();
    auto put = [&](const Raw8<T> &r, int64_t i) {
        if (kHalf) {
            reinterpret_cast<uint4 *>(out)[row * n8 + i] = q.halves(r);
        } else {
            float v[8];
            q.integers(r, v);
            uint32_t w[2] = {0u, 0u};
#pragma unroll
            for (int e = 0; e < 8; e++)
                w[e / 4] |= ((uint32_t)(int)v[e] & 255u) << (8 * (e % 4));
            reinterpret_cast<uint2 *>(out)[row * n8 + i] = make_uint2(w[0], w[1]);
        }
    };
#pragma unroll
    for (int u = 0; u < kHold; u++) {
        const int64_t i = tid + (int64_t)u * threads;
        if (i < n8)
            put(held[u], i);
    }
    for (int64_t i = tid + (int64_t)kHold * threads; i < n8; i += threads) {
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

template <typename T, bool kHalf>
cudaError_t run_rows(const Int8QuantArgs &a, cudaStream_t s)
{
    // four or five groups a thread: loads in flight, and few warps to meet for the maximum; one each in rows of up to 128
    const int64_t n8 = a.cols / 8;
    const dim3 grid((unsigned)a.rows);
    if (n8 <= 128)
        return launch_dependent(int8_quantize_kernel<T, kHalf, 1>, grid, (int)((n8 + 31) / 32 * 32), 0, s, (const T *)a.x,
                                a.ld, a.cols, a.out, a.scale);
    if (n8 <= 1024)
        return launch_dependent(int8_quantize_kernel<T, kHalf, 4>, grid, n8 <= 512 ? 128 : 256, 0, s, (const T *)a.x, a.ld,
                                a.cols, a.out, a.scale);
    return launch_dependent(int8_quantize_kernel<T, kHalf, 5>, grid, kIqMax, 0, s, (const T *)a.x, a.ld, a.cols, a.out,
                            a.scale);
}

template <typename T>
cudaError_t run_quantize(const Int8QuantArgs &a, cudaStream_t s)
{
    return a.half ? run_rows<T, true>(a, s) : run_rows<T, false>(a, s);
}

}  // namespace

cudaError_t launch_int8_quantize(const Int8QuantArgs &a, cudaStream_t s)
{
    return a.x_fp32 ? run_quantize<float>(a, s) : run_quantize<__nv_bfloat16>(a, s);
}

cudaError_t launch_int8_widen(const int8_t *in, int64_t n, void *out, cudaStream_t s)
{
    return launch_dependent(int8_widen_kernel, dim3((unsigned)((n / 16 + 255) / 256)), 256, 0, s, (const uint8_t *)in,
                            n / 16, (uint4 *)out);
}

}  // namespace nvfp4
