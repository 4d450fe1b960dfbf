// int8_codec.cuh -- a row of bf16 or FP32 numbers as 8-bit integers with one scale.
//
// Mathematics.  With a the largest magnitude of a row, s = a / 127 (FP32) and
// q = the integer next to 127 x / a, ties to even.  The product of x and 127 / a
// in FP32 decides unless it comes within 1e-4 of a tie h; then the sign of 127 x
// - h a does.  Both products are sums of two FP32 numbers (a product and its
// remainder by a fused multiply-add), their first halves are within a factor
// of two of one another and cancel exactly, so the sign is exact.  (Ties are not
// rare: where 254 / a is a power of two, a quarter of a bf16 row can be ties;
// decided by a division in 64 bits they took 52 us for 16 rows of 18944.)  Rows
// whose a is far from 1 are multiplied by a power of two first, so that no
// remainder underflows.  A row of zeros has s = 0 and codes 0, a row with an
// infinity or a NaN s = NaN and codes 0.
#pragma once

#include "common.cuh"
#include "mx_codec.cuh"

namespace nvfp4 {

__device__ __forceinline__ float int8_round(float v, float inv, float amax)
{
    const float a = fabsf(v), f = a * inv;
    float r = rintf(f);
    if (fabsf(f - r) >= 0.4999f) {
        // the nearest tie h, and the sign of 127 a - h amax from the products' exact halves (rounded here for
        // certain: a product that the compiler fused with th - ph would count its remainder twice)
        const float h = f >= r ? r + 0.5f : r - 0.5f;
        const float th = __fmul_rn(127.0f, a), tl = fmaf(127.0f, a, -th), ph = __fmul_rn(h, amax), pl = fmaf(h, amax, -ph);
        const float d = __fadd_rn(__fsub_rn(th, ph), __fsub_rn(tl, pl));
        r = d > 0.0f ? h + 0.5f : d < 0.0f ? h - 0.5f : rintf(h);
    }
    return copysignf(r, v);
}

// What a row's largest magnitude (its bits) makes of its elements.
struct Int8Row {
    float amax, bring, top, inv;
    bool none;   // codes 0
    __device__ __forceinline__ explicit Int8Row(uint32_t bits)
    {
        amax = __uint_as_float(bits);
        none = bits == 0u || bits >= 0x7F800000u;
        // exact: 2^100 below 2^-60; 2^-16 above 2^110, where only elements far below one step lose bits
        bring = amax < 0x1p-60f ? 0x1p100f : amax > 0x1p110f ? 0x1p-16f : 1.0f;
        top = amax * bring;
        inv = 127.0f / top;
    }
    __device__ __forceinline__ float scale() const
    {
        return amax < INFINITY ? __fdiv_rn(amax, 127.0f) : __uint_as_float(0x7FC00000u);
    }
    template <typename T>
    __device__ __forceinline__ void integers(const Raw8<T> &r, float (&v)[8]) const
    {
        r.floats(v);
#pragma unroll
        for (int e = 0; e < 8; e++)
            v[e] = none ? 0.0f : int8_round(v[e] * bring, inv, top);
    }
    // The integers as fp16 (exact).
    template <typename T>
    __device__ __forceinline__ uint4 halves(const Raw8<T> &r) const
    {
        float v[8];
        integers(r, v);
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const __half2 p = __floats2half2_rn(v[2 * e], v[2 * e + 1]);
            h[e] = *reinterpret_cast<const uint32_t *>(&p);
        }
        return make_uint4(h[0], h[1], h[2], h[3]);
    }
};

}  // namespace nvfp4
