// mx_codec.cuh -- MXFP4 blocks in registers: the E8M0 byte, E2M1 codes and their
// values, from bf16 or FP32 elements (the format is described in mx_quant.cu).
#pragma once

#include "common.cuh"

namespace nvfp4 {

// Eight floats -> eight E2M1 codes (element 0 in the low nibble).
__device__ __forceinline__ uint32_t e2m1_encode8(const float (&v)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Eight floats times a power of two -> eight codes (two products an instruction).
__device__ __forceinline__ uint32_t e2m1_encode8_scaled(const float (&v)[8], float f)
{
    float u[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2)
        asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmul.rn.f32x2 a, a, b;\n\t"
            "mov.b64 {%0, %1}, a;\n\t}"
            : "=f"(u[i]), "=f"(u[i + 1])
            : "f"(v[i]), "f"(v[i + 1]), "f"(f));
    return e2m1_encode8(u);
}

// The block's E8M0 byte from the magnitude bits of its largest element.
__device__ __forceinline__ uint32_t e8m0_of(uint32_t amax_bits)
{
    const uint32_t f = amax_bits >> 23;
    return f == 255u ? 255u : f > 2u ? f - 2u : 0u;
}

// 2^(byte - 127); byte 255 gives a NaN.
__device__ __forceinline__ float e8m0_scale(uint32_t byte)
{
    return byte == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

// 2^(127 - byte) for byte <= 252.
__device__ __forceinline__ float e8m0_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi)
{
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}

__device__ __forceinline__ float2 h2_to_f2(uint32_t h)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Eight codes times their block scale as bf16 pairs (exact).
__device__ __forceinline__ uint4 decode8_bf16(uint32_t codes, float scale)
{
    uint32_t h[4];
    e2m1x8_to_h2x4(codes, h);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 f = h2_to_f2(h[i]);
        o[i] = pack_bf2(__fmul_rn(f.x, scale), __fmul_rn(f.y, scale));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Eight consecutive elements as magnitude-preserving floats, from the raw
// 16-byte words of a row (bf16: one word, FP32: two).
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = ld_once_u4(p); }
    __device__ __forceinline__ void store_shared(__nv_bfloat16 *p) const { *reinterpret_cast<uint4 *>(p) = a; }
    __device__ __forceinline__ void zero() { a = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void floats(float (&v)[8]) const
    {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    // Codes under the scale that the block's largest magnitude gives; its byte
    __device__ __forceinline__ uint32_t encode(uint32_t amax, uint32_t &byte) const
    {
        byte = e8m0_of(amax);
        // 2^(127 - byte) twice; the products are exact (or far below the smallest code)
        const uint32_t f = (254u - byte) * 0x00800080u;
        const __nv_bfloat162 ff = *reinterpret_cast<const __nv_bfloat162 *>(&f);
        const uint4 u = make_uint4(mul(a.x, ff), mul(a.y, ff), mul(a.z, ff), mul(a.w, ff));
        Raw8 scaled;
        scaled.a = u;
        float v[8];
        scaled.floats(v);
        return byte == 255u ? 0u : e2m1_encode8(v);
    }
    static __device__ __forceinline__ uint32_t mul(uint32_t x, __nv_bfloat162 f)
    {
        const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&x), f);
        return *reinterpret_cast<const uint32_t *>(&y);
    }
    __device__ __forceinline__ uint32_t amax_bits() const
    {
        const uint32_t k = 0x7FFF7FFFu;
        const uint32_t m = __vmaxu2(__vmaxu2(a.x & k, a.y & k), __vmaxu2(a.z & k, a.w & k));
        return max(m << 16, m & 0xFFFF0000u);
    }
};
template <>
struct Raw8<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = ld_once_u4(p);
        b = ld_once_u4(p + 4);
    }
    __device__ __forceinline__ void store_shared(float *p) const
    {
        reinterpret_cast<uint4 *>(p)[0] = a;
        reinterpret_cast<uint4 *>(p)[1] = b;
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0u, 0u, 0u, 0u); }
    __device__ __forceinline__ void floats(float (&v)[8]) const
    {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; i++)
            v[i] = __uint_as_float(w[i]);
    }
    __device__ __forceinline__ uint32_t encode(uint32_t amax, uint32_t &byte) const
    {
        byte = e8m0_of(amax);
        float v[8];
        floats(v);
        return byte == 255u ? 0u : e2m1_encode8_scaled(v, e8m0_inverse(byte));
    }
    __device__ __forceinline__ uint32_t amax_bits() const
    {
        const uint32_t k = 0x7FFFFFFFu;
        return max(max(max(a.x & k, a.y & k), max(a.z & k, a.w & k)),
                   max(max(b.x & k, b.y & k), max(b.z & k, b.w & k)));
    }
};

}  // namespace nvfp4
