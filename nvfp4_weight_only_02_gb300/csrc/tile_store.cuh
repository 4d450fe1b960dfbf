// tile_store.cuh -- accumulators with the output's columns on TMEM lanes and its
// rows on TMEM columns, on their way to a row-major matrix.
//
// Four warps have 128 lanes x 32 columns at a time: 128 outputs n of 32 rows.
// Stored straight from the lanes, a warp would write 64 bytes (bf16) of a row an
// instruction.  In bf16 the accumulator is loaded in the fragment layout (a thread
// has two neighbouring rows of an output), packed, and written transposed to
// shared memory by stmatrix; in FP32 a lane writes its output of each row.  The
// four warps then read shared memory 16 bytes a lane and store whole pieces of
// rows, 256 (512) bytes each: 19456 rows of 8 experts of 2048 x 2048 take 40.3 us in
// FP32 and 34.5 in bf16, 44.0 and 34.0 with element stores, 28 without any.
#pragma once

#include "common.cuh"
#include "sm100.cuh"

namespace nvfp4 {

using namespace sm100;

constexpr int kStageOut = 8192;   // bytes of shared memory for four warps

// Lanes 0-15 and 16-31 of a warp's quarter, 32 columns each, fragment layout: v[16 h + 4 j + r] is lane 16 h + 8 (r /
// 2) + T / 4, column 8 j + 2 (T % 4) + r % 2 of thread T.
__device__ __forceinline__ void tmem_ld_frag_start(uint32_t taddr, uint32_t (&v)[32])
{
#pragma unroll
    for (int h = 0; h < 2; h++)
        asm volatile(
            "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(v[16 * h]), "=r"(v[16 * h + 1]), "=r"(v[16 * h + 2]), "=r"(v[16 * h + 3]), "=r"(v[16 * h + 4]),
              "=r"(v[16 * h + 5]), "=r"(v[16 * h + 6]), "=r"(v[16 * h + 7]), "=r"(v[16 * h + 8]), "=r"(v[16 * h + 9]),
              "=r"(v[16 * h + 10]), "=r"(v[16 * h + 11]), "=r"(v[16 * h + 12]), "=r"(v[16 * h + 13]), "=r"(v[16 * h + 14]),
              "=r"(v[16 * h + 15])
            : "r"(taddr + ((uint32_t)(16 * h) << 16)));
}

// The load that store_rows of this type wants.
template <bool kF32>
__device__ __forceinline__ void tile_ld_start(uint32_t taddr, uint32_t (&v)[32])
{
    if constexpr (kF32)
        tmem_ld32_start(taddr, v);
    else
        tmem_ld_frag_start(taddr, v);
}

__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}

// Rows row0 .. row0 + left - 1 (32 at most) of y (row-major, N columns), columns n0 .. n0 + 127 as far as they exist, by
// the four warps of a group; v: quarter `quad` of the lanes.  stage: the group's kStageOut bytes, bar: its named barrier.
// All four warps make the same calls, whatever happens, with write = false where there is nothing to be written.
template <bool kF32>
__device__ __forceinline__ void store_rows(const uint32_t (&v)[32], uint8_t *stage, int bar, void *y, int64_t row0, int left,
                                           int N, int n0, int quad, int lane, bool write)
{
    if constexpr (kF32) {
        float *out = reinterpret_cast<float *>(y) + row0 * N + n0;
        // 16 rows of 512 bytes at a time
#pragma unroll
        for (int h = 0; h < 2; h++) {
            if (16 * h >= left)
                break;
            named_sync(bar, 128);
#pragma unroll
            for (int t = 0; t < 16; t++)
                *reinterpret_cast<uint32_t *>(stage + t * 512 + quad * 128 + lane * 4) = v[16 * h + t];
            named_sync(bar, 128);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int t = 4 * quad + i;
                if (!write || 16 * h + t >= left)
                    continue;
                float *dst = out + (int64_t)(16 * h + t) * N;
                const uint8_t *src = stage + t * 512;
                if (N % 4 == 0) {
                    if (n0 + 4 * lane < N)
                        *reinterpret_cast<uint4 *>(dst + 4 * lane) = *reinterpret_cast<const uint4 *>(src + lane * 16);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        if (n0 + 32 * e + lane < N)
                            dst[32 * e + lane] = *reinterpret_cast<const float *>(src + (32 * e + lane) * 4);
                }
            }
        }
    } else {
        __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(y) + row0 * N + n0;
        auto pack = [](uint32_t a, uint32_t b) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(a), __uint_as_float(b));
            return *reinterpret_cast<const uint32_t *>(&h);
        };
        // rows of 256 bytes, 16-byte pieces exchanged so that neither side meets a bank twice
        auto at = [](int t, int q) { return t * 256 + ((q ^ (t & 7)) << 4); };
        named_sync(bar, 128);
#pragma unroll
        for (int j = 0; j < 4; j++)
            stmatrix_x4_trans(smem_addr(stage) + at(8 * j + (lane & 7), 4 * quad + (lane >> 3)), pack(v[4 * j], v[4 * j + 1]),
                              pack(v[4 * j + 2], v[4 * j + 3]), pack(v[16 + 4 * j], v[16 + 4 * j + 1]),
                              pack(v[16 + 4 * j + 2], v[16 + 4 * j + 3]));
        named_sync(bar, 128);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int t = 8 * quad + 2 * i + (lane >> 4), q = lane & 15;
            if (!write || t >= left)
                continue;
            __nv_bfloat16 *dst = out + (int64_t)t * N;
            if (N % 8 == 0) {
                if (n0 + 8 * q < N)
                    *reinterpret_cast<uint4 *>(dst + 8 * q) = *reinterpret_cast<const uint4 *>(stage + at(t, q));
            } else {
                // eight columns a lane, 16 apart, so that a half warp's stores are neighbours
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const int n = 16 * e + q;
                    if (n0 + n < N)
                        dst[n] = *reinterpret_cast<const __nv_bfloat16 *>(stage + at(t, n >> 3) + (n & 7) * 2);
                }
            }
        }
    }
}

}  // namespace nvfp4
