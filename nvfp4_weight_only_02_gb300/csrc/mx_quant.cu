// mx_quant.cu -- MXFP4: blocks of 32 elements along the contraction axis, one
// E8M0 byte per block, E2M1 codes.
//
// Mathematics.  For a block with largest magnitude a, the shared exponent is
// floor(log2 a) - 2 (the OCP microscaling rule; 2 = exponent of the grid's
// top binade [4, 8)), so with the FP32 exponent field f of a the E8M0 byte is
// max(f - 2, 0): integer arithmetic on the bits, subnormals included.  The
// scale is a power of two, so x / scale is one exact multiplication, a code
// is one rounding (nearest, ties to even, at most 6), and code times scale
// is exact in bf16.  A block that holds an infinity or a NaN has f = 255 and
// takes byte 255 (E8M0 NaN) and codes 0: its values are NaN, and so is every
// product that uses it.
//
// Scale layout.  The block-scaled tensor-core MMA takes scales through a copy
// of 32 lanes x 16 bytes, so they are kept in tiles of 128 rows x 4 blocks
// (512 bytes): byte 16 (r % 32) + 4 (r % 128 / 32) + j % 4 of tile
// (r / 128, j / 4).  Padding bytes are written as 0.
#include "common.cuh"
#include "internal.h"
#include "mx_codec.cuh"

namespace nvfp4 {

namespace {

constexpr int kMqTile = 128;     // rows and columns of a block's tile: one scale tile in each direction
constexpr int kMqThreads = 256;

// Two neighbouring columns of one row.
__device__ __forceinline__ float2 pair_floats(uint32_t v)
{
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
__device__ __forceinline__ float2 pair_floats(float2 v) { return v; }
// Running largest magnitudes of the two columns, and their bits as FP32 in the end.
struct PairMax16 {
    uint32_t m = 0u;
    __device__ __forceinline__ void add(uint32_t v) { m = __vmaxu2(m, v & 0x7FFF7FFFu); }
    __device__ __forceinline__ uint2 bits() const { return make_uint2(m << 16, m & 0xFFFF0000u); }
};
struct PairMax32 {
    uint2 m = {0u, 0u};
    __device__ __forceinline__ void add(float2 v)
    {
        m.x = max(m.x, __float_as_uint(v.x) & 0x7FFFFFFFu);
        m.y = max(m.y, __float_as_uint(v.y) & 0x7FFFFFFFu);
    }
    __device__ __forceinline__ uint2 bits() const { return m; }
};
template <typename T>
struct PairOf;
template <>
struct PairOf<__nv_bfloat16> {
    using type = uint32_t;
    using amax = PairMax16;
};
template <>
struct PairOf<float> {
    using type = float2;
    using amax = PairMax32;
};

// One 128 x 128 tile per block, read once.  Row direction: four lanes hold a
// block of 32 (16 bytes of input each), so loads, codes and values are
// coalesced.  Column direction: the tile goes through shared memory and a
// thread takes two neighbouring columns of a 32-row block.  Memory bound: at
// bf16 input it reads 2 bytes and writes 17/32 bytes an element and direction.
template <typename T, bool kRow, bool kCol>
__global__ void __launch_bounds__(kMqThreads)
    mx_quantize_kernel(const T *__restrict__ x, int64_t rows, int64_t cols, int64_t ld, uint8_t *__restrict__ codes,
                       uint8_t *__restrict__ scales, uint16_t *__restrict__ values, uint8_t *__restrict__ codes_t,
                       uint8_t *__restrict__ scales_t, uint16_t *__restrict__ values_t)
{
    extern __shared__ __align__(16) uint8_t s_tile_raw[];
    __shared__ __align__(16) uint8_t s_sc[512], s_sct[512];
    T *s_tile = reinterpret_cast<T *>(s_tile_raw);
    // A product launched behind this kernel starts its weight copies as soon as
    // every block is here; by then all kernels before this one are complete.
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t ctiles = (cols + kMqTile - 1) / kMqTile, rtiles = (rows + kMqTile - 1) / kMqTile;
    const int64_t rt = blockIdx.x / ctiles, ct = blockIdx.x % ctiles;
    const int64_t r0 = rt * kMqTile, c0 = ct * kMqTile;
    if (kCol && tid < 128)
        reinterpret_cast<uint32_t *>(s_sct)[tid] = 0u;

    const int lr = warp * 2 + (lane >> 4), c8 = (lane & 15) * 8;
    const bool cok = c0 + c8 < cols;
    Raw8<T> raw[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int64_t r = r0 + i * 16 + lr;
        if (cok && r < rows)
            raw[i].load(x + r * ld + c0 + c8);
        else
            raw[i].zero();
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const int rl = i * 16 + lr;
        const int64_t r = r0 + rl;
        if (kCol)
            raw[i].store(s_tile + rl * kMqTile + c8);
        if (kRow) {
            uint32_t m = raw[i].amax_bits();
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const uint32_t byte = e8m0_of(m);
            if ((lane & 3) == 0)
                s_sc[(rl & 31) * 16 + (rl >> 5) * 4 + (c8 >> 5)] = (uint8_t)byte;
            if (cok && r < rows) {
                float v[8];
                raw[i].floats(v);
                const uint32_t q = byte != 255u ? e2m1_encode8_scaled(v, e8m0_inverse(byte)) : 0u;
                if (codes)
                    *reinterpret_cast<uint32_t *>(codes + r * (cols / 2) + (c0 + c8) / 2) = q;
                if (values)
                    *reinterpret_cast<uint4 *>(values + r * cols + c0 + c8) = decode8_bf16(q, e8m0_scale(byte));
            }
        }
    }
    __syncthreads();
    if (kRow && scales && tid < 128)
        reinterpret_cast<uint32_t *>(scales + (rt * ctiles + ct) * 512)[tid] =
            reinterpret_cast<const uint32_t *>(s_sc)[tid];
    if (!kCol)
        return;

    const int64_t rows32 = (rows + 31) / 32 * 32;
    const int rb = warp & 3, c = (warp >> 2) * 64 + lane * 2;
    if (r0 + rb * 32 < rows && c0 + c < cols) {
        using P = typename PairOf<T>::type;
        P v[32];
        typename PairOf<T>::amax amax;
#pragma unroll
        for (int i = 0; i < 32; i++) {
            v[i] = *reinterpret_cast<const P *>(s_tile + (rb * 32 + i) * kMqTile + c);
            amax.add(v[i]);
        }
        const uint32_t b0 = e8m0_of(amax.bits().x), b1 = e8m0_of(amax.bits().y);
        s_sct[(c & 31) * 16 + (c >> 5) * 4 + rb] = (uint8_t)b0;
        s_sct[((c + 1) & 31) * 16 + (c >> 5) * 4 + rb] = (uint8_t)b1;
        const float i0 = b0 == 255u ? 0.0f : e8m0_inverse(b0), i1 = b1 == 255u ? 0.0f : e8m0_inverse(b1);
        uint32_t q0[4], q1[4];
#pragma unroll
        for (int g = 0; g < 4; g++) {
            float f0[8], f1[8];
#pragma unroll
            for (int e = 0; e < 8; e++) {
                const float2 f = pair_floats(v[8 * g + e]);
                f0[e] = f.x;
                f1[e] = f.y;
            }
            q0[g] = b0 == 255u ? 0u : e2m1_encode8_scaled(f0, i0);
            q1[g] = b1 == 255u ? 0u : e2m1_encode8_scaled(f1, i1);
        }
        if (codes_t) {
            uint8_t *dst = codes_t + (c0 + c) * (rows32 / 2) + (r0 + rb * 32) / 2;
            *reinterpret_cast<uint4 *>(dst) = make_uint4(q0[0], q0[1], q0[2], q0[3]);
            *reinterpret_cast<uint4 *>(dst + rows32 / 2) = make_uint4(q1[0], q1[1], q1[2], q1[3]);
        }
        if (values_t) {
            const float s0 = e8m0_scale(b0), s1 = e8m0_scale(b1);
#pragma unroll
            for (int g = 0; g < 4; g++) {
                uint32_t h0[4], h1[4];
                e2m1x8_to_h2x4(q0[g], h0);
                e2m1x8_to_h2x4(q1[g], h1);
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const float2 a = h2_to_f2(h0[e]), b = h2_to_f2(h1[e]);
                    const int64_t r = r0 + rb * 32 + 8 * g + 2 * e;
                    uint16_t *dst = values_t + r * cols + c0 + c;
                    if (r < rows)
                        *reinterpret_cast<uint32_t *>(dst) = pack_bf2(__fmul_rn(a.x, s0), __fmul_rn(b.x, s1));
                    if (r + 1 < rows)
                        *reinterpret_cast<uint32_t *>(dst + cols) = pack_bf2(__fmul_rn(a.y, s0), __fmul_rn(b.y, s1));
                }
            }
        }
    }
    __syncthreads();
    if (scales_t && tid < 128)
        reinterpret_cast<uint32_t *>(scales_t + (ct * rtiles + rt) * 512)[tid] =
            reinterpret_cast<const uint32_t *>(s_sct)[tid];
}

// Codes and tiled scales -> bf16 or FP32, eight elements a thread (exact).
template <bool kF32>
__global__ void __launch_bounds__(256)
    mx_dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, int64_t rows,
                         int64_t cols, void *__restrict__ out)
{
    const int64_t n8 = rows * (cols / 8), stride = (int64_t)gridDim.x * blockDim.x;
    const int64_t kt = (cols + 127) / 128;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n8; i += stride) {
        const int64_t r = i / (cols / 8), c = i % (cols / 8) * 8, j = c / 32;
        const uint32_t q = ld_stream_u32(codes + i * 4);
        const uint32_t byte = scales[((r >> 7) * kt + (j >> 2)) * 512 + (r & 31) * 16 + ((r & 127) >> 5) * 4 + (j & 3)];
        const float s = e8m0_scale(byte);
        if (kF32) {
            uint32_t h[4];
            e2m1x8_to_h2x4(q, h);
            float4 *dst = reinterpret_cast<float4 *>(out) + i * 2;
#pragma unroll
            for (int e = 0; e < 2; e++) {
                const float2 a = h2_to_f2(h[2 * e]), b = h2_to_f2(h[2 * e + 1]);
                dst[e] = make_float4(__fmul_rn(a.x, s), __fmul_rn(a.y, s), __fmul_rn(b.x, s), __fmul_rn(b.y, s));
            }
        } else {
            reinterpret_cast<uint4 *>(out)[i] = decode8_bf16(q, s);
        }
    }
}

// Row-major scale bytes (rows x nb) -> tiles, one 4-byte word a thread.
__global__ void __launch_bounds__(256) tile_scales_kernel(const uint8_t *__restrict__ in, int64_t rows, int64_t nb,
                                                          uint32_t *__restrict__ out)
{
    const int64_t kt = (nb + 3) / 4, words = (rows + 127) / 128 * kt * 128;
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < words; i += stride) {
        const int64_t tile = i >> 7, w = i & 127;
        const int64_t r = tile / kt * 128 + (w & 3) * 32 + (w >> 2), j = tile % kt * 4;
        uint32_t v = 0u;
        if (r < rows) {
#pragma unroll
            for (int e = 0; e < 4; e++)
                if (j + e < nb)
                    v |= (uint32_t)in[r * nb + j + e] << (8 * e);
        }
        out[i] = v;
    }
}

template <typename T, bool kRow, bool kCol>
cudaError_t run_quantize(const MxQuantArgs &a, cudaStream_t s, const DeviceInfo &dev)
{
    const int64_t tiles = ((a.rows + kMqTile - 1) / kMqTile) * ((a.cols + kMqTile - 1) / kMqTile);
    const size_t smem = kCol ? sizeof(T) * kMqTile * kMqTile : 0;
    if (smem > 48 * 1024) {
        const cudaError_t e = allow_smem<mx_quantize_kernel<T, kRow, kCol>>(smem, dev);
        if (e != cudaSuccess)
            return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)tiles);
    cfg.blockDim = dim3(kMqThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.overlap ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, mx_quantize_kernel<T, kRow, kCol>, (const T *)a.x, a.rows, a.cols, a.ld, a.codes,
                              a.scales, a.values, a.codes_t, a.scales_t, a.values_t);
}

template <typename T>
cudaError_t run_quantize_dirs(const MxQuantArgs &a, cudaStream_t s, const DeviceInfo &dev)
{
    const bool row = a.codes || a.values, col = a.codes_t || a.values_t;
    return row && col ? run_quantize<T, true, true>(a, s, dev)
           : row      ? run_quantize<T, true, false>(a, s, dev)
                      : run_quantize<T, false, true>(a, s, dev);
}

unsigned grid_for(int64_t n, const DeviceInfo &dev)
{
    const int64_t want = (n + 255) / 256, most = (int64_t)dev.num_sms * 8;
    return (unsigned)(want < most ? want : most);
}

}  // namespace

cudaError_t launch_mx_quantize(const MxQuantArgs &a, cudaStream_t s, const DeviceInfo &dev)
{
    return a.x_fp32 ? run_quantize_dirs<float>(a, s, dev) : run_quantize_dirs<__nv_bfloat16>(a, s, dev);
}

cudaError_t launch_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols, void *out,
                                 bool fp32, cudaStream_t s, const DeviceInfo &dev)
{
    const unsigned g = grid_for(rows * (cols / 8), dev);
    if (fp32)
        mx_dequantize_kernel<true><<<g, 256, 0, s>>>(codes, scales, rows, cols, out);
    else
        mx_dequantize_kernel<false><<<g, 256, 0, s>>>(codes, scales, rows, cols, out);
    return cudaGetLastError();
}

cudaError_t launch_tile_scales(const uint8_t *in, int64_t rows, int64_t nb, uint8_t *out, cudaStream_t s,
                               const DeviceInfo &dev)
{
    const int64_t words = (rows + 127) / 128 * ((nb + 3) / 4) * 128;
    tile_scales_kernel<<<grid_for(words, dev), 256, 0, s>>>(in, rows, nb, reinterpret_cast<uint32_t *>(out));
    return cudaGetLastError();
}

}  // namespace nvfp4
