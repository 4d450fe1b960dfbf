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

constexpr int kMqRows = 128;      // rows of a tile

// What depends on the input's type.  A tile is 128 rows of 256 bytes: 128 bf16
// columns (one scale tile in each direction) or 64 FP32 ones (half of one).  In
// the column direction a thread takes kPer neighbouring columns of 32 rows.
template <typename T>
struct MqShape;
template <>
struct MqShape<__nv_bfloat16> {
    static constexpr int kCols = 128, kPer = 2;
    using Word = uint32_t;       // kPer columns of a row
    uint32_t m = 0u;             // running largest magnitudes
    __device__ __forceinline__ void add(uint32_t v) { m = __vmaxu2(m, v & 0x7FFF7FFFu); }
    __device__ __forceinline__ uint32_t amax_bits(int i) const { return i ? m & 0xFFFF0000u : m << 16; }
    static __device__ __forceinline__ float value(uint32_t v, int i)
    {
        return __uint_as_float(i ? v & 0xFFFF0000u : v << 16);
    }
};
template <>
struct MqShape<float> {
    static constexpr int kCols = 64, kPer = 1;
    using Word = float;
    uint32_t m = 0u;
    __device__ __forceinline__ void add(float v) { m = max(m, __float_as_uint(v) & 0x7FFFFFFFu); }
    __device__ __forceinline__ uint32_t amax_bits(int) const { return m; }
    static __device__ __forceinline__ float value(float v, int) { return v; }
};

struct MqParams {
    int64_t rows, cols;
    int64_t ctiles;   // tiles along a row
    uint8_t *codes, *scales, *codes_t, *scales_t;
    uint16_t *values, *values_t;
    MoeRows moe;      // grouped rows: where they come from
};

// Where a tile's rows come from and go to: a matrix; one of several behind one
// another (blockIdx.y); rows grouped by expert, gathered into blocks of 128
// that belong to one expert each.
enum MqSource { kMatrix, kBatch, kExpertRows };

// One read of x for both directions, a tile a CTA: 16 bytes a thread and row
// at a time, all of them on their way before the first is used.  Row direction,
// from registers: four lanes hold a block of 32 (eight elements each), so codes
// and values are coalesced.  Column direction: the tile goes through shared
// memory, a thread takes its columns of a 32-row block; the codes return there
// too and leave as 64 contiguous bytes a column.  Rows and columns outside the
// matrix are zeros, so padding bytes of the scale tiles come out as 0 by
// themselves.
//
// What bounds it: 2 (4) bytes read and 17/32 written an element and direction.
// 16384 x 3584 bf16: rows alone 23.2 us (6.4 TB/s, 94 % of the copy rate), with
// values 41.9 us (94 %); columns alone 30.1 us (73 %); both 37.8 us (70 %), with
// values 65.9 us (93 %).  8192 x 3584 FP32, both: 32.0 us (68 %).  Both directions
// are bound by issue, 17 instructions an element: 71 % of the slots over the
// whole kernel, and a warp waits for its slot longer than for anything else; the
// rest goes to the first loads and to shared memory (40 % of its wavefronts are
// bank conflicts).
// Measured against it, both directions: codes straight from the column pass's
// registers, 16 bytes a column, 40.9 us; a persistent CTA with tiles brought by
// TMA 41.5 us (rows 26.2); registers capped for five CTAs an SM 44.5 us.
constexpr int kMqThreads = 256;

template <typename T, bool kRow, bool kCol, MqSource kSource>
__global__ void __launch_bounds__(kMqThreads)
    mx_quantize_kernel(const T *__restrict__ x, const int64_t ld, const MqParams params)
{
    MqParams p = params;
    using S = MqShape<T>;
    constexpr int kCols = S::kCols, kPer = S::kPer, kGroups = kCols / 32;   // 32-column groups of a tile
    constexpr int kLanes = kCols / 8, kStep = kMqThreads / kLanes;          // lanes to a row, rows at a time
    constexpr int kIter = kMqRows / kStep;
    __shared__ __align__(16) T tile[kCol ? kMqRows * kCols : 1];
    __shared__ uint32_t s_sc[kMqRows], s_sct[kCols];   // the tile's scale bytes, a word a row (column)
    __shared__ uint4 s_q[kCol ? kCols * 5 : 1];        // the tile's codes in the column direction, 80 bytes a column
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t rows = p.rows, cols = p.cols, rows32 = (rows + 31) / 32 * 32;
    const int64_t rtiles = (rows + kMqRows - 1) / kMqRows, ktiles = (cols + 127) / 128;
    const int64_t rt = blockIdx.x / p.ctiles, ct = blockIdx.x % p.ctiles, r0 = rt * kMqRows, c0 = ct * kCols;
    int left = (int)min(rows - r0, (int64_t)kMqRows);                       // rows of the tile that exist
    // A product launched behind this kernel starts its weight copies as soon as
    // every block is here; by then all kernels before this one are complete.
    pdl_wait();
    pdl_launch_dependents();
    if constexpr (kSource == kBatch) {
        const int64_t b = blockIdx.y;
        x += b * rows * ld;
        p.codes += p.codes ? b * rows * (cols / 2) : 0;
        p.scales += p.scales ? b * rtiles * ktiles * 512 : 0;
        p.codes_t += p.codes_t ? b * cols * (rows32 / 2) : 0;
        p.scales_t += p.scales_t ? b * ktiles * rtiles * 512 : 0;
    }
    int64_t row0 = 0;        // grouped: the block's first row
    if constexpr (kSource == kExpertRows) {
        if (rt >= p.moe.header[1])
            return;
        const int4 block = p.moe.blocks[rt];
        row0 = block.z;
        left = block.w;
    }
    // rows of the tile in the column direction: a group's last block is padded with zeros
    const int cleft = kSource == kExpertRows ? kMqRows : left;

    const int lr = tid / kLanes, c8 = tid % kLanes * 8;
    const bool cok = c0 + c8 < cols;
    Raw8<T> raw[kIter];
    const T *src = x + (r0 + lr) * ld + c0 + c8;
#pragma unroll
    for (int i = 0; i < kIter; i++) {
        raw[i].zero();
        if (cok && i * kStep + lr < left) {
            if constexpr (kSource == kExpertRows) {
                const int64_t r = row0 + i * kStep + lr;
                raw[i].load(x + (p.moe.k ? p.moe.order[r] / p.moe.k : r) * ld + c0 + c8);
            } else {
                raw[i].load(src + (int64_t)(i * kStep) * ld);
            }
        }
    }
    if (kCol) {
#pragma unroll
        for (int i = 0; i < kIter; i++)
            raw[i].store_shared(tile + (i * kStep + lr) * kCols + c8);
    }
    if (kRow) {
        const int64_t at = (r0 + lr) * cols + c0 + c8, step = kStep * cols;
        uint8_t *code = p.codes + at / 2;
        uint16_t *value = p.values + at;
#pragma unroll
        for (int i = 0; i < kIter; i++) {
            const int rl = i * kStep + lr;
            uint32_t m = raw[i].amax_bits();
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            uint32_t byte;
            const uint32_t q = raw[i].encode(m, byte);
            if ((lane & 3) == 0)
                reinterpret_cast<uint8_t *>(&s_sc[rl])[c8 >> 5] = (uint8_t)byte;
            if (cok && rl < left) {
                if (p.codes)
                    *reinterpret_cast<uint32_t *>(code) = q;
                if (p.values)
                    *reinterpret_cast<uint4 *>(value) = decode8_bf16(q, e8m0_scale(byte));
            }
            code += step / 2;
            value += step;
        }
    }
    if (kCol) {
        __syncthreads();   // the tile is in shared memory
        const int rb = warp & 3, c = ((warp >> 2) * 32 + lane) * kPer;
        typename S::Word v[32];
        S amax;
#pragma unroll
        for (int i = 0; i < 32; i++) {
            v[i] = *reinterpret_cast<const typename S::Word *>(tile + (rb * 32 + i) * kCols + c);
            amax.add(v[i]);
        }
        uint32_t byte[kPer], q[kPer][4];
#pragma unroll
        for (int j = 0; j < kPer; j++) {
            byte[j] = e8m0_of(amax.amax_bits(j));
            reinterpret_cast<uint8_t *>(&s_sct[c + j])[rb] = (uint8_t)byte[j];
            const float inv = byte[j] != 255u ? e8m0_inverse(byte[j]) : 0.0f;
#pragma unroll
            for (int g = 0; g < 4; g++) {
                float f[8];
#pragma unroll
                for (int e = 0; e < 8; e++)
                    f[e] = S::value(v[8 * g + e], j);
                q[j][g] = byte[j] != 255u ? e2m1_encode8_scaled(f, inv) : 0u;
            }
        }
#pragma unroll
        for (int j = 0; j < kPer; j++)
            s_q[(c + j) * 5 + rb] = make_uint4(q[j][0], q[j][1], q[j][2], q[j][3]);
        if (rb * 32 < cleft && c0 + c < cols) {
            if (p.values_t) {
#pragma unroll
                for (int g = 0; g < 4; g++) {
                    uint32_t h[kPer][4];
#pragma unroll
                    for (int j = 0; j < kPer; j++)
                        e2m1x8_to_h2x4(q[j][g], h[j]);
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const int rl = rb * 32 + 8 * g + e;
                        uint16_t *dst = p.values_t + (r0 + rl) * cols + c0 + c;
                        const float2 a = h2_to_f2(h[0][e / 2]), b = h2_to_f2(h[kPer - 1][e / 2]);
                        const uint32_t w = pack_bf2(__fmul_rn(e & 1 ? a.y : a.x, e8m0_scale(byte[0])),
                                                    __fmul_rn(e & 1 ? b.y : b.x, e8m0_scale(byte[kPer - 1])));
                        if (rl < left) {
                            if (kPer == 2)
                                *reinterpret_cast<uint32_t *>(dst) = w;
                            else
                                *dst = (uint16_t)w;
                        }
                    }
                }
            }
        }
    }
    __syncthreads();   // the scale bytes and the column codes are complete
    if (kCol && p.codes_t) {
        // 64 contiguous bytes a column, four threads
        uint8_t *dst = p.codes_t + c0 * (rows32 / 2) + r0 / 2;
#pragma unroll
        for (int i = tid; i < kCols * 4; i += kMqThreads) {
            const int c = i >> 2, rb = i & 3;
            if (rb * 32 < cleft && c0 + c < cols)
                *reinterpret_cast<uint4 *>(dst + c * (rows32 / 2) + rb * 16) = s_q[c * 5 + rb];
        }
    }
    // FP32: this tile's two blocks a row are one half of the scale tile's four
    const int half = kCols == 128 ? 0 : (int)(ct & 1);
    const bool alone = kCols != 128 && half == 0 && c0 + kCols >= cols;   // there is no other half
    if (kRow && p.scales && tid < kMqRows) {
        const uint32_t w = s_sc[(tid >> 2) + 32 * (tid & 3)];
        uint8_t *dst = p.scales + (rt * ktiles + c0 / 128) * 512 + tid * 4;
        if (kCols == 128) {
            *reinterpret_cast<uint32_t *>(dst) = w;
        } else {
            *reinterpret_cast<uint16_t *>(dst + half * 2) = (uint16_t)w;
            if (alone)
                *reinterpret_cast<uint16_t *>(dst + 2) = 0;
        }
    }
    if (kCol && p.scales_t && tid >= kMqThreads - kCols) {
        const int w = tid - (kMqThreads - kCols);
        uint32_t *dst = reinterpret_cast<uint32_t *>(p.scales_t + (c0 / 128 * rtiles + rt) * 512) + w / kGroups * 4 +
                        w % kGroups;
        dst[half * kGroups] = s_sct[w / kGroups + 32 * (w % kGroups)];
        if (alone)
            dst[kGroups] = 0u;
    }
}

// Rows of x to their places in the experts' order, each read once: a lane takes
// a block of 32 elements and writes its codes, 16 bytes, to every place that the
// row has (a token has one for each of its experts); four lanes put their scale
// bytes into a word and store it to four places at a time.  The rows behind an
// expert's last one are left as they are: a product's output rows depend on their
// own row only.
//
// What bounds it: bytes.  8192 tokens of 4096 with 8 places each: 36 us (6.1 TB/s,
// 89 % of the copy rate); with a block over four lanes, exchanged by shuffles for
// 16-byte stores, 38, with 4-byte stores 66 (issue).  Measured against it: one copy of
// the codes, whose rows the product gathers by TMA (four rows an instruction: 18
// cycles a row, three times what its MMAs take) or by cp.async (the product takes 21
// us longer, this kernel 12 us less).
constexpr int kMrChunk = 1024;

template <typename T>
__global__ void __launch_bounds__(256)
    mx_quantize_rows_kernel(const T *__restrict__ x, const int64_t ld, const int64_t rows, const int64_t cols,
                            uint8_t *__restrict__ codes, uint8_t *__restrict__ scales, const MoeRows m)
{
    const int lane = threadIdx.x & 31;
    const int64_t chunks = (cols + kMrChunk - 1) / kMrChunk, ktiles = (cols + 127) / 128;
    const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5), r = i / chunks;
    const int64_t c = i % chunks * kMrChunk + lane * 32;   // this lane's block
    pdl_wait();
    pdl_launch_dependents();
    if (r >= (m.k ? rows : min(rows, (int64_t)m.header[0])))   // grouped rows that there are
        return;
    Raw8<T> raw[4];
#pragma unroll
    for (int u = 0; u < 4; u++) {
        raw[u].zero();
        if (c < cols)
            raw[u].load_near(x + r * ld + c + u * 8);
    }
    const int n = m.k ? m.k : 1;
    // lane j: place j of the row
    int mine = -1;
    if (lane < n)
        mine = m.padded[m.k ? r * n + lane : m.order[r]];
    uint32_t a = 0, byte, q[4];
#pragma unroll
    for (int u = 0; u < 4; u++)
        a = max(a, raw[u].amax_bits());
#pragma unroll
    for (int u = 0; u < 4; u++)
        q[u] = raw[u].encode(a, byte);
    uint32_t word = byte << (lane & 3) * 8;
    word |= __shfl_xor_sync(0xffffffffu, word, 1);
    word |= __shfl_xor_sync(0xffffffffu, word, 2);
    const int64_t kt = c / 128;
    for (int j0 = 0; j0 < n; j0 += 4) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int at = j0 + j < n ? __shfl_sync(0xffffffffu, mine, j0 + j) : -1;
            if (at >= 0 && c < cols)
                *reinterpret_cast<uint4 *>(codes + ((int64_t)at * cols + c) / 2) = make_uint4(q[0], q[1], q[2], q[3]);
        }
        const int at = __shfl_sync(0xffffffffu, mine, (j0 + (lane & 3)) & 31);
        if (j0 + (lane & 3) < n && at >= 0 && kt < ktiles)
            *reinterpret_cast<uint32_t *>(scales + ((int64_t)(at >> 7) * ktiles + kt) * 512 + (at & 31) * 16 +
                                          (at & 127) / 32 * 4) = word;
    }
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

template <typename T, bool kRow, bool kCol, MqSource kSource = kMatrix>
cudaError_t run_quantize(const MxQuantArgs &a, cudaStream_t s, const MoeRows &moe = {}, int batch = 1)
{
    constexpr int kCols = MqShape<T>::kCols;
    MqParams p;
    p.moe = moe;
    p.rows = a.rows;
    p.cols = a.cols;
    p.ctiles = (a.cols + kCols - 1) / kCols;
    p.codes = a.codes;
    p.scales = a.scales;
    p.codes_t = a.codes_t;
    p.scales_t = a.scales_t;
    p.values = a.values;
    p.values_t = a.values_t;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((a.rows + kMqRows - 1) / kMqRows * p.ctiles), (unsigned)batch);
    cfg.blockDim = dim3(kMqThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.overlap ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, mx_quantize_kernel<T, kRow, kCol, kSource>, (const T *)a.x, a.ld, p);
}

template <typename T, MqSource kSource = kMatrix>
cudaError_t run_quantize_dirs(const MxQuantArgs &a, cudaStream_t s, const MoeRows &moe = {}, int batch = 1)
{
    const bool row = a.codes || a.values, col = a.codes_t || a.values_t;
    return row && col ? run_quantize<T, true, true, kSource>(a, s, moe, batch)
           : row      ? run_quantize<T, true, false, kSource>(a, s, moe, batch)
                      : run_quantize<T, false, true, kSource>(a, s, moe, batch);
}

template <typename T>
cudaError_t run_quantize_rows(const MxQuantArgs &a, const MoeRows &m, cudaStream_t s)
{
    const int64_t tasks = a.rows * ((a.cols + kMrChunk - 1) / kMrChunk), per = 8;
    return launch_dependent(mx_quantize_rows_kernel<T>, dim3((unsigned)((tasks + per - 1) / per)), 256, 0, s,
                            (const T *)a.x, a.ld, a.rows, a.cols, a.codes, a.scales, m);
}

unsigned grid_for(int64_t n, const DeviceInfo &dev)
{
    const int64_t want = (n + 255) / 256, most = (int64_t)dev.num_sms * 8;
    return (unsigned)(want < most ? want : most);
}

}  // namespace

cudaError_t launch_mx_quantize(const MxQuantArgs &a, cudaStream_t s)
{
    return a.x_fp32 ? run_quantize_dirs<float>(a, s) : run_quantize_dirs<__nv_bfloat16>(a, s);
}

cudaError_t launch_mx_quantize_rows(const MxQuantArgs &a, const MoeRows &m, cudaStream_t s)
{
    return a.x_fp32 ? run_quantize_rows<float>(a, m, s) : run_quantize_rows<__nv_bfloat16>(a, m, s);
}

cudaError_t launch_mx_quantize_groups(const MxQuantArgs &a, const MoeRows &m, cudaStream_t s)
{
    MxQuantArgs g = a;
    g.rows = m.max_blocks * kMqRows;
    return a.x_fp32 ? run_quantize_dirs<float, kExpertRows>(g, s, m) : run_quantize_dirs<__nv_bfloat16, kExpertRows>(g, s, m);
}

cudaError_t launch_mx_quantize_batch(const MxQuantArgs &a, int batch, cudaStream_t s)
{
    return a.x_fp32 ? run_quantize_dirs<float, kBatch>(a, s, {}, batch)
                    : run_quantize_dirs<__nv_bfloat16, kBatch>(a, s, {}, batch);
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
