// internal.h -- host-side declarations shared by the library's translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/nvfp4.h"

namespace nvfp4 {

struct DeviceInfo {
    int device = -1;
    int num_sms = 0;
    int cc_major = 0, cc_minor = 0;
    int decode_blocks_per_sm[2] = {0, 0};  // residency of the decode main kernel (MP 8, 16)
    int fused_quant_blocks = 0;            // grid of the fused dynamic quantiser (0: unavailable)
    bool stream_ok = false;                // the streaming decode kernel fits on this device
};

// Lets a kernel take `bytes` of dynamic shared memory (always the same number
// for a kernel): a call once per kernel and device.
template <auto kKernel>
inline cudaError_t allow_smem(size_t bytes, const DeviceInfo &dev)
{
    static std::atomic<uint64_t> done{0};
    const uint64_t bit = 1ull << dev.device;
    if (done.load(std::memory_order_relaxed) & bit)
        return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess)
        done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Cached per-device facts; nullptr (and *st set) when the device is unusable.
const DeviceInfo *device_info(nvfp4_status *st);

cudaError_t launch_quantize(const void *w, int64_t N, int64_t K, uint8_t *codes, uint8_t *scales,
                            float *tensor_scale, bool given, uint32_t *ctl, cudaStream_t s,
                            const DeviceInfo &dev);
cudaError_t launch_dequantize(const uint8_t *codes, const uint8_t *scales, const float *tensor_scale,
                              int64_t N, int64_t K, void *out, bool fp32, cudaStream_t s,
                              const DeviceInfo &dev);
cudaError_t launch_round_scales(const float *param, const float *tensor_scale, int64_t n,
                                uint8_t *out, uint32_t *ctl, cudaStream_t s, const DeviceInfo &dev);
cudaError_t launch_encode_debug(const float *x, int64_t n, int which, uint8_t *out, cudaStream_t s,
                                const DeviceInfo &dev);
cudaError_t launch_quotient_check(uint32_t lo, uint32_t hi, unsigned long long *mismatches,
                                  cudaStream_t s);

struct GemmArgs {
    const uint16_t *x;  // M x K bf16
    int64_t M, N, K, r;
    const uint8_t *codes, *scales;
    const float *tensor_scale;
    const uint16_t *lora_a, *lora_b;  // r x K, N x r (bf16) or null
    float lora_scale;
    const float *noise;  // K or null
    void *y;
    bool y_fp32;
    uint8_t *ws;
    size_t ws_bytes;
};

// Occupancy of the fused quantiser; called once per device by device_info().
void query_quantize_occupancy(DeviceInfo &dev);

// Occupancy of the decode kernels; called once per device by device_info().
void query_decode_occupancy(DeviceInfo &dev);

size_t decode_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t r, const DeviceInfo &dev);
cudaError_t launch_decode_gemm(const GemmArgs &a, cudaStream_t s, const DeviceInfo &dev);

// Streaming decode kernel (bulk copies through a shared-memory ring) for
// K % 256 == 0; other K use the register-streaming decode kernel above.
void query_stream_occupancy(DeviceInfo &dev);
bool stream_supported(int64_t N, int64_t K, int64_t r, const DeviceInfo &dev);
size_t stream_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t r, const DeviceInfo &dev);
cudaError_t launch_stream_gemm(const GemmArgs &a, cudaStream_t s, const DeviceInfo &dev);
// A list of projections with the same M, r and output type (list[0] gives
// them and the workspace) in launches of up to 64 projections: one
// activation-preparation launch and one streaming launch over all their
// units.  0 / cudaErrorInvalidConfiguration when a projection does not fit
// the streaming kernel.
size_t stream_list_workspace_bytes(const GemmArgs *list, int count, const DeviceInfo &dev);
cudaError_t launch_stream_list(const GemmArgs *list, int count, cudaStream_t s, const DeviceInfo &dev);

// Tensor-core (tcgen05) path for many tokens; smaller M uses the decode kernel.
constexpr int64_t kPrefillMinM = 64;
bool prefill_supported(int64_t M, int64_t N, int64_t K, int64_t r);
size_t prefill_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t r);
cudaError_t launch_prefill_gemm(const GemmArgs &a, cudaStream_t s, const DeviceInfo &dev);

// Input gradient dX = (dY deq(W) + s (dY B) A) diag(z) on the same tensor-core
// kernel (any M >= 1; N and K multiples of 64, r <= 64).  GemmArgs: x = dY
// (M x N), y = dX (M x K), noise = z (K) or null.
bool dgrad_supported(int64_t M, int64_t N, int64_t K, int64_t r);
size_t dgrad_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t r);
cudaError_t launch_dgrad_gemm(const GemmArgs &a, cudaStream_t s, const DeviceInfo &dev);

// LoRA factor gradients dA = s (dY B)^T X' (r x K) and dB = s dY^T (X' A^T)
// (N x r), FP32 (1 <= r <= 64; N and K multiples of 64; any M >= 1).
struct LoraGradArgs {
    const uint16_t *x, *dy;       // M x K, M x N bf16
    const float *noise;           // K or null
    int64_t M, N, K, r;
    const uint16_t *lora_a, *lora_b;
    float lora_scale;
    float *grad_a, *grad_b;       // r x K, N x r
    uint8_t *ws;
};
bool lora_grads_supported(int64_t M, int64_t N, int64_t K, int64_t r);
size_t lora_grads_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t r);
cudaError_t launch_lora_grads(const LoraGradArgs &a, cudaStream_t s, const DeviceInfo &dev);

// 2-D tiled tensor map (row-major, `row_bytes` between rows, box of
// box_inner x box_outer elements, zero fill outside) through the driver's
// encoder, looked up once.
cudaError_t encode_tensor_map_2d(CUtensorMap *map, CUtensorMapDataType dt, const void *base, uint64_t inner,
                                 uint64_t outer, uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer,
                                 CUtensorMapSwizzle swizzle);

// MXFP4 quantisation of a rows x cols matrix (csrc/mx_quant.cu); each output
// may be null, codes and scales of a direction go together.
struct MxQuantArgs {
    const void *x;
    bool x_fp32;
    int64_t rows, cols, ld;
    uint8_t *codes, *scales;      // blocks along the rows
    uint16_t *values;             // bf16, rows x cols
    uint8_t *codes_t, *scales_t;  // blocks along the columns, transposed
    uint16_t *values_t;           // bf16, rows x cols
    bool overlap;                 // its launch overlaps the end of the kernel before it
};
cudaError_t launch_mx_quantize(const MxQuantArgs &a, cudaStream_t s);
cudaError_t launch_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols, void *out,
                                 bool fp32, cudaStream_t s, const DeviceInfo &dev);
cudaError_t launch_tile_scales(const uint8_t *in, int64_t rows, int64_t nb, uint8_t *out, cudaStream_t s,
                               const DeviceInfo &dev);

// Block-scaled product of two 4-bit operands (csrc/gemm_w4a4.cu).
struct W4A4Args {
    bool nvfp4;                    // blocks of 16 with E4M3 scales (else 32, E8M0)
    const uint8_t *a_codes, *a_scales, *w_codes, *w_scales;
    const float *a_ts, *w_ts;      // tensor scales or null (1)
    const void *x;                 // tokens to be quantised on the way (M x K, ldx) instead of a_codes, or null
    bool x_fp32;
    int64_t ldx;
    int64_t M, N, K;
    void *y;
    bool y_fp32;
    uint32_t *ctl;
    bool after_quantise;           // launched right behind the quantiser of A on the same stream
};
cudaError_t launch_w4a4(const W4A4Args &a, cudaStream_t s, const DeviceInfo &dev);
// Whether launch_w4a4 takes unquantised tokens (MXFP4) of these sizes and type.
bool w4a4_takes_tokens(int64_t M, int64_t N, int64_t K, bool fp32, const DeviceInfo &dev);
// The variant for many tokens (csrc/gemm_w4a4_tile.cu).
cudaError_t launch_w4a4_tile(const W4A4Args &a, cudaStream_t s, const DeviceInfo &dev);
// Tiled scales (row_tiles x ktiles tiles of 512 bytes) as a tensor map whose
// box is box_rows x box_k tiles, in that order in shared memory.
cudaError_t encode_scale_map(CUtensorMap *map, const uint8_t *scales, uint64_t ktiles, uint64_t row_tiles,
                             uint32_t box_k, uint32_t box_rows);

// Distillation loss and gradient (csrc/distill.cu).
constexpr int kDistillMaxK = 1024;             // teacher entries per row
constexpr int64_t kDistillMaxSlice = 200 * 1024;  // bytes of a row one CTA (of up to 8) holds
constexpr float kLog2e = 1.4426950408889634f;  // exponents are base 2 and scaled by kLog2e * inv_tau, which is finite
struct DistillArgs {
    const void *z;
    bool z_fp32;
    int64_t T, V, ldz;
    const void *idx;
    bool idx64;
    const void *val;
    bool val_fp32;
    int k;
    float tau, inv_tau;
    bool tail;
    const float *weight;      // T or null
    const float *grad_loss;   // T, 1 or null
    bool grad_rows;           // grad_loss has T values
    float *loss;              // T or null
    void *dz;                 // T x V (leading dimension lddz) or null
    int64_t lddz;
    uint32_t *ctl;            // status words or null
    bool give_up;             // self-check: waits for copies give up at once
};
cudaError_t launch_distill(const DistillArgs &a, cudaStream_t s, const DeviceInfo &dev);

bool aligned16(const void *p);

// All host-side checks of nvfp4_w4a16_lora_gemm's arguments (pointers, enum
// values, shapes, alignment, device, workspace size); on NVFP4_OK *a and
// *dev describe the call.  Launches nothing.
nvfp4_status gemm_host_checks(const void *x_bf16, int64_t M, int64_t N, int64_t K, const uint8_t *codes,
                              const uint8_t *scales_e4m3, const float *tensor_scale, const void *lora_a_bf16,
                              const void *lora_b_bf16, int64_t r, float lora_scale, const float *noise_fp32,
                              void *y, nvfp4_dtype y_dtype, void *workspace, size_t ws_bytes, GemmArgs *a,
                              const DeviceInfo **dev);

// The kernels of one checked GEMM call (prefill, streaming or register-streaming decode).
cudaError_t launch_gemm(const GemmArgs &a, cudaStream_t s, const DeviceInfo &dev);

// Workspace of nvfp4_w4a16_lora_gemm for these sizes (0: unsupported).
inline size_t gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t r, const DeviceInfo &dev)
{
    if (prefill_supported(M, N, K, r))
        return prefill_workspace_bytes(M, N, K, r);
    if (stream_supported(N, K, r, dev))
        return stream_workspace_bytes(M, N, K, r, dev);
    return decode_workspace_bytes(M, N, K, r, dev);
}

}  // namespace nvfp4
