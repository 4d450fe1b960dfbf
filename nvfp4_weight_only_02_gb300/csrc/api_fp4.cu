// api_fp4.cu -- extern "C" entry points of the 4-bit activation operators
// (MXFP4 quantiser, W4A4 product and layer) and of the distillation loss:
// argument checks on the host, then launches on the caller's stream.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"

using namespace nvfp4;

namespace {

constexpr int64_t kMaxDim = 1LL << 30;

bool dtype_ok(nvfp4_dtype d) { return d == NVFP4_OUT_BF16 || d == NVFP4_OUT_FP32; }
bool format_ok(nvfp4_fp4_format f) { return f == NVFP4_FORMAT_MXFP4 || f == NVFP4_FORMAT_NVFP4; }
size_t align256(size_t v) { return (v + 255) / 256 * 256; }
int64_t up32(int64_t v) { return (v + 31) / 32 * 32; }

// rows x cols operand with blocks along cols
bool operand_ok(int64_t rows, int64_t cols)
{
    return rows >= 1 && rows <= kMaxDim && cols >= 32 && cols <= kMaxDim && cols % 32 == 0;
}

size_t scale_bytes(int64_t rows, int64_t cols, int64_t block)
{
    const int64_t nb = (cols + block - 1) / block;
    return (size_t)((rows + 127) / 128) * (size_t)((nb + 3) / 4) * 512;
}

size_t code_bytes(int64_t rows, int64_t cols) { return (size_t)rows * (size_t)(cols / 2); }

// tiles of 128 x 128 in one launch
bool tiles_ok(int64_t rows, int64_t cols)
{
    return ((rows + 127) / 128) * ((cols + 127) / 128) <= (1LL << 29);
}

nvfp4_status from_cuda(cudaError_t e) { return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }

bool opt_aligned(const void *p) { return !p || aligned16(p); }

// rows of x start on 16-byte boundaries
bool ld_aligned(int64_t ld, nvfp4_dtype d) { return ld % (d == NVFP4_OUT_FP32 ? 4 : 8) == 0; }

MxQuantArgs quant_args(const void *x, nvfp4_dtype dt, int64_t rows, int64_t cols, int64_t ld)
{
    MxQuantArgs a = {};
    a.x = x;
    a.x_fp32 = dt == NVFP4_OUT_FP32;
    a.rows = rows;
    a.cols = cols;
    a.ld = ld;
    return a;
}

// Checks of nvfp4_distill_topk's arguments; what its launch takes.
nvfp4_status distill_args(DistillArgs &a, const void *z, nvfp4_dtype z_dtype, int64_t T, int64_t V, int64_t ldz,
                          const void *index, int index_bytes, const void *teacher, nvfp4_dtype teacher_dtype,
                          int64_t k, float temperature, int rest_class, const float *row_weight,
                          const float *grad_loss, int64_t grad_loss_count, float *loss, void *dz, int64_t lddz,
                          void *workspace, size_t ws_bytes)
{
    const float inv_tau = 1.0f / temperature;
    if (!z || !index || !teacher || (!loss && !dz) || !dtype_ok(z_dtype) || !dtype_ok(teacher_dtype) ||
        (index_bytes != 4 && index_bytes != 8) || !(temperature > 0.0f) || !std::isfinite(temperature) ||
        !std::isfinite(inv_tau * kLog2e) || inv_tau == 0.0f || (grad_loss && !dz))
        return NVFP4_ERR_INVALID_ARG;
    const int64_t size = z_dtype == NVFP4_OUT_FP32 ? 4 : 2;
    // 8 CTAs hold a row, each slice rounded up to 16 bytes
    if (T < 1 || T > (1LL << 27) || V < 1 || V > kMaxDim || V * size > 8 * (kDistillMaxSlice - 16) || ldz < V || k < 1 ||
        k > kDistillMaxK || (dz && lddz < V) || ldz > (1LL << 40) || (dz && lddz > (1LL << 40)) ||
        (grad_loss && grad_loss_count != 1 && grad_loss_count != T))
        return NVFP4_ERR_SHAPE;
    if (!aligned16(z) || !aligned16(index) || !aligned16(teacher) || !opt_aligned(row_weight) ||
        !opt_aligned(grad_loss) || !opt_aligned(loss) || !opt_aligned(dz) || !opt_aligned(workspace))
        return NVFP4_ERR_ALIGNMENT;
    if (workspace && ws_bytes < kCtlBytes)
        return NVFP4_ERR_WORKSPACE;
    a = {};
    a.z = z;
    a.z_fp32 = z_dtype == NVFP4_OUT_FP32;
    a.T = T;
    a.V = V;
    a.ldz = ldz;
    a.idx = index;
    a.idx64 = index_bytes == 8;
    a.val = teacher;
    a.val_fp32 = teacher_dtype == NVFP4_OUT_FP32;
    a.k = (int)k;
    a.tau = temperature;
    a.inv_tau = inv_tau;
    a.tail = rest_class != 0;
    a.weight = row_weight;
    a.grad_loss = grad_loss;
    a.grad_rows = grad_loss_count == T && T > 1;
    a.loss = loss;
    a.dz = dz;
    a.lddz = lddz;
    a.ctl = (uint32_t *)workspace;
    return NVFP4_OK;
}

}  // namespace

#define NVFP4_TRY_DEVICE(devp)                  \
    nvfp4_status _st;                           \
    const DeviceInfo *devp = device_info(&_st); \
    if (!devp)                                  \
        return _st;

extern "C" {

size_t nvfp4_tiled_scale_bytes(int64_t rows, int64_t cols, nvfp4_fp4_format format)
{
    if (!format_ok(format) || rows < 1 || cols < 1 || rows > kMaxDim || cols > kMaxDim ||
        cols % (format == NVFP4_FORMAT_NVFP4 ? 16 : 32) != 0)
        return 0;
    return scale_bytes(rows, cols, format == NVFP4_FORMAT_NVFP4 ? 16 : 32);
}

nvfp4_status nvfp4_tile_scales(const uint8_t *scales, int64_t rows, int64_t cols, nvfp4_fp4_format format,
                               uint8_t *tiled, void *stream)
{
    if (!scales || !tiled || !format_ok(format))
        return NVFP4_ERR_INVALID_ARG;
    if (nvfp4_tiled_scale_bytes(rows, cols, format) == 0)
        return NVFP4_ERR_SHAPE;
    if (!aligned16(scales) || !aligned16(tiled))
        return NVFP4_ERR_ALIGNMENT;
    NVFP4_TRY_DEVICE(dev);
    return from_cuda(launch_tile_scales(scales, rows, cols / (format == NVFP4_FORMAT_NVFP4 ? 16 : 32), tiled,
                                        (cudaStream_t)stream, *dev));
}

nvfp4_status nvfp4_mx_quantize(const void *x, nvfp4_dtype x_dtype, int64_t rows, int64_t cols, int64_t ld,
                               uint8_t *codes, uint8_t *scales, void *values_bf16, uint8_t *codes_t,
                               uint8_t *scales_t, void *values_t_bf16, void *stream)
{
    // sizes first: an empty tensor has a null pointer too
    if (!operand_ok(rows, cols) || ld < cols || ld > kMaxDim || !tiles_ok(rows, cols))
        return NVFP4_ERR_SHAPE;
    if (!x || !dtype_ok(x_dtype) || (!codes) != (!scales) || (!codes_t) != (!scales_t) ||
        (!codes && !values_bf16 && !codes_t && !values_t_bf16))
        return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(x) || !ld_aligned(ld, x_dtype) || !opt_aligned(codes) || !opt_aligned(scales) ||
        !opt_aligned(values_bf16) || !opt_aligned(codes_t) || !opt_aligned(scales_t) || !opt_aligned(values_t_bf16))
        return NVFP4_ERR_ALIGNMENT;
    NVFP4_TRY_DEVICE(dev);
    (void)dev;
    MxQuantArgs a = quant_args(x, x_dtype, rows, cols, ld);
    a.codes = codes;
    a.scales = scales;
    a.values = (uint16_t *)values_bf16;
    a.codes_t = codes_t;
    a.scales_t = scales_t;
    a.values_t = (uint16_t *)values_t_bf16;
    return from_cuda(launch_mx_quantize(a, (cudaStream_t)stream));
}

nvfp4_status nvfp4_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols, void *out,
                                 nvfp4_dtype out_dtype, void *stream)
{
    if (!codes || !scales || !out || !dtype_ok(out_dtype))
        return NVFP4_ERR_INVALID_ARG;
    if (!operand_ok(rows, cols))
        return NVFP4_ERR_SHAPE;
    if (!aligned16(codes) || !aligned16(scales) || !aligned16(out))
        return NVFP4_ERR_ALIGNMENT;
    NVFP4_TRY_DEVICE(dev);
    return from_cuda(launch_mx_dequantize(codes, scales, rows, cols, out, out_dtype == NVFP4_OUT_FP32,
                                          (cudaStream_t)stream, *dev));
}

size_t nvfp4_w4a4_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    if (!operand_ok(M, K) || !operand_ok(N, K) || !tiles_ok(M, N))
        return 0;
    return align256(kWsHeaderBytes);   // scratch always starts behind the counters, which other calls count on
}

nvfp4_status nvfp4_w4a4_gemm(nvfp4_fp4_format format, const uint8_t *a_codes, const uint8_t *a_scales,
                             const float *a_tensor_scale, const uint8_t *w_codes, const uint8_t *w_scales,
                             const float *w_tensor_scale, int64_t M, int64_t N, int64_t K, void *y,
                             nvfp4_dtype y_dtype, void *workspace, size_t ws_bytes, void *stream)
{
    if (!a_codes || !a_scales || !w_codes || !w_scales || !y || !workspace || !dtype_ok(y_dtype) ||
        !format_ok(format))
        return NVFP4_ERR_INVALID_ARG;
    const size_t need = nvfp4_w4a4_workspace_bytes(M, N, K);
    if (need == 0)
        return NVFP4_ERR_SHAPE;
    if (!aligned16(a_codes) || !aligned16(a_scales) || !opt_aligned(a_tensor_scale) || !aligned16(w_codes) ||
        !aligned16(w_scales) || !opt_aligned(w_tensor_scale) || !aligned16(y) || !aligned16(workspace))
        return NVFP4_ERR_ALIGNMENT;
    if (ws_bytes < need)
        return NVFP4_ERR_WORKSPACE;
    NVFP4_TRY_DEVICE(dev);
    W4A4Args a = {};
    a.nvfp4 = format == NVFP4_FORMAT_NVFP4;
    a.a_codes = a_codes;
    a.a_scales = a_scales;
    a.w_codes = w_codes;
    a.w_scales = w_scales;
    a.a_ts = a_tensor_scale;
    a.w_ts = w_tensor_scale;
    a.M = M;
    a.N = N;
    a.K = K;
    a.y = y;
    a.y_fp32 = y_dtype == NVFP4_OUT_FP32;
    a.ctl = (uint32_t *)workspace;
    return from_cuda(launch_w4a4(a, (cudaStream_t)stream, *dev));
}

size_t nvfp4_mx_linear_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    if (nvfp4_w4a4_workspace_bytes(M, N, K) == 0 || !tiles_ok(M, K))
        return 0;
    return nvfp4_w4a4_workspace_bytes(M, N, K) + align256(code_bytes(M, K)) + align256(scale_bytes(M, K, 32));
}

nvfp4_status nvfp4_mx_linear(const void *x, nvfp4_dtype x_dtype, int64_t ldx, int64_t M, int64_t N, int64_t K,
                             const uint8_t *w_codes, const uint8_t *w_scales, void *y, nvfp4_dtype y_dtype,
                             void *workspace, size_t ws_bytes, void *stream)
{
    if (!x || !w_codes || !w_scales || !y || !workspace || !dtype_ok(x_dtype) || !dtype_ok(y_dtype))
        return NVFP4_ERR_INVALID_ARG;
    const size_t need = nvfp4_mx_linear_workspace_bytes(M, N, K);
    if (need == 0 || ldx < K || ldx > kMaxDim)
        return NVFP4_ERR_SHAPE;
    if (!aligned16(x) || !ld_aligned(ldx, x_dtype) || !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(y) ||
        !aligned16(workspace))
        return NVFP4_ERR_ALIGNMENT;
    if (ws_bytes < need)
        return NVFP4_ERR_WORKSPACE;
    NVFP4_TRY_DEVICE(dev);
    W4A4Args a = {};
    if (w4a4_takes_tokens(M, N, K, x_dtype == NVFP4_OUT_FP32, *dev)) {
        a.x = x;
        a.x_fp32 = x_dtype == NVFP4_OUT_FP32;
        a.ldx = ldx;
    } else {
        MxQuantArgs q = quant_args(x, x_dtype, M, K, ldx);
        q.codes = (uint8_t *)workspace + nvfp4_w4a4_workspace_bytes(M, N, K);
        q.scales = q.codes + align256(code_bytes(M, K));
        // behind a product that streams weights the quantiser may start early (16 tokens: 10.9 us a call and
        // 12.4 without, N = 18944, K = 3584); the tile kernel then starts late (1024 tokens: 34.9 and 31.6)
        q.overlap = M <= 64;
        const cudaError_t e = launch_mx_quantize(q, (cudaStream_t)stream);
        if (e != cudaSuccess)
            return NVFP4_ERR_CUDA;
        a.a_codes = q.codes;
        a.a_scales = q.scales;
        a.after_quantise = true;
    }
    a.w_codes = w_codes;
    a.w_scales = w_scales;
    a.M = M;
    a.N = N;
    a.K = K;
    a.y = y;
    a.y_fp32 = y_dtype == NVFP4_OUT_FP32;
    a.ctl = (uint32_t *)workspace;
    return from_cuda(launch_w4a4(a, (cudaStream_t)stream, *dev));
}

size_t nvfp4_mx_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    // dX = Q(dY) Q_c(W): M x K over N;  dW = Q_c(dY)^T Q_c(X): N x K over M
    if (M < 1 || M > kMaxDim - 31 || nvfp4_w4a4_workspace_bytes(M, K, N) == 0 ||
        nvfp4_w4a4_workspace_bytes(N, K, up32(M)) == 0 || K % 32 != 0 || !tiles_ok(M, N))
        return 0;
    return nvfp4_w4a4_workspace_bytes(M, N, K) + align256(code_bytes(M, N)) + align256(scale_bytes(M, N, 32)) +
           align256(code_bytes(N, up32(M))) + align256(scale_bytes(N, up32(M), 32));
}

nvfp4_status nvfp4_mx_linear_backward(const void *dy, nvfp4_dtype dy_dtype, int64_t lddy, int64_t M, int64_t N,
                                      int64_t K, const uint8_t *x_codes_t, const uint8_t *x_scales_t,
                                      const uint8_t *w_codes_t, const uint8_t *w_scales_t, void *dx,
                                      nvfp4_dtype dx_dtype, void *dw, nvfp4_dtype dw_dtype, void *workspace,
                                      size_t ws_bytes, void *stream)
{
    if (!dy || !workspace || !dtype_ok(dy_dtype) || !dtype_ok(dx_dtype) || !dtype_ok(dw_dtype) || (!dx && !dw) ||
        (dx && (!w_codes_t || !w_scales_t)) || (dw && (!x_codes_t || !x_scales_t)))
        return NVFP4_ERR_INVALID_ARG;
    const size_t need = nvfp4_mx_linear_backward_workspace_bytes(M, N, K);
    if (need == 0 || lddy < N || lddy > kMaxDim)
        return NVFP4_ERR_SHAPE;
    if (!aligned16(dy) || !ld_aligned(lddy, dy_dtype) || !opt_aligned(x_codes_t) || !opt_aligned(x_scales_t) ||
        !opt_aligned(w_codes_t) || !opt_aligned(w_scales_t) || !opt_aligned(dx) || !opt_aligned(dw) ||
        !aligned16(workspace))
        return NVFP4_ERR_ALIGNMENT;
    if (ws_bytes < need)
        return NVFP4_ERR_WORKSPACE;
    NVFP4_TRY_DEVICE(dev);
    cudaStream_t s = (cudaStream_t)stream;
    uint8_t *at = (uint8_t *)workspace + nvfp4_w4a4_workspace_bytes(M, N, K);
    MxQuantArgs q = quant_args(dy, dy_dtype, M, N, lddy);
    uint8_t *codes = at, *scales = codes + align256(code_bytes(M, N));
    uint8_t *codes_t = scales + align256(scale_bytes(M, N, 32));
    uint8_t *scales_t = codes_t + align256(code_bytes(N, up32(M)));
    if (dx) {
        q.codes = codes;
        q.scales = scales;
    }
    if (dw) {
        q.codes_t = codes_t;
        q.scales_t = scales_t;
    }
    cudaError_t e = launch_mx_quantize(q, s);
    W4A4Args a = {};
    a.ctl = (uint32_t *)workspace;
    a.after_quantise = true;
    if (e == cudaSuccess && dx) {
        a.a_codes = codes;
        a.a_scales = scales;
        a.w_codes = w_codes_t;
        a.w_scales = w_scales_t;
        a.M = M;
        a.N = K;
        a.K = N;
        a.y = dx;
        a.y_fp32 = dx_dtype == NVFP4_OUT_FP32;
        e = launch_w4a4(a, s, *dev);
        a.after_quantise = false;
    }
    if (e == cudaSuccess && dw) {
        a.a_codes = codes_t;
        a.a_scales = scales_t;
        a.w_codes = x_codes_t;
        a.w_scales = x_scales_t;
        a.M = N;
        a.N = K;
        a.K = up32(M);
        a.y = dw;
        a.y_fp32 = dw_dtype == NVFP4_OUT_FP32;
        e = launch_w4a4(a, s, *dev);
    }
    return from_cuda(e);
}

nvfp4_status nvfp4_distill_topk(const void *z, nvfp4_dtype z_dtype, int64_t T, int64_t V, int64_t ldz,
                                const void *index, int index_bytes, const void *teacher, nvfp4_dtype teacher_dtype,
                                int64_t k, float temperature, int rest_class, const float *row_weight,
                                const float *grad_loss, int64_t grad_loss_count, float *loss, void *dz,
                                int64_t lddz, void *workspace, size_t ws_bytes, void *stream)
{
    DistillArgs a;
    const nvfp4_status st = distill_args(a, z, z_dtype, T, V, ldz, index, index_bytes, teacher, teacher_dtype, k,
                                         temperature, rest_class, row_weight, grad_loss, grad_loss_count, loss, dz,
                                         lddz, workspace, ws_bytes);
    if (st != NVFP4_OK)
        return st;
    NVFP4_TRY_DEVICE(dev);
    return from_cuda(launch_distill(a, (cudaStream_t)stream, *dev));
}

nvfp4_status nvfp4_distill_wait_selftest(const void *z, nvfp4_dtype z_dtype, int64_t T, int64_t V,
                                         const int32_t *index, const float *teacher, int64_t k, int rest_class,
                                         const float *row_weight, float *loss, void *dz, void *workspace,
                                         size_t ws_bytes, void *stream)
{
    DistillArgs a;
    const nvfp4_status st = distill_args(a, z, z_dtype, T, V, V, index, 4, teacher, NVFP4_OUT_FP32, k, 1.0f, rest_class,
                                         row_weight, nullptr, 0, loss, dz, V, workspace, ws_bytes);
    if (st != NVFP4_OK)
        return st;
    a.give_up = true;
    NVFP4_TRY_DEVICE(dev);
    return from_cuda(launch_distill(a, (cudaStream_t)stream, *dev));
}

}  // extern "C"
