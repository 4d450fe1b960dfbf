// api_int8.cu -- extern "C" entry points of the 8-bit integer operators
// (quantiser of rows, product, layer): argument checks on the host, then
// launches on the caller's stream.
#include "common.cuh"
#include "internal.h"

using namespace nvfp4;

namespace {

// Sums are 2^31 in magnitude at most, and with codes of one sign within 2e-3 of the exact ones (gemm_int8.cu).
constexpr int64_t kMaxK = 131072;
constexpr int64_t kMaxDim = 1LL << 30;

bool dtype_ok(nvfp4_dtype d) { return d == NVFP4_OUT_BF16 || d == NVFP4_OUT_FP32; }
size_t align256(size_t v) { return (v + 255) / 256 * 256; }
bool ld_aligned(int64_t ld, nvfp4_dtype d) { return ld % (d == NVFP4_OUT_FP32 ? 4 : 8) == 0; }
nvfp4_status from_cuda(cudaError_t e) { return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }

bool matrix_ok(int64_t rows, int64_t K)
{
    return rows >= 1 && rows <= kMaxDim && K >= 16 && K <= kMaxK && K % 16 == 0 && rows * K <= (1LL << 42);
}

Int8GemmArgs gemm_args(const void *x, const float *x_scale, const int8_t *w, const float *w_scale, int64_t M, int64_t N,
                       int64_t K, void *y, nvfp4_dtype dt, void *ws)
{
    Int8GemmArgs a = {};
    a.x = x;
    a.x_scale = x_scale;
    a.w = w;
    a.w_scale = w_scale;
    a.M = M;
    a.N = N;
    a.K = K;
    a.y = y;
    a.y_fp32 = dt == NVFP4_OUT_FP32;
    a.ctl = (uint32_t *)ws;
    return a;
}

}  // namespace

#define NVFP4_TRY_DEVICE(devp)                  \
    nvfp4_status _st;                           \
    const DeviceInfo *devp = device_info(&_st); \
    if (!devp)                                  \
        return _st;

extern "C" {

nvfp4_status nvfp4_int8_quantize(const void *x, nvfp4_dtype x_dtype, int64_t rows, int64_t cols, int64_t ld,
                                 int8_t *codes, float *scales, void *stream)
{
    if (!matrix_ok(rows, cols) || ld < cols || ld > kMaxDim)
        return NVFP4_ERR_SHAPE;
    if (!x || !codes || !scales || !dtype_ok(x_dtype))
        return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(x) || !ld_aligned(ld, x_dtype) || !aligned16(codes) || !aligned16(scales))
        return NVFP4_ERR_ALIGNMENT;
    NVFP4_TRY_DEVICE(dev);
    (void)dev;
    Int8QuantArgs q = {x, x_dtype == NVFP4_OUT_FP32, rows, cols, ld, codes, false, scales};
    return from_cuda(launch_int8_quantize(q, (cudaStream_t)stream));
}

size_t nvfp4_int8_linear_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    // tiles of a launch
    if (!matrix_ok(M, K) || !matrix_ok(N, K) || ((M + 127) / 128) * ((N + 127) / 128) > (1LL << 28))
        return 0;
    return align256(kWsHeaderBytes) + align256((size_t)M * K * 2) + align256((size_t)M * 4);
}

nvfp4_status nvfp4_int8_gemm(const int8_t *a_codes, const float *a_scales, const int8_t *w_codes, const float *w_scales,
                             int64_t M, int64_t N, int64_t K, void *y, nvfp4_dtype y_dtype, void *workspace,
                             size_t ws_bytes, void *stream)
{
    const size_t need = nvfp4_int8_linear_workspace_bytes(M, N, K);
    if (need == 0)
        return NVFP4_ERR_SHAPE;
    if (!a_codes || !a_scales || !w_codes || !w_scales || !y || !workspace || !dtype_ok(y_dtype))
        return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(a_codes) || !aligned16(a_scales) || !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(y) ||
        !aligned16(workspace))
        return NVFP4_ERR_ALIGNMENT;
    if (ws_bytes < need)
        return NVFP4_ERR_WORKSPACE;
    NVFP4_TRY_DEVICE(dev);
    uint8_t *x = (uint8_t *)workspace + align256(kWsHeaderBytes);
    cudaError_t e = launch_int8_widen(a_codes, M * K, x, (cudaStream_t)stream);
    if (e == cudaSuccess)
        e = launch_int8_gemm(gemm_args(x, a_scales, w_codes, w_scales, M, N, K, y, y_dtype, workspace),
                             (cudaStream_t)stream, *dev);
    return from_cuda(e);
}

nvfp4_status nvfp4_int8_linear(const void *x, nvfp4_dtype x_dtype, int64_t ldx, int64_t M, int64_t N, int64_t K,
                               const int8_t *w_codes, const float *w_scales, void *y, nvfp4_dtype y_dtype,
                               void *workspace, size_t ws_bytes, void *stream)
{
    const size_t need = nvfp4_int8_linear_workspace_bytes(M, N, K);
    if (need == 0 || ldx < K || ldx > kMaxDim)
        return NVFP4_ERR_SHAPE;
    if (!x || !w_codes || !w_scales || !y || !workspace || !dtype_ok(x_dtype) || !dtype_ok(y_dtype))
        return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(x) || !ld_aligned(ldx, x_dtype) || !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(y) ||
        !aligned16(workspace))
        return NVFP4_ERR_ALIGNMENT;
    if (ws_bytes < need)
        return NVFP4_ERR_WORKSPACE;
    NVFP4_TRY_DEVICE(dev);
    if (int8_takes_tokens(M, N, K, *dev)) {
        Int8GemmArgs a = gemm_args(x, nullptr, w_codes, w_scales, M, N, K, y, y_dtype, workspace);
        a.raw = true;
        a.raw_fp32 = x_dtype == NVFP4_OUT_FP32;
        a.ldx = ldx;
        return from_cuda(launch_int8_gemm(a, (cudaStream_t)stream, *dev));
    }
    uint8_t *q = (uint8_t *)workspace + align256(kWsHeaderBytes);
    float *scale = (float *)(q + align256((size_t)M * K * 2));
    const Int8QuantArgs qa = {x, x_dtype == NVFP4_OUT_FP32, M, K, ldx, q, true, scale};
    cudaError_t e = launch_int8_quantize(qa, (cudaStream_t)stream);
    if (e == cudaSuccess)
        e = launch_int8_gemm(gemm_args(q, scale, w_codes, w_scales, M, N, K, y, y_dtype, workspace), (cudaStream_t)stream,
                             *dev);
    return from_cuda(e);
}

}  // extern "C"
