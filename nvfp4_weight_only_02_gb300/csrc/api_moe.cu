// api_moe.cu -- extern "C" entry points of the mixture-of-experts operators
// (routing, grouping, the layer grouped by expert and its backward pass, the
// weighted sum back): argument checks on the host, then launches on the
// caller's stream.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "moe_plan.h"

using namespace nvfp4;

namespace {

constexpr int64_t kMaxDim = 1LL << 24;

bool dtype_ok(nvfp4_dtype d) { return d == NVFP4_OUT_BF16 || d == NVFP4_OUT_FP32; }
size_t align256(size_t v) { return (v + 255) / 256 * 256; }
bool opt_aligned(const void *p) { return !p || aligned16(p); }
bool ld_aligned(int64_t ld, nvfp4_dtype d) { return ld % (d == NVFP4_OUT_FP32 ? 4 : 8) == 0; }
nvfp4_status from_cuda(cudaError_t e) { return e == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA; }

size_t scale_bytes(int64_t rows, int64_t cols)
{
    return (size_t)((rows + 127) / 128) * (size_t)((cols + 127) / 128) * 512;
}
size_t code_bytes(int64_t rows, int64_t cols) { return (size_t)rows * (size_t)(cols / 2); }

// A contraction axis, and with it the blocks.
bool contraction_ok(int64_t K) { return K >= 32 && K <= kMaxDim && K % 32 == 0; }

bool layer_ok(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K)
{
    if (!moe_sizes_ok(T, k, E) || N < 1 || N > kMaxDim || !contraction_ok(K))
        return false;
    const MoeLayout l(T, k, (int)E);
    // tiles of a launch, of the product's and of the quantiser's
    return l.max_tiles * ((N + 127) / 128) <= (1LL << 27) && l.max_blocks * ((K + 63) / 64) <= (1LL << 30) &&
           E * ((N + 127) / 128) <= (1LL << 27);
}

// What every call that takes a plan checks of it.
nvfp4_status plan_ok(const void *plan, size_t plan_bytes, int64_t T, int64_t k, int64_t E)
{
    if (!moe_sizes_ok(T, k, E))
        return NVFP4_ERR_SHAPE;
    if (!plan)
        return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(plan))
        return NVFP4_ERR_ALIGNMENT;
    return plan_bytes < nvfp4_moe_plan_bytes(T, k, E) ? NVFP4_ERR_WORKSPACE : NVFP4_OK;
}

MoeRows rows_of(const MoeLayout &l, const void *plan, int64_t k, bool sorted)
{
    const int32_t *w = (const int32_t *)plan;
    MoeRows m = {};
    m.header = w;
    m.order = w + l.order;
    m.padded = w + l.padded;
    m.blocks = (const int4 *)(w + l.blocks);
    m.max_blocks = l.max_blocks;
    m.k = sorted ? 0 : (int)k;
    return m;
}

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

MoeGemmArgs gemm_args(const MoeLayout &l, const void *plan, int64_t N, int64_t K, void *y, nvfp4_dtype dt, void *ws)
{
    const int32_t *w = (const int32_t *)plan;
    MoeGemmArgs a = {};
    a.padded_rows = l.padded_rows();
    a.N = N;
    a.K = K;
    a.E = l.experts;
    a.header = w;
    a.tiles = (const int4 *)(w + l.tiles);
    a.max_tiles = l.max_tiles;
    a.tile_rows = l.tile_rows;
    a.y = y;
    a.y_fp32 = dt == NVFP4_OUT_FP32;
    a.ctl = (uint32_t *)ws;
    return a;
}

bool scoring_ok(nvfp4_moe_scoring s) { return s == NVFP4_MOE_SOFTMAX || s == NVFP4_MOE_SIGMOID; }

}  // namespace

#define NVFP4_TRY_DEVICE(devp)                  \
    nvfp4_status _st;                           \
    const DeviceInfo *devp = device_info(&_st); \
    if (!devp)                                  \
        return _st;

extern "C" {

size_t nvfp4_moe_plan_bytes(int64_t T, int64_t k, int64_t E)
{
    return moe_sizes_ok(T, k, E) ? (size_t)MoeLayout(T, k, (int)E).total * 4 : 0;
}

size_t nvfp4_moe_plan_part(int64_t T, int64_t k, int64_t E, nvfp4_moe_part part)
{
    if (!moe_sizes_ok(T, k, E))
        return 0;
    const MoeLayout l(T, k, (int)E);
    switch (part) {
    case NVFP4_MOE_OFFSETS:
        return (size_t)l.offsets * 4;
    case NVFP4_MOE_ORDER:
        return (size_t)l.order * 4;
    case NVFP4_MOE_POSITION:
        return (size_t)l.position * 4;
    }
    return 0;
}

int64_t nvfp4_moe_padded_rows(int64_t T, int64_t k, int64_t E)
{
    return moe_sizes_ok(T, k, E) ? MoeLayout(T, k, (int)E).padded_rows() : 0;
}

nvfp4_status nvfp4_moe_route(const void *z, nvfp4_dtype z_dtype, int64_t T, int64_t E, int64_t ldz, int64_t k,
                             nvfp4_moe_scoring scoring, int renormalise, const float *bias, float scale, float *weights,
                             int32_t *experts, void *plan, size_t plan_bytes, void *stream)
{
    if (!moe_sizes_ok(T, k, E) || k > E || ldz < E || ldz > (1LL << 40))
        return NVFP4_ERR_SHAPE;
    if (!z || !weights || !experts || !dtype_ok(z_dtype) || !scoring_ok(scoring) || !std::isfinite(scale))
        return NVFP4_ERR_INVALID_ARG;
    const nvfp4_status ps = plan_ok(plan, plan_bytes, T, k, E);
    if (ps != NVFP4_OK)
        return ps;
    if (!aligned16(z) || !opt_aligned(bias) || !aligned16(weights) || !aligned16(experts))
        return NVFP4_ERR_ALIGNMENT;
    NVFP4_TRY_DEVICE(dev);
    MoeRouteArgs a = {};
    a.z = z;
    a.z_fp32 = z_dtype == NVFP4_OUT_FP32;
    a.T = T;
    a.ldz = ldz;
    a.E = (int)E;
    a.k = (int)k;
    a.sigmoid = scoring == NVFP4_MOE_SIGMOID;
    a.renorm = renormalise != 0;
    a.bias = bias;
    a.scale = scale;
    a.weights = weights;
    a.experts = experts;
    a.plan = (int32_t *)plan;
    return from_cuda(launch_moe_route(a, (cudaStream_t)stream, *dev));
}

nvfp4_status nvfp4_moe_route_backward(const float *dweights, const void *z, nvfp4_dtype z_dtype, int64_t T, int64_t E,
                                      int64_t ldz, int64_t k, nvfp4_moe_scoring scoring, int renormalise, float scale,
                                      const float *weights, const int32_t *experts, void *dz, int64_t lddz, void *stream)
{
    if (!moe_sizes_ok(T, k, E) || k > E || ldz < E || lddz < E || ldz > (1LL << 40) || lddz > (1LL << 40))
        return NVFP4_ERR_SHAPE;
    if (!dweights || !z || !weights || !experts || !dz || !dtype_ok(z_dtype) || !scoring_ok(scoring) ||
        !std::isfinite(scale))
        return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(dweights) || !aligned16(z) || !aligned16(weights) || !aligned16(experts) || !aligned16(dz))
        return NVFP4_ERR_ALIGNMENT;
    NVFP4_TRY_DEVICE(dev);
    (void)dev;
    MoeRouteArgs a = {};
    a.z = z;
    a.z_fp32 = z_dtype == NVFP4_OUT_FP32;
    a.T = T;
    a.ldz = ldz;
    a.E = (int)E;
    a.k = (int)k;
    a.sigmoid = scoring == NVFP4_MOE_SIGMOID;
    a.renorm = renormalise != 0;
    a.scale = scale;
    a.weights = const_cast<float *>(weights);
    a.experts = const_cast<int32_t *>(experts);
    return from_cuda(launch_moe_route_backward(a, dweights, dz, lddz, (cudaStream_t)stream));
}

nvfp4_status nvfp4_moe_plan(const int32_t *experts, int64_t T, int64_t k, int64_t E, void *plan, size_t plan_bytes,
                            void *workspace, size_t ws_bytes, void *stream)
{
    const nvfp4_status ps = plan_ok(plan, plan_bytes, T, k, E);
    if (ps != NVFP4_OK)
        return ps;
    if (!experts)
        return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(experts) || !opt_aligned(workspace))
        return NVFP4_ERR_ALIGNMENT;
    if (workspace && ws_bytes < kCtlBytes)
        return NVFP4_ERR_WORKSPACE;
    NVFP4_TRY_DEVICE(dev);
    MoeRouteArgs a = {};
    a.T = T;
    a.E = (int)E;
    a.k = (int)k;
    a.experts = const_cast<int32_t *>(experts);
    a.plan = (int32_t *)plan;
    a.ctl = (uint32_t *)workspace;
    return from_cuda(launch_moe_route(a, (cudaStream_t)stream, *dev));
}

nvfp4_status nvfp4_moe_combine(const void *y, nvfp4_dtype y_dtype, const float *weights, const void *plan,
                               size_t plan_bytes, int64_t T, int64_t k, int64_t E, int64_t N, const void *base, void *out,
                               nvfp4_dtype out_dtype, void *stream)
{
    const nvfp4_status ps = plan_ok(plan, plan_bytes, T, k, E);
    if (ps != NVFP4_OK)
        return ps;
    if (N < 1 || N > kMaxDim || T * N > (1LL << 38))
        return NVFP4_ERR_SHAPE;
    if (!y || !out || !dtype_ok(y_dtype) || !dtype_ok(out_dtype))
        return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(y) || !opt_aligned(weights) || !opt_aligned(base) || !aligned16(out))
        return NVFP4_ERR_ALIGNMENT;
    NVFP4_TRY_DEVICE(dev);
    (void)dev;
    MoeCombineArgs a = {};
    a.y = y;
    a.y_fp32 = y_dtype == NVFP4_OUT_FP32;
    a.weights = weights;
    a.position = (const int32_t *)plan + MoeLayout(T, k, (int)E).position;
    a.T = T;
    a.N = N;
    a.k = (int)k;
    a.base = base;
    a.out = out;
    a.out_fp32 = out_dtype == NVFP4_OUT_FP32;
    return from_cuda(launch_moe_combine(a, (cudaStream_t)stream));
}

nvfp4_status nvfp4_moe_combine_backward(const void *dout, const void *y, nvfp4_dtype dtype, const float *weights,
                                        const void *plan, size_t plan_bytes, int64_t T, int64_t k, int64_t E, int64_t N,
                                        void *dy, float *dweights, void *stream)
{
    const nvfp4_status ps = plan_ok(plan, plan_bytes, T, k, E);
    if (ps != NVFP4_OK)
        return ps;
    if (N < 1 || N > kMaxDim || T * N > (1LL << 38))
        return NVFP4_ERR_SHAPE;
    if (!dout || !weights || (!dy && !dweights) || (dweights && !y) || !dtype_ok(dtype))
        return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(dout) || !opt_aligned(y) || !aligned16(weights) || !opt_aligned(dy) || !opt_aligned(dweights))
        return NVFP4_ERR_ALIGNMENT;
    NVFP4_TRY_DEVICE(dev);
    (void)dev;
    MoeCombineArgs a = {};
    a.y = y;
    a.y_fp32 = dtype == NVFP4_OUT_FP32;
    a.weights = weights;
    a.position = (const int32_t *)plan + MoeLayout(T, k, (int)E).position;
    a.T = T;
    a.N = N;
    a.k = (int)k;
    a.dout = dout;
    a.dy = dy;
    a.dw = dweights;
    return from_cuda(launch_moe_combine_backward(a, (cudaStream_t)stream));
}

nvfp4_status nvfp4_mx_quantize_experts(const void *w, nvfp4_dtype w_dtype, int64_t E, int64_t N, int64_t K,
                                       uint8_t *codes, uint8_t *scales, uint8_t *codes_t, uint8_t *scales_t,
                                       void *stream)
{
    if (E < 1 || E > kMoeMaxExperts || N < 1 || N > kMaxDim || !contraction_ok(K) ||
        ((N + 127) / 128) * ((K + 63) / 64) > (1LL << 30))
        return NVFP4_ERR_SHAPE;
    if (!w || !dtype_ok(w_dtype) || (!codes) != (!scales) || (!codes_t) != (!scales_t) || (!codes && !codes_t))
        return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(w) || !opt_aligned(codes) || !opt_aligned(scales) || !opt_aligned(codes_t) || !opt_aligned(scales_t))
        return NVFP4_ERR_ALIGNMENT;
    NVFP4_TRY_DEVICE(dev);
    (void)dev;
    MxQuantArgs a = quant_args(w, w_dtype, N, K, K);
    a.codes = codes;
    a.scales = scales;
    a.codes_t = codes_t;
    a.scales_t = scales_t;
    return from_cuda(launch_mx_quantize_batch(a, (int)E, (cudaStream_t)stream));
}

nvfp4_status nvfp4_moe_quantize(const void *x, nvfp4_dtype x_dtype, int64_t ldx, int sorted_rows, const void *plan,
                                size_t plan_bytes, int64_t T, int64_t k, int64_t E, int64_t K, uint8_t *codes,
                                uint8_t *scales, uint8_t *codes_t, uint8_t *scales_t, void *stream)
{
    const nvfp4_status ps = plan_ok(plan, plan_bytes, T, k, E);
    if (ps != NVFP4_OK)
        return ps;
    if (!layer_ok(T, k, E, 1, K) || ldx < K || ldx > (1LL << 30))
        return NVFP4_ERR_SHAPE;
    if (!x || !dtype_ok(x_dtype) || (!codes) != (!scales) || (!codes_t) != (!scales_t) || (!codes && !codes_t))
        return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(x) || !ld_aligned(ldx, x_dtype) || !opt_aligned(codes) || !opt_aligned(scales) ||
        !opt_aligned(codes_t) || !opt_aligned(scales_t))
        return NVFP4_ERR_ALIGNMENT;
    NVFP4_TRY_DEVICE(dev);
    (void)dev;
    const MoeLayout l(T, k, (int)E);
    MxQuantArgs a = quant_args(x, x_dtype, sorted_rows ? l.slots : T, K, ldx);
    a.codes = codes;
    a.scales = scales;
    a.codes_t = codes_t;
    a.scales_t = scales_t;
    const MoeRows m = rows_of(l, plan, k, sorted_rows != 0);
    return from_cuda(codes_t ? launch_mx_quantize_groups(a, m, (cudaStream_t)stream)
                             : launch_mx_quantize_rows(a, m, (cudaStream_t)stream));
}

size_t nvfp4_moe_gemm_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K)
{
    return layer_ok(T, k, E, N, K) ? align256(kWsHeaderBytes) : 0;
}

nvfp4_status nvfp4_moe_gemm(const uint8_t *x_codes, const uint8_t *x_scales, const uint8_t *w_codes,
                            const uint8_t *w_scales, const void *plan, size_t plan_bytes, int64_t T, int64_t k, int64_t E,
                            int64_t N, int64_t K, void *y, nvfp4_dtype y_dtype, void *workspace, size_t ws_bytes,
                            void *stream)
{
    const nvfp4_status ps = plan_ok(plan, plan_bytes, T, k, E);
    if (ps != NVFP4_OK)
        return ps;
    const size_t need = nvfp4_moe_gemm_workspace_bytes(T, k, E, N, K);
    if (need == 0)
        return NVFP4_ERR_SHAPE;
    if (!x_codes || !x_scales || !w_codes || !w_scales || !y || !workspace || !dtype_ok(y_dtype))
        return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(x_codes) || !aligned16(x_scales) || !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(y) ||
        !aligned16(workspace))
        return NVFP4_ERR_ALIGNMENT;
    if (ws_bytes < need)
        return NVFP4_ERR_WORKSPACE;
    NVFP4_TRY_DEVICE(dev);
    MoeGemmArgs a = gemm_args(MoeLayout(T, k, (int)E), plan, N, K, y, y_dtype, workspace);
    a.x_codes = x_codes;
    a.x_scales = x_scales;
    a.w_codes = w_codes;
    a.w_scales = w_scales;
    return from_cuda(launch_moe_gemm(a, (cudaStream_t)stream, *dev));
}

size_t nvfp4_moe_linear_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K)
{
    if (!layer_ok(T, k, E, N, K))
        return 0;
    const int64_t P = nvfp4_moe_padded_rows(T, k, E);
    return align256(kWsHeaderBytes) + align256(code_bytes(P, K)) + align256(scale_bytes(P, K));
}

nvfp4_status nvfp4_moe_linear(const void *x, nvfp4_dtype x_dtype, int64_t ldx, int sorted_rows, const uint8_t *w_codes,
                              const uint8_t *w_scales, const void *plan, size_t plan_bytes, int64_t T, int64_t k, int64_t E,
                              int64_t N, int64_t K, void *y, nvfp4_dtype y_dtype, void *workspace, size_t ws_bytes,
                              void *stream)
{
    const nvfp4_status ps = plan_ok(plan, plan_bytes, T, k, E);
    if (ps != NVFP4_OK)
        return ps;
    const size_t need = nvfp4_moe_linear_workspace_bytes(T, k, E, N, K);
    if (need == 0 || ldx < K || ldx > (1LL << 30))
        return NVFP4_ERR_SHAPE;
    if (!x || !w_codes || !w_scales || !y || !workspace || !dtype_ok(x_dtype) || !dtype_ok(y_dtype))
        return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(x) || !ld_aligned(ldx, x_dtype) || !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(y) ||
        !aligned16(workspace))
        return NVFP4_ERR_ALIGNMENT;
    if (ws_bytes < need)
        return NVFP4_ERR_WORKSPACE;
    NVFP4_TRY_DEVICE(dev);
    const MoeLayout l(T, k, (int)E);
    MxQuantArgs q = quant_args(x, x_dtype, sorted_rows ? l.slots : T, K, ldx);
    q.codes = (uint8_t *)workspace + align256(kWsHeaderBytes);
    q.scales = q.codes + align256(code_bytes(l.padded_rows(), K));
    cudaError_t e = launch_mx_quantize_rows(q, rows_of(l, plan, k, sorted_rows != 0), (cudaStream_t)stream);
    if (e == cudaSuccess) {
        MoeGemmArgs a = gemm_args(l, plan, N, K, y, y_dtype, workspace);
        a.x_codes = q.codes;
        a.x_scales = q.scales;
        a.w_codes = w_codes;
        a.w_scales = w_scales;
        a.after_quantise = true;
        e = launch_moe_gemm(a, (cudaStream_t)stream, *dev);
    }
    return from_cuda(e);
}

size_t nvfp4_moe_linear_backward_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K)
{
    // dX = Q(dY) Q_c(W): over N;  dW = Q_c(dY)^T Q_c(X): over the rows
    if (!layer_ok(T, k, E, N, K) || !layer_ok(T, k, E, K, N) ||
        E * ((N + 255) / 256) * ((K + 255) / 256) > (1LL << 30))
        return 0;
    const int64_t P = nvfp4_moe_padded_rows(T, k, E);
    return align256(kWsHeaderBytes) + align256(code_bytes(P, N)) + align256(scale_bytes(P, N)) +
           align256(code_bytes(N, P)) + align256(scale_bytes(N, P));
}

nvfp4_status nvfp4_moe_linear_backward(const void *dy, nvfp4_dtype dy_dtype, int64_t lddy, const uint8_t *x_codes_t,
                                       const uint8_t *x_scales_t, const uint8_t *w_codes_t, const uint8_t *w_scales_t,
                                       const void *plan, size_t plan_bytes, int64_t T, int64_t k, int64_t E, int64_t N,
                                       int64_t K, void *dx, nvfp4_dtype dx_dtype, void *dw, nvfp4_dtype dw_dtype,
                                       void *workspace, size_t ws_bytes, void *stream)
{
    const nvfp4_status ps = plan_ok(plan, plan_bytes, T, k, E);
    if (ps != NVFP4_OK)
        return ps;
    const size_t need = nvfp4_moe_linear_backward_workspace_bytes(T, k, E, N, K);
    if (need == 0 || lddy < N || lddy > (1LL << 30))
        return NVFP4_ERR_SHAPE;
    if (!dy || !workspace || !dtype_ok(dy_dtype) || !dtype_ok(dx_dtype) || !dtype_ok(dw_dtype) || (!dx && !dw) ||
        (dx && (!w_codes_t || !w_scales_t)) || (dw && (!x_codes_t || !x_scales_t)))
        return NVFP4_ERR_INVALID_ARG;
    if (!aligned16(dy) || !ld_aligned(lddy, dy_dtype) || !opt_aligned(x_codes_t) || !opt_aligned(x_scales_t) ||
        !opt_aligned(w_codes_t) || !opt_aligned(w_scales_t) || !opt_aligned(dx) || !opt_aligned(dw) ||
        !aligned16(workspace))
        return NVFP4_ERR_ALIGNMENT;
    if (ws_bytes < need)
        return NVFP4_ERR_WORKSPACE;
    NVFP4_TRY_DEVICE(dev);
    cudaStream_t s = (cudaStream_t)stream;
    const MoeLayout l(T, k, (int)E);
    const int64_t P = l.padded_rows();
    uint8_t *codes = (uint8_t *)workspace + align256(kWsHeaderBytes), *scales = codes + align256(code_bytes(P, N));
    uint8_t *codes_t = scales + align256(scale_bytes(P, N)), *scales_t = codes_t + align256(code_bytes(N, P));
    MxQuantArgs q = quant_args(dy, dy_dtype, l.slots, N, lddy);
    if (dx) {
        q.codes = codes;
        q.scales = scales;
    }
    if (dw) {
        q.codes_t = codes_t;
        q.scales_t = scales_t;
    }
    const MoeRows m = rows_of(l, plan, k, true);
    cudaError_t e = dw ? launch_mx_quantize_groups(q, m, s) : launch_mx_quantize_rows(q, m, s);
    if (e == cudaSuccess && dx) {
        MoeGemmArgs a = gemm_args(l, plan, K, N, dx, dx_dtype, workspace);
        a.x_codes = codes;
        a.x_scales = scales;
        a.w_codes = w_codes_t;
        a.w_scales = w_scales_t;
        a.after_quantise = true;
        e = launch_moe_gemm(a, s, *dev);
    }
    if (e == cudaSuccess && dw) {
        MoeWgradArgs a = {};
        a.a_codes = codes_t;
        a.a_scales = scales_t;
        a.x_codes = x_codes_t;
        a.x_scales = x_scales_t;
        a.padded_rows = P;
        a.N = N;
        a.K = K;
        a.E = (int)E;
        a.first_block = (const int32_t *)plan + l.first_block;
        a.dw = dw;
        a.dw_fp32 = dw_dtype == NVFP4_OUT_FP32;
        a.ctl = (uint32_t *)workspace;
        e = launch_moe_wgrad(a, s, *dev);
    }
    return from_cuda(e);
}

}  // extern "C"
