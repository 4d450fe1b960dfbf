/*
 * nvfp4.h -- C ABI of libnvfp4.so: the NVFP4 weight path on one GB300 (sm_103a).
 *
 * Two operations make up the path:
 *   1. Weight-only block quantisation of bf16 weights into NVFP4 (activations
 *      stay 16-bit: "RL with NVFP4 + LoRA" post, tggo.me/sberlogasci/42740,
 *      section "Метод").  Each weight becomes an E2M1 code plus the scale of
 *      its block ("Scale-QLoRA", rit.work, format paragraph).  Format: blocks
 *      of 16 consecutive elements of a row, one E4M3 scale byte per block, one
 *      FP32 tensor scale, E2M1 grid {0,.5,1,1.5,2,3,4,6}, round to nearest
 *      even, two codes per byte (even element in the low nibble).
 *   2. The memory-bound W4A16 GEMM used for rollouts ("Marlin-like kernel",
 *      same post, section "Эксперименты") with the parallel LoRA branch (as in
 *      QLoRA, section "Метод") and multiplicative noise applied through the
 *      RMSNorm gain before the projection (section "Метод"):
 *          X' = bf16(X * z),   Y = s_t * X' deq(W)^T + s * (X' A^T) B^T.
 *
 * Conventions for every entry point:
 *   - Pointers are DEVICE pointers owned by the caller, except where a
 *     comment says otherwise.  Arrays are row-major and contiguous; every
 *     pointer must be 16-byte aligned.  The library never allocates device
 *     memory on these paths; scratch space is the caller's workspace.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Calls are asynchronous on that stream, except the host-side
 *     argument checks, which run before anything is launched: when a call
 *     returns an error from the host checks, nothing was launched.
 *   - The current CUDA device must be an sm_103 GPU (GB300); otherwise
 *     NVFP4_ERR_UNSUPPORTED_DEVICE.
 *   - Data-dependent failures (non-finite weights or scales, a device wait
 *     that gave up) never trap: kernels record them in a status word inside
 *     the workspace, read with nvfp4_get_device_status().  Outputs of a call
 *     that recorded such a status are unspecified.
 *   - A workspace must be zero-filled once before its first use (e.g. with
 *     cudaMemsetAsync); every call that completes normally leaves its
 *     counters at zero again.  After a call whose device wait gave up
 *     (NVFP4_ERR_TIMEOUT), its counters and flags may be left mid-way: call
 *     nvfp4_get_device_status() on that workspace, which returns the timeout
 *     and sets them back to zero, before the workspace is used again.  One
 *     workspace serves one call at a time: calls that share a workspace must
 *     be ordered on one stream.
 *
 * Shapes: W is N x K (out x in, the PyTorch Linear layout); codes are N x K/2
 * bytes; scales are N x K/16 bytes; X is M x K; Y is M x N; LoRA A is r x K,
 * LoRA B is N x r; the noise vector z has K floats.  K must be a multiple of
 * 16 (no partial blocks); M, N >= 1; 0 <= r <= 256.
 */
#ifndef NVFP4_H
#define NVFP4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum nvfp4_status {
    NVFP4_OK = 0,
    NVFP4_ERR_INVALID_ARG = 1,        /* null pointer, bad enum value        */
    NVFP4_ERR_SHAPE = 2,              /* K % 16 != 0, M/N < 1, r out of range */
    NVFP4_ERR_ALIGNMENT = 3,          /* a pointer is not 16-byte aligned    */
    NVFP4_ERR_WORKSPACE = 4,          /* workspace missing or too small      */
    NVFP4_ERR_UNSUPPORTED_DEVICE = 5, /* current device is not sm_103        */
    NVFP4_ERR_CUDA = 6,               /* a CUDA runtime call or launch failed */
    NVFP4_ERR_NONFINITE = 7,          /* device: non-finite weight or scale  */
    NVFP4_ERR_TIMEOUT = 8,            /* device: a bounded wait gave up      */
    NVFP4_ERR_INDEX = 9               /* device: an index beyond its range   */
} nvfp4_status;

typedef enum nvfp4_dtype {
    NVFP4_OUT_BF16 = 0,
    NVFP4_OUT_FP32 = 1
} nvfp4_dtype;

/* Bytes of workspace needed by nvfp4_w4a16_lora_gemm for these sizes; also
 * enough for nvfp4_quantize and nvfp4_round_scales (which need only the
 * 256-byte control block at its start).  Returns 0 for invalid sizes. */
size_t nvfp4_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t r);

/* Quantise a bf16 weight matrix W (N x K) into NVFP4.
 *   use_given_tensor_scale == 0 ("dynamic", Nemotron NVFP4/QAD page, section
 *     03 "Dynamic Scale QAD": scales recomputed from the current tensor):
 *     s_t = amax|W| / 2688 (2688 = 6 * 448) is computed on the device and
 *     written to *tensor_scale.
 *   use_given_tensor_scale != 0 ("frozen", same section, "Frozen Scale QAD"):
 *     *tensor_scale is read and used as is; it must be finite and >= 0.
 * Per block b of 16 elements: e_b = E4M3_RNE(amax_b / (6 s_t)) (saturating at
 * 448; 0 when s_t == 0), S_b = fl32(dec(e_b) * s_t); each code is
 * E2M1_RNE(fl32(w / S_b)) with the sign of w, and 0 for the whole block when
 * S_b == 0.  Codes and scales are bit-identical to the CPU definition.
 * Non-finite weights (or a bad frozen scale) record NVFP4_ERR_NONFINITE.
 * Outputs: codes (N x K/2 bytes), scales_e4m3 (N x K/16 bytes),
 * tensor_scale (1 float, device).  workspace: >= 256 bytes. */
nvfp4_status nvfp4_quantize(const void *w_bf16, int64_t N, int64_t K,
                            uint8_t *codes, uint8_t *scales_e4m3, float *tensor_scale,
                            int use_given_tensor_scale, void *workspace, size_t ws_bytes,
                            void *stream);

/* Dequantise ("Scale-QLoRA", rit.work, format paragraph: a weight is its
 * E2M1 code times the shared scale of its block; here times the FP32 tensor
 * scale as well): out[n][k] = fl32(fl32(v(q) * dec(e_b)) * s_t) (the inner
 * product is exact), written as FP32 or rounded to bf16 (RNE).
 * Inputs: codes (N x K/2 bytes), scales_e4m3 (N x K/16 bytes), tensor_scale
 * (1 float, device).  out: N x K floats or bf16 values.  No workspace; nothing
 * is recorded on the device. */
nvfp4_status nvfp4_dequantize(const uint8_t *codes, const uint8_t *scales_e4m3,
                              const float *tensor_scale, int64_t N, int64_t K,
                              void *out, nvfp4_dtype out_dtype, void *stream);

/* Y = s_t * X' deq(W)^T + lora_scale * (X' A^T) B^T, X' = bf16(X * z).
 *   x_bf16: M x K; noise_fp32: K floats or NULL (then X' = X);
 *   lora_a_bf16: r x K, lora_b_bf16: N x r (both NULL or r == 0: no LoRA);
 *   y: M x N, FP32 or bf16 (RNE of the FP32 result).
 * Accumulation is FP32.  M < 64 takes a weight-streaming decode path (per
 * 16 tokens: an activation-preparation kernel, then the GEMM kernel, chained
 * by programmatic dependent launch); M >= 64 takes the tensor-core (tcgen05)
 * prefill kernel, whose workspace holds a bf16 copy of v(q) dec(e) (2 N K
 * bytes) and of X' (2 M K bytes); nvfp4_gemm_kernel() says which.  Any
 * finite tensor scale works on both paths, subnormal ones included: where
 * s / s_t leaves [2^-40, 2^40] the prefill kernel accumulates the LoRA term
 * apart from the weights' term.
 * workspace: nvfp4_workspace_bytes(M, N, K, r) bytes. */
nvfp4_status nvfp4_w4a16_lora_gemm(const void *x_bf16, int64_t M, int64_t N, int64_t K,
                                   const uint8_t *codes, const uint8_t *scales_e4m3,
                                   const float *tensor_scale,
                                   const void *lora_a_bf16, const void *lora_b_bf16,
                                   int64_t r, float lora_scale, const float *noise_fp32,
                                   void *y, nvfp4_dtype y_dtype,
                                   void *workspace, size_t ws_bytes, void *stream);

/* One entry of nvfp4_w4a16_lora_gemm_list.  Each field means what the
 * argument of nvfp4_w4a16_lora_gemm with the same name means (device
 * pointers); the struct array itself is in host memory and is read before the
 * call returns. */
typedef struct nvfp4_projection {
    const void *x_bf16;          /* M x K bf16 (entries may share one X)   */
    const uint8_t *codes;        /* N x K/2 bytes                          */
    const uint8_t *scales_e4m3;  /* N x K/16 bytes                         */
    const float *tensor_scale;   /* 1 float                                */
    const void *lora_a_bf16;     /* r x K bf16; ignored when r == 0        */
    const void *lora_b_bf16;     /* N x r bf16; ignored when r == 0        */
    const float *noise_fp32;     /* K floats or NULL (then X' = X)         */
    void *y;                     /* M x N of the call's y_dtype            */
    int64_t N, K;
    float lora_scale;
} nvfp4_projection;

/* Bytes of workspace for nvfp4_w4a16_lora_gemm_list with these entries (host
 * array of `count`); 0 when the host checks of that call would fail. */
size_t nvfp4_gemm_list_workspace_bytes(const nvfp4_projection *list, int count, int64_t M, int64_t r);

/* Several independent projections of the same token count in one call: for
 * every entry i,
 *     y_i = s_t,i X'_i deq(W_i)^T + lora_scale_i (X'_i A_i^T) B_i^T,
 *     X'_i = bf16(X_i * z_i),
 * the layer of nvfp4_w4a16_lora_gemm ("RL with NVFP4 + LoRA" post, section
 * "Метод"), on the weight-streaming decode path of that call (rollouts are
 * memory-bound on the weights: same post, section "Эксперименты").  This is
 * the shape of a decoder layer's projections that read one input (q, k and v;
 * gate and up), or of any batch of independent GEMMs.
 * One activation-preparation launch serves all entries, then one streaming
 * launch moves every entry's weight bytes back to back, so the fixed cost of
 * a call (the dependency chain from the preparation kernel, filling the
 * ring, the last tile's epilogue) is paid once per launch instead of once per
 * projection.  Entries go 64 at a time into a launch (fewer if their
 * 128-row tiles exceed 8192); M > 16 runs in groups of 16 tokens.
 * Each y_i agrees with nvfp4_w4a16_lora_gemm's result for that entry to
 * FP32 summation order (the split of K over blocks can differ); a one-entry
 * list computes exactly what nvfp4_w4a16_lora_gemm computes for M < 64.
 * Requirements (checked on the host before anything is launched):
 *   list != NULL, 1 <= count <= 65536 (else NVFP4_ERR_INVALID_ARG /
 *   NVFP4_ERR_SHAPE); 1 <= M <= 2^31, 0 <= r <= 64; per entry: 256 <= K
 *   <= 2^30 and K % 256 == 0, 1 <= N <= 1048576 (NVFP4_ERR_SHAPE); x, codes,
 *   scales, tensor_scale and y non-null, and A and B non-null when r > 0
 *   (NVFP4_ERR_INVALID_ARG); every pointer 16-byte aligned
 *   (NVFP4_ERR_ALIGNMENT).
 * No y_i may overlap another entry's y or any input of the list.
 * workspace: nvfp4_gemm_list_workspace_bytes(list, count, M, r) bytes. */
nvfp4_status nvfp4_w4a16_lora_gemm_list(const nvfp4_projection *list, int count, int64_t M, int64_t r,
                                        nvfp4_dtype y_dtype, void *workspace, size_t ws_bytes,
                                        void *stream);

/* Input gradient of nvfp4_w4a16_lora_gemm's layer.  The quantised weight is
 * frozen and only the LoRA factors are trained ("RL with NVFP4 + LoRA"
 * post, section "Метод"), so the backward pass needs the gradient with
 * respect to the layer input:
 *     dX = (dY deq(W) + lora_scale (dY B) A) diag(z),
 * deq(W) = s_t v(q) dec(e) untransposed (N x K), the bf16 rounding of
 * X' = X z taken as the identity.
 *   dy_bf16: M x N (device); dx: M x K, FP32 or bf16 (RNE of the FP32
 *   result); codes, scales_e4m3, tensor_scale as in nvfp4_w4a16_lora_gemm;
 *   lora_a_bf16: r x K, lora_b_bf16: N x r (both NULL or r == 0: no LoRA);
 *   noise_fp32: the forward's z (K floats) or NULL.
 * Shapes: M >= 1; N and K multiples of 64; r <= 64 (else NVFP4_ERR_SHAPE).
 * Runs on the tensor-core (tcgen05) kernel of the forward with the roles of
 * the weight's rows and columns exchanged; its workspace holds a bf16 copy of
 * (v(q) dec(e))^T (2 N K bytes) and of dY (2 M N bytes).  Accumulation is
 * FP32; any finite tensor scale works.  Every check runs before anything is
 * queued.  workspace: nvfp4_dgrad_workspace_bytes(M, N, K, r) bytes, 16-byte
 * aligned, owned by the caller; calls that share a workspace must not overlap
 * in time. */
nvfp4_status nvfp4_w4a16_lora_gemm_dgrad(const void *dy_bf16, int64_t M, int64_t N, int64_t K,
                                         const uint8_t *codes, const uint8_t *scales_e4m3,
                                         const float *tensor_scale,
                                         const void *lora_a_bf16, const void *lora_b_bf16,
                                         int64_t r, float lora_scale, const float *noise_fp32,
                                         void *dx, nvfp4_dtype dx_dtype,
                                         void *workspace, size_t ws_bytes, void *stream);

/* Bytes of workspace needed by nvfp4_w4a16_lora_gemm_dgrad (0 for shapes it
 * does not take). */
size_t nvfp4_dgrad_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t r);

/* Gradients of the LoRA factors of nvfp4_w4a16_lora_gemm's layer, the
 * parameters the RL post trains on a frozen NVFP4 weight ("RL with NVFP4 +
 * LoRA", section "Метод"):
 *     grad_b = lora_scale dY^T (X' A^T)      (N x r, FP32),
 *     grad_a = lora_scale (dY B)^T X'        (r x K, FP32),
 * X' = bf16(X z) as in the forward.
 *   x_bf16: M x K, noise_fp32: K floats or NULL, dy_bf16: M x N (device);
 *   lora_a_bf16: r x K, lora_b_bf16: N x r; grad_a, grad_b: device FP32,
 *   overwritten (not accumulated).
 * Shapes: M >= 1; N and K multiples of 64; 1 <= r <= 64 (else
 * NVFP4_ERR_SHAPE).  The token sums run in FP32 on the tensor cores with the
 * (X' A^T) and (dY B) rows as bf16 hi + lo pairs; the token ranges' partial sums are
 * added in a fixed order, so results do not depend on scheduling.  Every
 * check runs before anything is queued.  workspace:
 * nvfp4_lora_grads_workspace_bytes(M, N, K, r) bytes, 16-byte aligned, owned
 * by the caller; calls that share a workspace must not overlap in time. */
nvfp4_status nvfp4_lora_grads(const void *x_bf16, const float *noise_fp32, const void *dy_bf16,
                              int64_t M, int64_t N, int64_t K,
                              const void *lora_a_bf16, const void *lora_b_bf16, int64_t r,
                              float lora_scale, float *grad_a, float *grad_b,
                              void *workspace, size_t ws_bytes, void *stream);

/* Bytes of workspace needed by nvfp4_lora_grads (0 for shapes it does not
 * take). */
size_t nvfp4_lora_grads_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t r);

/* Scale-QLoRA forward (Scale-QLoRA post, method): the block scales are
 * trainable FP32 parameters (decoded block scales in weight units, N x K/16,
 * as for nvfp4_round_scales) and the codes stay frozen.  Each call rounds the
 * parameters to E4M3 against *tensor_scale into scales_e4m3 (exactly
 * nvfp4_round_scales: parameters <= 0 give 0, non-finite ones record
 * NVFP4_ERR_NONFINITE) and then runs nvfp4_w4a16_lora_gemm with codes,
 * scales_e4m3 and the same remaining arguments, on the same stream.  On
 * return scales_e4m3 holds the merged model's scales: merging is this
 * rounding, with the codes copied verbatim.  scales_e4m3: N x K/16 bytes,
 * caller-owned, 16-byte aligned.  Every host check of both steps runs before
 * anything is launched.  workspace: nvfp4_workspace_bytes(M, N, K, r). */
nvfp4_status nvfp4_scale_qlora_gemm(const void *x_bf16, int64_t M, int64_t N, int64_t K,
                                    const uint8_t *codes, const float *scale_param,
                                    const float *tensor_scale, uint8_t *scales_e4m3,
                                    const void *lora_a_bf16, const void *lora_b_bf16,
                                    int64_t r, float lora_scale, const float *noise_fp32,
                                    void *y, nvfp4_dtype y_dtype,
                                    void *workspace, size_t ws_bytes, void *stream);

/* Which kernel family nvfp4_w4a16_lora_gemm runs for these sizes on the
 * current device (no counterpart on the pages): "prefill_tcgen05" (M >= 64,
 * K % 64 == 0, r <= 64), "decode_stream" (TMA-streaming decode GEMM:
 * K % 256 == 0, r <= 64), "decode_registers" (any other shape), or NULL for
 * invalid sizes or an unsupported device.  A static string. */
const char *nvfp4_gemm_kernel(int64_t M, int64_t N, int64_t K, int64_t r);

/* Diagnostics (no counterpart on the pages): make one of the library's
 * bounded device-side waits run out on purpose -- which == 0: an mbarrier
 * wait that no arrival completes; which == 1: a grid barrier expecting one
 * block more than are launched; which == 2: an mbarrier wait in a kernel
 * that has already counted arrivals at four output tiles, as a decode GEMM
 * block does, so its tile counters are left non-zero.  The wait gives up
 * after about two seconds and records NVFP4_ERR_TIMEOUT in the workspace
 * status word; nvfp4_get_device_status reports it and sets the counters back
 * to zero.  The context stays usable.  workspace: zero-filled, >= 256 bytes
 * for which 0 and 1, >= nvfp4_workspace_bytes(1, 128, 256, 0) for which 2. */
nvfp4_status nvfp4_wait_selftest(void *workspace, int which, void *stream);

/* nvfp4_w4a16_lora_gemm without a workspace argument, for callers that
 * cannot allocate device memory: code running inside a host framework that
 * owns every device allocation and hands its plugins no scratch, or a
 * latency-critical loop that cannot afford cudaMalloc's implicit device-wide
 * synchronisation.  (No counterpart on the pages.)
 *   - Scratch is a fixed 8 MiB array inside the library (a file-scope
 *     __device__ array), held on every GPU that loads the library until the
 *     process exits.  Problems whose workspace (nvfp4_workspace_bytes) exceeds
 *     8 MiB are rejected with NVFP4_ERR_WORKSPACE; every Qwen2.5-7B and -32B
 *     projection at M <= 16 fits.
 *   - Allocates nothing: no cudaMalloc, cudaFree or allocating library call.
 *     The caller still passes inputs and outputs as for the workspace variant.
 *   - The first call on a device looks up the array's device address (once per
 *     device and driver context, with that device current) and caches it;
 *     make that first call before any stream capture.  After a device reset
 *     the next call looks the address up again.
 *   - Every host check of nvfp4_w4a16_lora_gemm (and the size limit) runs
 *     before anything is queued.  Then the call clears the array's control
 *     words (an asynchronous memset on `stream`) and launches; all calls share
 *     the one array, so two calls whose executions overlap on the GPU
 *     (different streams, no ordering) race on it and give wrong results.
 *   - The device status word lives in the shared array and is cleared by the
 *     next call; this variant does not report device-side statuses. */
nvfp4_status nvfp4_w4a16_lora_gemm_static(const void *x_bf16, int64_t M, int64_t N, int64_t K,
                                          const uint8_t *codes, const uint8_t *scales_e4m3,
                                          const float *tensor_scale,
                                          const void *lora_a_bf16, const void *lora_b_bf16,
                                          int64_t r, float lora_scale, const float *noise_fp32,
                                          void *y, nvfp4_dtype y_dtype, void *stream);

/* Scale-only update (Scale-QLoRA page: codes frozen, trained block-scale
 * corrections rounded onto the target scale grid; the merge writes only the
 * scale bytes, so merged weights are bit-identical to the training forward;
 * the guarantee holds while format, scale grid, blocking and codes are
 * unchanged).  scales_e4m3[i] = E4M3_RNE(scale_param[i] / s_t), saturating;
 * 0 for a parameter <= 0 or for s_t == 0.  scale_param holds the effective
 * block scale in weight units (N x K/16 floats).  Codes are not an argument.
 * A non-finite parameter records NVFP4_ERR_NONFINITE and gives byte 0. */
nvfp4_status nvfp4_round_scales(const float *scale_param, const float *tensor_scale,
                                int64_t N, int64_t K, uint8_t *scales_e4m3,
                                void *workspace, size_t ws_bytes, void *stream);

/* Synchronises `stream`, returns the device status recorded in `workspace`
 * since the last read (NVFP4_OK if none) and clears it. */
nvfp4_status nvfp4_get_device_status(void *workspace, void *stream);

/* Static description of a status code. */
const char *nvfp4_status_string(nvfp4_status s);

/* Diagnostics (no counterpart on the pages): run the device's scalar
 * encoders on n device floats x and write one byte per input:
 *   which == 0: the E2M1 code of x (magnitude code 0..7, sign in bit 3);
 *   which == 1: the E4M3 byte of x (x >= 0, round to nearest even,
 *               saturating at 448).
 * Lets the tests compare the device encoders with the CPU definition over
 * large input sets. */
nvfp4_status nvfp4_encode_debug(const float *x, int64_t n, int which, uint8_t *out,
                                void *stream);

/* Diagnostics (no counterpart on the pages): the quantiser forms w / S_b
 * without a division per element (one correctly rounded reciprocal per block
 * and a fused remainder correction).  This sweeps every bf16 significand w
 * against every fp32 significand of S in [sig_lo, sig_hi) (23-bit values),
 * for quotient exponents -3..3, and adds to *mismatches (device u64) the
 * number of pairs where that quotient differs from IEEE division. */
nvfp4_status nvfp4_quotient_check(uint32_t sig_lo, uint32_t sig_hi,
                                  unsigned long long *mismatches, void *stream);

/* ------------------------------------------------------------------------
 * Four-bit activations and distillation: the operators of a quantisation-
 * aware distillation step (Nemotron NVFP4/QAD page, section 03: a student in
 * 4 bits trained against a teacher) and of a layer whose activations are in 4
 * bits as well (W4A4).
 *
 * A 4-bit operand is a rows x cols matrix with its blocks along cols (the
 * axis that a product contracts): E2M1 codes, rows x cols/2 bytes, even
 * element in the low nibble, and one scale byte per block:
 *   NVFP4_FORMAT_MXFP4: blocks of 32, E8M0 scales (byte e stands for
 *     2^(e-127), 255 for NaN);
 *   NVFP4_FORMAT_NVFP4: blocks of 16, E4M3 scales, one FP32 tensor scale.
 * cols is a multiple of 32 in the entry points below.
 * Scales are TILED, the layout the tensor cores copy: tiles of 128 rows x 4
 * blocks, 512 bytes each, the tiles of 128 rows one after the other along
 * cols; block j of row r is byte 16 (r % 32) + 4 (r % 128 / 32) + j % 4 of
 * tile (r / 128, j / 4).  Bytes of rows and blocks that do not exist are 0.
 */
typedef enum nvfp4_fp4_format {
    NVFP4_FORMAT_MXFP4 = 0,
    NVFP4_FORMAT_NVFP4 = 1
} nvfp4_fp4_format;

/* Bytes of the tiled scales of a rows x cols operand (0 for invalid sizes;
 * cols a multiple of the block: 32, or 16 for NVFP4). */
size_t nvfp4_tiled_scale_bytes(int64_t rows, int64_t cols, nvfp4_fp4_format format);

/* Row-major scale bytes (rows x cols/block, as nvfp4_quantize writes them for
 * NVFP4 and as checkpoints hold them) -> tiled. */
nvfp4_status nvfp4_tile_scales(const uint8_t *scales, int64_t rows, int64_t cols, nvfp4_fp4_format format,
                               uint8_t *tiled, void *stream);

/* MXFP4 quantisation of x (rows x cols, bf16 or FP32, ld elements between
 * rows), in one read of x:
 *   codes, scales: blocks along cols (an operand rows x cols);
 *   codes_t, scales_t: blocks along rows, transposed: an operand cols x
 *     rows32, rows32 = rows rounded up to 32, the missing rows taken as 0
 *     (what a product that contracts over the rows needs: a layer's weight
 *     gradient, and its input gradient for the weight);
 *   values_bf16, values_t_bf16: rows x cols, x as its codes and scales stand
 *     for it (exact in bf16), with the blocks along cols and along rows.
 * Each output may be NULL; codes and scales of a direction go together; at
 * least one output.  Per block: scale byte max(F - 2, 0), F the FP32 exponent
 * field of the largest magnitude, i.e. exponent floor(log2 amax) - 2 (the
 * microscaling formats' rule: magnitudes above 6 scales saturate); code
 * E2M1_RNE(x / scale) with the sign of x.  A block with an infinity or a NaN
 * has byte 255 and codes 0: its values are NaN.
 * rows >= 1, cols a positive multiple of 32, both <= 2^30, ld >= cols; x and
 * every row of it on 16-byte boundaries (ld a multiple of 8, FP32: 4). */
nvfp4_status nvfp4_mx_quantize(const void *x, nvfp4_dtype x_dtype, int64_t rows, int64_t cols, int64_t ld,
                               uint8_t *codes, uint8_t *scales, void *values_bf16,
                               uint8_t *codes_t, uint8_t *scales_t, void *values_t_bf16, void *stream);

/* The values of an MXFP4 operand (tiled scales) as FP32 or bf16, exact:
 * out is rows x cols. */
nvfp4_status nvfp4_mx_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows, int64_t cols,
                                 void *out, nvfp4_dtype out_dtype, void *stream);

/* Y = s_a s_w A W^T from two 4-bit operands of one format (A: M x K, W: N x
 * K, tiled scales), FP32 accumulation on the block-scaled tensor cores; Y: M x
 * N, FP32 or bf16 (RNE of the FP32 result).  a_tensor_scale, w_tensor_scale:
 * one device float each, or NULL for 1.  1 <= M, N <= 2^30, 32 <= K <= 2^30,
 * K % 32 == 0.  Results do not depend on scheduling.  workspace:
 * nvfp4_w4a4_workspace_bytes(M, N, K) bytes (0 for sizes it does not take). */
size_t nvfp4_w4a4_workspace_bytes(int64_t M, int64_t N, int64_t K);
nvfp4_status nvfp4_w4a4_gemm(nvfp4_fp4_format format, const uint8_t *a_codes, const uint8_t *a_scales,
                             const float *a_tensor_scale, const uint8_t *w_codes, const uint8_t *w_scales,
                             const float *w_tensor_scale, int64_t M, int64_t N, int64_t K, void *y,
                             nvfp4_dtype y_dtype, void *workspace, size_t ws_bytes, void *stream);

/* A layer with 4-bit weights and activations: Y = Q(X) W^T, X: M x K bf16 or
 * FP32 (ldx elements between rows, as in nvfp4_mx_quantize), Q the MXFP4
 * quantiser along K, W an MXFP4 operand N x K.  The same Y as
 * nvfp4_mx_quantize followed by nvfp4_w4a4_gemm, any M >= 1 (one token
 * upwards).  workspace: nvfp4_mx_linear_workspace_bytes(M, N, K) bytes. */
size_t nvfp4_mx_linear_workspace_bytes(int64_t M, int64_t N, int64_t K);
nvfp4_status nvfp4_mx_linear(const void *x, nvfp4_dtype x_dtype, int64_t ldx, int64_t M, int64_t N, int64_t K,
                             const uint8_t *w_codes, const uint8_t *w_scales, void *y, nvfp4_dtype y_dtype,
                             void *workspace, size_t ws_bytes, void *stream);

/* The layer's backward pass with straight-through quantisers, both products
 * on 4-bit operands quantised along the axis they contract:
 *     dX = Q(dY) Q_c(W)          (M x K, over N),
 *     dW = Q_c(dY)^T Q_c(X)      (N x K, over M),
 * dY: M x N bf16 or FP32 (lddy elements between rows); Q_c(X) and Q_c(W) are
 * the codes_t, scales_t that nvfp4_mx_quantize wrote for X (K x M32) and W (K
 * x N).  dx, dw: FP32 or bf16, overwritten; either may be NULL (then its
 * operand may be NULL too).  M >= 1, N and K multiples of 32.
 * workspace: nvfp4_mx_linear_backward_workspace_bytes(M, N, K) bytes. */
size_t nvfp4_mx_linear_backward_workspace_bytes(int64_t M, int64_t N, int64_t K);
nvfp4_status nvfp4_mx_linear_backward(const void *dy, nvfp4_dtype dy_dtype, int64_t lddy, int64_t M, int64_t N,
                                      int64_t K, const uint8_t *x_codes_t, const uint8_t *x_scales_t,
                                      const uint8_t *w_codes_t, const uint8_t *w_scales_t, void *dx,
                                      nvfp4_dtype dx_dtype, void *dw, nvfp4_dtype dw_dtype, void *workspace,
                                      size_t ws_bytes, void *stream);

/* Distillation from a teacher's top logits, loss and gradient (Nemotron
 * NVFP4/QAD page, section 03: KL divergence between the teacher's and the
 * 4-bit student's output distributions).  Per row t of the student's logits z
 * (T x V, bf16 or FP32, ldz elements between rows) with q = softmax(z / tau)
 * and the teacher's k entries (index[t][j], teacher[t][j]):
 *   rest_class == 0: teacher values are logits, p = softmax_j(teacher / tau);
 *     loss[t] = w tau^2 sum_j p_j (log p_j - log q_j);
 *   rest_class != 0: teacher values are log-probabilities at temperature tau,
 *     p_j = exp(teacher_j); the mass the teacher did not list is one more
 *     class, p_r = max(0, 1 - sum_j p_j), q_r = the sum of q over the entries
 *     not listed (no such class when every entry of the vocabulary is listed):
 *     loss[t] = w tau^2 [sum_j p_j (log p_j - log q_j) + p_r (log p_r - log q_r)].
 * w = row_weight[t] (NULL: 1).  dz (T x V, z's type, lddz elements between
 * rows) = grad_loss[t] times the derivative of loss[t]; grad_loss: T floats,
 * or one for all rows (grad_loss_count 1), or NULL for 1.  dz may be z itself
 * (with lddz == ldz) and must not overlap it otherwise.  loss or dz may be
 * NULL; dz alone is the backward pass.
 *   - A negative index marks an unused slot, whose value is not looked at.
 *     Used indices of a row are distinct, as a top-k's are.  An index >= V is
 *     taken as unused and recorded as NVFP4_ERR_INDEX when there is a
 *     workspace (zero-filled, >= 256 bytes; NULL: not recorded).
 *   - A teacher value of -inf has p = 0.  A row of weight 0, without a used
 *     slot, or (rest_class == 0) whose used values are all -inf gives loss 0
 *     and gradient 0, whatever its logits hold.
 *   - A student logit of -inf has q = 0: the loss is +inf where the teacher
 *     gives it mass, the gradient stays finite.  A NaN or +inf among the
 *     logits, or a row of nothing but -inf, makes the row's loss and gradient
 *     NaN.
 *   - A device-side wait that gives up makes the loss and gradient of its row
 *     (and of the rows behind it in the same block) NaN, and is recorded as
 *     NVFP4_ERR_TIMEOUT when there is a workspace.
 * T >= 1; 1 <= V, a row of at most 1638272 bytes; 1 <= k <= 1024; index_bytes
 * 4 or 8; temperature positive, it and log2(e) / temperature finite (FP32).
 * z, dz 16-byte aligned as every pointer; ldz, lddz >= V arbitrary. */
nvfp4_status nvfp4_distill_topk(const void *z, nvfp4_dtype z_dtype, int64_t T, int64_t V, int64_t ldz,
                                const void *index, int index_bytes, const void *teacher,
                                nvfp4_dtype teacher_dtype, int64_t k, float temperature, int rest_class,
                                const float *row_weight, const float *grad_loss, int64_t grad_loss_count,
                                float *loss, void *dz, int64_t lddz, void *workspace, size_t ws_bytes,
                                void *stream);

/* Self-check: nvfp4_distill_topk (contiguous logits, int32 indices, FP32
 * teacher values, temperature 1, no grad_loss) in which every wait for a copy
 * gives up at once.  Rows of weight 0 or without an entry give 0 as ever, the
 * others NaN. */
nvfp4_status nvfp4_distill_wait_selftest(const void *z, nvfp4_dtype z_dtype, int64_t T, int64_t V,
                                         const int32_t *index, const float *teacher, int64_t k, int rest_class,
                                         const float *row_weight, float *loss, void *dz, void *workspace,
                                         size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Mixtures of experts on MXFP4 operands: routing, the layer with one weight
 * matrix an expert and ragged numbers of rows, and the weighted sum back to
 * the tokens, forward and backward.
 *
 * A token t has k choices; slot t k + j is choice j of token t.  The slots
 * that have an expert are grouped: sorted by expert, in the order of their
 * numbers within one.  Rows of the experts' inputs and outputs are compact in
 * that order: row r belongs to slot order[r].  Rows behind the last one (slots
 * without an expert leave some) are neither read nor written.  The grouping is
 * held in a PLAN, a device buffer of nvfp4_moe_plan_bytes(T, k, E) bytes that
 * the calls below read (int32 arrays, at the byte offsets that
 * nvfp4_moe_plan_part gives):
 *   NVFP4_MOE_OFFSETS:  E + 1: rows offsets[e] .. offsets[e + 1] - 1 are expert e's;
 *   NVFP4_MOE_ORDER:    T k: slot of each row, -1 behind the last one;
 *   NVFP4_MOE_POSITION: T k: row of each slot, -1 without an expert.
 * 1 <= T, T k <= 2^24, 1 <= k <= 32, 1 <= E <= 1024.
 */
typedef enum nvfp4_moe_part {
    NVFP4_MOE_OFFSETS = 0,
    NVFP4_MOE_ORDER = 1,
    NVFP4_MOE_POSITION = 2
} nvfp4_moe_part;
typedef enum nvfp4_moe_scoring {
    NVFP4_MOE_SOFTMAX = 0,
    NVFP4_MOE_SIGMOID = 1
} nvfp4_moe_scoring;

size_t nvfp4_moe_plan_bytes(int64_t T, int64_t k, int64_t E);   /* 0 for sizes it does not take */
size_t nvfp4_moe_plan_part(int64_t T, int64_t k, int64_t E, nvfp4_moe_part part);

/* The k experts of every token from its logits z (T x E, bf16 or FP32, ldz
 * elements between rows), their weights, and the plan.
 *   score s = softmax(z) or sigmoid(z) (elementwise);
 *   experts: the k largest of s + bias in FP32 (E floats; NULL: of z), in
 *     descending order, equal ones by index; k <= E;
 *   weights: scale * s_j, or with renormalise != 0 scale * s_j / (sum of the
 *     k scores taken).  The bias chooses and is not part of the weight.
 * An expert whose logit is -inf (or whose s + bias is -inf or NaN) is not taken: a slot that finds none
 * has expert -1 and weight 0, and a row of nothing but -inf has no expert.  A
 * NaN among a token's logits (softmax: or +inf) makes its weights NaN.
 * weights: T x k floats, experts: T x k int32, both written. */
nvfp4_status nvfp4_moe_route(const void *z, nvfp4_dtype z_dtype, int64_t T, int64_t E, int64_t ldz, int64_t k,
                             nvfp4_moe_scoring scoring, int renormalise, const float *bias, float scale,
                             float *weights, int32_t *experts, void *plan, size_t plan_bytes, void *stream);

/* dz (T x E, z's type, lddz elements between rows) from the gradient of the
 * weights (T x k floats), with z, weights and experts as nvfp4_moe_route took
 * and gave them.  The choice itself has no gradient; slots without an expert
 * add nothing.  dz must not overlap z. */
nvfp4_status nvfp4_moe_route_backward(const float *dweights, const void *z, nvfp4_dtype z_dtype, int64_t T,
                                      int64_t E, int64_t ldz, int64_t k, nvfp4_moe_scoring scoring,
                                      int renormalise, float scale, const float *weights, const int32_t *experts,
                                      void *dz, int64_t lddz, void *stream);

/* The plan of given experts (T x k int32; negative: the slot has none).  A
 * token may have an expert twice.  An index >= E is taken as none and recorded
 * as NVFP4_ERR_INDEX when there is a workspace (zero-filled, >= 256 bytes;
 * NULL: not recorded).  Rows that are sorted by expert already are tokens with
 * k = 1: order is then the identity. */
nvfp4_status nvfp4_moe_plan(const int32_t *experts, int64_t T, int64_t k, int64_t E, void *plan, size_t plan_bytes,
                            void *workspace, size_t ws_bytes, void *stream);

/* out[t] = base[t] + sum over j of weights[t][j] y[position[t][j]], FP32
 * sums in the order of j.  y: rows x N; weights: T x k floats or NULL for 1
 * (a slot without an expert adds nothing, unless its weight is a NaN); base: T
 * x N of out's type or NULL; out: T x N, may be base.  bf16 or FP32. */
nvfp4_status nvfp4_moe_combine(const void *y, nvfp4_dtype y_dtype, const float *weights, const void *plan,
                               size_t plan_bytes, int64_t T, int64_t k, int64_t E, int64_t N, const void *base,
                               void *out, nvfp4_dtype out_dtype, void *stream);

/* Its backward pass: dy[position[t][j]] = weights[t][j] dout[t] (rows x N) and
 * dweights[t][j] = <dout[t], y[position[t][j]]> (0 without an expert).  dout,
 * y, dy of one type; either output may be NULL, and y with dweights.  dy may
 * be y.  The gradient of base is dout. */
nvfp4_status nvfp4_moe_combine_backward(const void *dout, const void *y, nvfp4_dtype dtype, const float *weights,
                                        const void *plan, size_t plan_bytes, int64_t T, int64_t k, int64_t E,
                                        int64_t N, void *dy, float *dweights, void *stream);

/* MXFP4 operands of the experts' products.  Every expert's rows begin on a
 * multiple of 128 in them: P = nvfp4_moe_padded_rows(T, k, E) rows.
 *   codes, scales: P x K, blocks along K (what a row's padding holds is
 *     unspecified: it is not part of any product);
 *   codes_t, scales_t: K x P, blocks of 32 along an expert's own rows, zeros
 *     behind its last.
 * x: T x K tokens (sorted_rows == 0), a token's row going to each of its
 * experts, or T k rows in the experts' order, of which the last ones may be
 * unused; bf16 or FP32, ldx elements between rows (16-byte aligned). */
int64_t nvfp4_moe_padded_rows(int64_t T, int64_t k, int64_t E);   /* 0 for sizes it does not take */
nvfp4_status nvfp4_moe_quantize(const void *x, nvfp4_dtype x_dtype, int64_t ldx, int sorted_rows, const void *plan,
                                size_t plan_bytes, int64_t T, int64_t k, int64_t E, int64_t K, uint8_t *codes,
                                uint8_t *scales, uint8_t *codes_t, uint8_t *scales_t, void *stream);

/* The experts' weights (E x N x K, contiguous, bf16 or FP32) as E operands
 * behind one another, each as nvfp4_mx_quantize writes it: codes (E x N x
 * K/2) and tiled scales; codes_t (E x K x N32/2) and scales_t. */
nvfp4_status nvfp4_mx_quantize_experts(const void *w, nvfp4_dtype w_dtype, int64_t E, int64_t N, int64_t K,
                                       uint8_t *codes, uint8_t *scales, uint8_t *codes_t, uint8_t *scales_t,
                                       void *stream);

/* y (rows x N, FP32 or bf16) = x W_e^T for the rows of each expert e, FP32
 * accumulation; x as nvfp4_moe_quantize writes it, W: E operands N x K.
 * Results do not depend on scheduling.  1 <= N <= 2^24, K a multiple of 32 up
 * to 2^24.  workspace: nvfp4_moe_gemm_workspace_bytes(...) bytes (0 for sizes it
 * does not take). */
size_t nvfp4_moe_gemm_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K);
nvfp4_status nvfp4_moe_gemm(const uint8_t *x_codes, const uint8_t *x_scales, const uint8_t *w_codes,
                            const uint8_t *w_scales, const void *plan, size_t plan_bytes, int64_t T, int64_t k,
                            int64_t E, int64_t N, int64_t K, void *y, nvfp4_dtype y_dtype, void *workspace,
                            size_t ws_bytes, void *stream);

/* The layer: y (rows x N) = Q(x) W_e^T, x as nvfp4_moe_quantize takes it. */
size_t nvfp4_moe_linear_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K);
nvfp4_status nvfp4_moe_linear(const void *x, nvfp4_dtype x_dtype, int64_t ldx, int sorted_rows,
                              const uint8_t *w_codes, const uint8_t *w_scales, const void *plan, size_t plan_bytes,
                              int64_t T, int64_t k, int64_t E, int64_t N, int64_t K, void *y, nvfp4_dtype y_dtype,
                              void *workspace, size_t ws_bytes, void *stream);

/* The layer's backward pass with straight-through quantisers:
 *     dX_r = Q(dY_r) Q_c(W_e)           (rows x K, over N; sum it over a token's
 *                                        slots with nvfp4_moe_combine),
 *     dW_e = Q_c(dY_e)^T Q_c(X_e)       (E x N x K, over the expert's rows; zeros
 *                                        for an expert without any),
 * dY: T k rows x N in the experts' order, bf16 or FP32; Q_c(X), Q_c(W): the
 * codes_t, scales_t of nvfp4_moe_quantize and nvfp4_mx_quantize_experts.  dx,
 * dw: FP32 or bf16, overwritten; either may be NULL (then its operand may be
 * NULL too).  N and K multiples of 32. */
size_t nvfp4_moe_linear_backward_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t N, int64_t K);
nvfp4_status nvfp4_moe_linear_backward(const void *dy, nvfp4_dtype dy_dtype, int64_t lddy, const uint8_t *x_codes_t,
                                       const uint8_t *x_scales_t, const uint8_t *w_codes_t,
                                       const uint8_t *w_scales_t, const void *plan, size_t plan_bytes, int64_t T,
                                       int64_t k, int64_t E, int64_t N, int64_t K, void *dx, nvfp4_dtype dx_dtype,
                                       void *dw, nvfp4_dtype dw_dtype, void *workspace, size_t ws_bytes,
                                       void *stream);

/* ------------------------------------------------------------------------
 * 8-bit integers with one FP32 scale for each token and output channel, for
 * layers that 4 bits do not suit: quantiser of rows, product, layer.
 *
 * Quantisation of the rows of x (rows x cols, bf16 or FP32, ld elements between
 * rows): scale = amax / 127, code = the integer next to 127 x / amax, ties to
 * even (amax: the row's largest magnitude).  A row of zeros has scale 0 and
 * codes 0; a row with an infinity or a NaN scale NaN and codes 0.
 * 1 <= rows <= 2^30, cols a multiple of 16 up to 131072; x and its rows on
 * 16-byte boundaries. */
nvfp4_status nvfp4_int8_quantize(const void *x, nvfp4_dtype x_dtype, int64_t rows, int64_t cols, int64_t ld,
                                 int8_t *codes, float *scales, void *stream);

/* Y[m][n] = a_scales[m] w_scales[n] sum over k of a[m][k] w[n][k] (A: M x K,
 * W: N x K codes), FP32 or bf16 (RNE of the FP32 result).  The integers are
 * summed in FP32: exactly while the sums of a row's products stay below 2^24
 * in magnitude, as sums of codes of either sign do.  Beyond, 16 products are added
 * at a time with an error of up to 4.5 steps (2^-23) of the running sum: for codes
 * of one sign 3e-4 of the whole at K = 18944 and 2e-3 at 131072 (3e-5 and 5e-4
 * measured with uniform ones), and the digits behind that differ with M and N,
 * which decide how K is shared out.  Results do not depend on scheduling.  Codes
 * are -127 .. 127 (-128 is taken as it is).  K a multiple of 16 up to 131072.  workspace:
 * nvfp4_int8_linear_workspace_bytes(M, N, K) bytes (0 for sizes it does not take). */
size_t nvfp4_int8_linear_workspace_bytes(int64_t M, int64_t N, int64_t K);
nvfp4_status nvfp4_int8_gemm(const int8_t *a_codes, const float *a_scales, const int8_t *w_codes,
                             const float *w_scales, int64_t M, int64_t N, int64_t K, void *y, nvfp4_dtype y_dtype,
                             void *workspace, size_t ws_bytes, void *stream);

/* The layer: nvfp4_int8_quantize of the tokens x (M x K, bf16 or FP32, ldx
 * elements between rows), then nvfp4_int8_gemm, the same Y; any M >= 1. */
nvfp4_status nvfp4_int8_linear(const void *x, nvfp4_dtype x_dtype, int64_t ldx, int64_t M, int64_t N, int64_t K,
                               const int8_t *w_codes, const float *w_scales, void *y, nvfp4_dtype y_dtype,
                               void *workspace, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_H */
