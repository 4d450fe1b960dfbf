"""Out-of-bounds writes of the mixture-of-experts and 8-bit calls: every output buffer and workspace sits between guard
bytes of a fixed pattern."""
import pytest
import torch

from tests.test_gpu_guards import Guarded
from tests.test_gpu_guards_fp4 import _call, _intact

pytestmark = pytest.mark.gpu
bf16, f32, u8 = torch.bfloat16, torch.float32, torch.uint8


@pytest.mark.parametrize("T,k,E,N,K", [(1, 1, 1, 1, 32), (1, 8, 60, 96, 160), (37, 3, 5, 129, 96), (130, 2, 3, 264, 288),
                                       (500, 2, 7, 1001, 64), (2000, 1, 3, 520, 256), (3000, 8, 40, 32, 32)])
@pytest.mark.parametrize("dropped", [False, True])
def test_experts(nv, T, k, E, N, K, dropped):
    g = torch.Generator("cuda").manual_seed(T + N)
    lib = nv.load()
    pn = lib.nvfp4_moe_plan_bytes(T, k, E)
    P, R, N32 = lib.nvfp4_moe_padded_rows(T, k, E), T * k, (N + 31) // 32 * 32
    z = torch.randn(T, E, device="cuda", generator=g)
    if dropped:
        z[torch.rand(T, E, device="cuda", generator=g) < 0.5] = -float("inf")
    size = lambda rows, cols: nv.nvfp4_tiled_scale_bytes(rows, cols, nv.FORMAT_MXFP4)  # noqa: E731
    weights, experts, plan = Guarded(R * 4), Guarded(R * 4), Guarded(pn)
    if k <= E:
        for how in (0, 1):
            _call(nv, "nvfp4_moe_route", z.data_ptr(), nv.OUT_FP32, T, E, E, k, how, how, None, 1.0, weights, experts, plan, pn)
            _intact(weights, experts, plan)
            dz = Guarded(T * E * 4)
            _call(nv, "nvfp4_moe_route_backward", weights, z.data_ptr(), nv.OUT_FP32, T, E, E, k, how, how, 1.0, weights,
                  experts, dz, E)
            _intact(dz, weights, experts)
    ws0 = Guarded(256, fill=0)
    _call(nv, "nvfp4_moe_plan", experts, T, k, E, plan, pn, ws0, ws0.n)
    _intact(plan, ws0, experts)
    for dtype, es, code in ((bf16, 2, nv.OUT_BF16), (f32, 4, nv.OUT_FP32)):
        x = torch.randn(T, K, device="cuda", generator=g).to(dtype)
        w = torch.randn(E, N, K, device="cuda", generator=g).to(dtype)
        c, s, ct, st = Guarded(P * K // 2), Guarded(size(P, K)), Guarded(K * P // 2), Guarded(size(K, P))
        for q in ((c, s, None, None), (c, s, ct, st), (None, None, ct, st)):
            _call(nv, "nvfp4_moe_quantize", x.data_ptr(), code, K, 0, plan, pn, T, k, E, K, *q)
            _intact(c, s, ct, st, plan)
        wc, wsc = Guarded(E * N * K // 2), Guarded(E * size(N, K))
        wct, wst = Guarded(E * K * N32 // 2), Guarded(E * size(K, N32))
        _call(nv, "nvfp4_mx_quantize_experts", w.data_ptr(), code, E, N, K, wc, wsc, wct, wst)
        _intact(wc, wsc, wct, wst)
        y = Guarded(R * N * es)
        ws = Guarded(nv.nvfp4_moe_gemm_workspace_bytes(T, k, E, N, K), fill=0)
        _call(nv, "nvfp4_moe_gemm", c, s, wc, wsc, plan, pn, T, k, E, N, K, y, code, ws, ws.n)
        _intact(y, ws, c, s)
        ws = Guarded(nv.nvfp4_moe_linear_workspace_bytes(T, k, E, N, K), fill=0)
        _call(nv, "nvfp4_moe_linear", x.data_ptr(), code, K, 0, wc, wsc, plan, pn, T, k, E, N, K, y, code, ws, ws.n)
        _intact(y, ws)
        out, dw, dy = Guarded(T * N * es), Guarded(R * 4), Guarded(R * N * es)
        _call(nv, "nvfp4_moe_combine", y, code, weights, plan, pn, T, k, E, N, None, out, code)
        _intact(out, y)
        _call(nv, "nvfp4_moe_combine_backward", out, y, code, weights, plan, pn, T, k, E, N, dy, dw)
        _intact(dy, dw, y, out)
        if N % 32 == 0:
            dx, dwt = Guarded(R * K * es), Guarded(E * N * K * es)
            ws = Guarded(nv.nvfp4_moe_linear_backward_workspace_bytes(T, k, E, N, K), fill=0)
            _call(nv, "nvfp4_moe_linear_backward", y, code, N, ct, st, wct, wst, plan, pn, T, k, E, N, K, dx, code, dwt, code,
                  ws, ws.n)
            _intact(dx, dwt, ws, y)


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (3, 130, 48), (20, 257, 3584), (40, 77, 1040), (100, 300, 400), (130, 255, 288),
                                   (300, 1001, 512), (700, 20000, 64)])
def test_int8(nv, M, N, K):
    g = torch.Generator("cuda").manual_seed(M)
    w = torch.randn(N, K, device="cuda", generator=g)
    wc, wsc = Guarded(N * K), Guarded(N * 4)
    _call(nv, "nvfp4_int8_quantize", w.data_ptr(), nv.OUT_FP32, N, K, K, wc, wsc)
    _intact(wc, wsc)
    for dtype, es, code in ((bf16, 2, nv.OUT_BF16), (f32, 4, nv.OUT_FP32)):
        x = torch.randn(M, K, device="cuda", generator=g).to(dtype)
        c, s, y = Guarded(M * K), Guarded(M * 4), Guarded(M * N * es)
        _call(nv, "nvfp4_int8_quantize", x.data_ptr(), code, M, K, K, c, s)
        _intact(c, s)
        ws = Guarded(nv.nvfp4_int8_linear_workspace_bytes(M, N, K), fill=0)
        _call(nv, "nvfp4_int8_gemm", c, s, wc, wsc, M, N, K, y, code, ws, ws.n)
        _intact(y, ws, c, s)
        _call(nv, "nvfp4_int8_linear", x.data_ptr(), code, K, M, N, K, wc, wsc, y, code, ws, ws.n)
        _intact(y, ws)
