"""Host-side checks of the 4-bit activation and distillation entry points (CPU).

Every call here is refused: nothing is launched, with or without a GPU.
"""
import ctypes

import pytest

from nvfp4_weight_only_02_gb300 import binding, build

P = ctypes.c_void_p
good, bad = P(4096), P(4096 + 4)   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def test_tiled_scale_bytes(lib):
    f = lib.nvfp4_tiled_scale_bytes
    assert f(1, 32, 0) == 512 and f(128, 128, 0) == 512 and f(129, 128, 0) == 1024 and f(128, 160, 0) == 1024
    assert f(1, 16, 1) == 512 and f(128, 64, 1) == 512 and f(300, 80, 1) == 3 * 2 * 512
    assert f(1, 16, 0) == 0 and f(0, 32, 0) == 0 and f(1, 0, 0) == 0 and f(1, 32, 2) == 0 and f(-1, 32, 0) == 0
    assert f(1 << 31, 32, 0) == 0


def test_tile_scales(lib):
    f = lib.nvfp4_tile_scales
    assert f(None, 4, 32, 0, good, None) == binding.ERR_INVALID_ARG
    assert f(good, 4, 32, 2, good, None) == binding.ERR_INVALID_ARG
    assert f(good, 4, 48, 0, good, None) == binding.ERR_SHAPE
    assert f(bad, 4, 32, 0, good, None) == binding.ERR_ALIGNMENT


def test_mx_quantize(lib):
    f = lambda x=good, dt=0, rows=8, cols=64, ld=64, c=good, s=good, v=None, ct=None, st=None, vt=None: \
        lib.nvfp4_mx_quantize(x, dt, rows, cols, ld, c, s, v, ct, st, vt, None)  # noqa: E731
    assert f(x=None) == binding.ERR_INVALID_ARG
    assert f(dt=2) == binding.ERR_INVALID_ARG
    assert f(c=None, s=None) == binding.ERR_INVALID_ARG           # no output
    assert f(s=None) == binding.ERR_INVALID_ARG                   # codes without scales
    assert f(ct=good) == binding.ERR_INVALID_ARG
    for kw in (dict(rows=0), dict(cols=0), dict(cols=48), dict(ld=32), dict(rows=(1 << 30) + 1),
               dict(rows=1 << 30, cols=1 << 20, ld=1 << 20)):
        assert f(**kw) == binding.ERR_SHAPE, kw
    for kw in (dict(x=bad), dict(ld=68), dict(dt=1, ld=66), dict(c=bad), dict(s=bad), dict(v=bad),
               dict(ct=bad, st=good), dict(ct=good, st=bad), dict(vt=bad)):
        assert f(**kw) == binding.ERR_ALIGNMENT, kw


def test_mx_dequantize(lib):
    f = lib.nvfp4_mx_dequantize
    assert f(good, None, 4, 32, good, 0, None) == binding.ERR_INVALID_ARG
    assert f(good, good, 4, 32, good, 3, None) == binding.ERR_INVALID_ARG
    assert f(good, good, 4, 40, good, 0, None) == binding.ERR_SHAPE
    assert f(good, good, 4, 32, bad, 0, None) == binding.ERR_ALIGNMENT


def test_w4a4_gemm(lib):
    f = lambda fmt=0, ac=good, asc=good, at=None, wc=good, wsc=good, wt=None, M=4, N=8, K=64, y=good, dt=0, ws=good, \
        n=1 << 30: lib.nvfp4_w4a4_gemm(fmt, ac, asc, at, wc, wsc, wt, M, N, K, y, dt, ws, n, None)  # noqa: E731
    for kw in (dict(fmt=2), dict(ac=None), dict(asc=None), dict(wc=None), dict(wsc=None), dict(y=None), dict(ws=None),
               dict(dt=5)):
        assert f(**kw) == binding.ERR_INVALID_ARG, kw
    for kw in (dict(M=0), dict(N=0), dict(K=0), dict(K=16), dict(fmt=1, K=48), dict(M=(1 << 30) + 1),
               dict(M=1 << 30, N=1 << 30)):
        assert f(**kw) == binding.ERR_SHAPE, kw
    for kw in (dict(ac=bad), dict(asc=bad), dict(at=bad), dict(wc=bad), dict(wsc=bad), dict(wt=bad), dict(y=bad),
               dict(ws=bad)):
        assert f(**kw) == binding.ERR_ALIGNMENT, kw
    need = lib.nvfp4_w4a4_workspace_bytes(4, 8, 64)
    assert need >= 256 and f(n=need - 1) == binding.ERR_WORKSPACE
    assert lib.nvfp4_w4a4_workspace_bytes(4, 8, 63) == 0


def test_mx_linear(lib):
    f = lambda x=good, dt=0, ld=64, M=4, N=8, K=64, wc=good, wsc=good, y=good, ydt=0, ws=good, n=1 << 30: \
        lib.nvfp4_mx_linear(x, dt, ld, M, N, K, wc, wsc, y, ydt, ws, n, None)  # noqa: E731
    for kw in (dict(x=None), dict(wc=None), dict(wsc=None), dict(y=None), dict(ws=None), dict(dt=2), dict(ydt=2)):
        assert f(**kw) == binding.ERR_INVALID_ARG, kw
    for kw in (dict(ld=32), dict(M=0), dict(N=0), dict(K=80, ld=80)):
        assert f(**kw) == binding.ERR_SHAPE, kw
    for kw in (dict(x=bad), dict(ld=68), dict(wc=bad), dict(wsc=bad), dict(y=bad), dict(ws=bad)):
        assert f(**kw) == binding.ERR_ALIGNMENT, kw
    need = lib.nvfp4_mx_linear_workspace_bytes(4, 8, 64)
    assert f(n=need - 1) == binding.ERR_WORKSPACE
    assert lib.nvfp4_mx_linear_workspace_bytes(0, 8, 64) == 0


def test_mx_linear_backward(lib):
    f = lambda dy=good, dt=0, ld=32, M=5, N=32, K=64, xc=good, xs=good, wc=good, wsc=good, dx=good, dxt=0, dw=good, \
        dwt=1, ws=good, n=1 << 30: lib.nvfp4_mx_linear_backward(dy, dt, ld, M, N, K, xc, xs, wc, wsc, dx, dxt, dw, dwt,
                                                                 ws, n, None)  # noqa: E731
    for kw in (dict(dy=None), dict(ws=None), dict(dx=None, dw=None), dict(xc=None), dict(xs=None), dict(wc=None),
               dict(wsc=None), dict(dt=2), dict(dxt=2), dict(dwt=2)):
        assert f(**kw) == binding.ERR_INVALID_ARG, kw
    for kw in (dict(M=0), dict(N=40, ld=40), dict(K=72), dict(ld=16)):
        assert f(**kw) == binding.ERR_SHAPE, kw
    for kw in (dict(dy=bad), dict(ld=36), dict(xc=bad), dict(xs=bad), dict(wc=bad), dict(wsc=bad), dict(dx=bad),
               dict(dw=bad), dict(ws=bad)):
        assert f(**kw) == binding.ERR_ALIGNMENT, kw
    need = lib.nvfp4_mx_linear_backward_workspace_bytes(5, 32, 64)
    assert f(n=need - 1) == binding.ERR_WORKSPACE
    assert lib.nvfp4_mx_linear_backward_workspace_bytes(5, 40, 64) == 0


def test_distill_topk(lib):
    f = lambda z=good, dt=0, T=2, V=100, ld=100, i=good, ib=4, t=good, tdt=0, k=4, tau=1.0, rest=0, w=None, g=None, \
        gn=0, loss=good, dz=good, lddz=100, ws=None, n=0: lib.nvfp4_distill_topk(
            z, dt, T, V, ld, i, ib, t, tdt, k, tau, rest, w, g, gn, loss, dz, lddz, ws, n, None)  # noqa: E731
    inf, nan = float("inf"), float("nan")
    for kw in (dict(z=None), dict(i=None), dict(t=None), dict(loss=None, dz=None), dict(dt=2), dict(tdt=2), dict(ib=2),
               dict(tau=0.0), dict(tau=-1.0), dict(tau=inf), dict(tau=nan), dict(tau=1e-40), dict(dz=None, g=good, gn=1)):
        assert f(**kw) == binding.ERR_INVALID_ARG, kw
    for kw in (dict(T=0), dict(V=0), dict(k=0), dict(k=1025), dict(ld=99), dict(lddz=99), dict(g=good, gn=3),
               dict(V=819137, ld=819137, lddz=819137), dict(dt=1, V=409569, ld=409569, lddz=409569)):
        assert f(**kw) == binding.ERR_SHAPE, kw
    for kw in (dict(z=bad), dict(i=bad), dict(t=bad), dict(w=bad), dict(g=bad, gn=1), dict(loss=bad), dict(dz=bad),
               dict(ws=bad, n=256)):
        assert f(**kw) == binding.ERR_ALIGNMENT, kw
    assert f(ws=good, n=255) == binding.ERR_WORKSPACE
    assert "range" in binding.status_string(binding.ERR_INDEX)
