"""Out-of-bounds writes of the 4-bit and distillation calls: every output buffer and workspace sits between guard bytes
of a fixed pattern, and columns between the rows of a strided gradient keep theirs."""
import pytest
import torch

from tests.test_gpu_guards import Guarded

pytestmark = pytest.mark.gpu

bf16, f32, u8 = torch.bfloat16, torch.float32, torch.uint8


def _call(nv, name, *args):
    nv._call(name, *[a.buf.data_ptr() + 4096 if isinstance(a, Guarded) else a for a in args], nv._raw_stream())


def _intact(*guarded):
    for g in guarded:
        assert g is None or g.intact()


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (5, 96), (33, 160), (129, 224), (300, 1056), (64, 3584)])
def test_quantiser(nv, rows, cols, dtype):
    x = torch.randn(rows, cols, device="cuda").to(dtype)
    code = nv.OUT_BF16 if dtype == bf16 else nv.OUT_FP32
    r32 = (rows + 31) // 32 * 32
    for fwd, back in ((1, 1), (1, 0), (0, 1)):
        q = Guarded(rows * cols // 2) if fwd else None
        s = Guarded(nv.nvfp4_tiled_scale_bytes(rows, cols, nv.FORMAT_MXFP4)) if fwd else None
        v = Guarded(rows * cols * 2) if fwd else None
        qt = Guarded(cols * r32 // 2) if back else None
        st = Guarded(nv.nvfp4_tiled_scale_bytes(cols, r32, nv.FORMAT_MXFP4)) if back else None
        vt = Guarded(rows * cols * 2) if back else None
        _call(nv, "nvfp4_mx_quantize", x.data_ptr(), code, rows, cols, cols, q, s, v, qt, st, vt)
        _intact(q, s, v, qt, st, vt)
        if fwd:
            for es, ocode in ((4, nv.OUT_FP32), (2, nv.OUT_BF16)):
                out = Guarded(rows * cols * es)
                _call(nv, "nvfp4_mx_dequantize", q, s, rows, cols, out, ocode)
                _intact(out, q, s)
    for fmt, block in ((nv.FORMAT_MXFP4, 32), (nv.FORMAT_NVFP4, 16)):
        plain = torch.randint(0, 100, (rows, cols // block), dtype=u8, device="cuda")
        tiled = Guarded(nv.nvfp4_tiled_scale_bytes(rows, cols, fmt))
        _call(nv, "nvfp4_tile_scales", plain.data_ptr(), rows, cols, fmt, tiled)
        _intact(tiled)


@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (3, 7, 64), (17, 130, 160), (64, 200, 544), (70, 130, 4128), (129, 255, 288),
                                   (300, 1001, 512), (257, 520, 96), (1000, 2312, 256)])
def test_products_and_layer(nv, M, N, K):
    g = torch.Generator("cuda").manual_seed(M + N)
    x = torch.randn(M, K, device="cuda", generator=g)
    w = torch.randn(N, K, device="cuda", generator=g)
    xq, wq = nv.mx_quantize(x).row, nv.mx_quantize(w).row
    one = torch.ones(4, device="cuda")
    nvx = [torch.randint(0, 256, (r, K // 2), dtype=u8, device="cuda") for r in (M, N)]
    nvs = [torch.full((nv.nvfp4_tiled_scale_bytes(r, K, nv.FORMAT_NVFP4),), 0x38, dtype=u8, device="cuda") for r in (M, N)]
    for es, code in ((4, nv.OUT_FP32), (2, nv.OUT_BF16)):
        y = Guarded(M * N * es)
        ws = Guarded(nv.nvfp4_w4a4_workspace_bytes(M, N, K), fill=0)
        lin = Guarded(nv.nvfp4_mx_linear_workspace_bytes(M, N, K), fill=0)
        for _ in range(2):
            _call(nv, "nvfp4_w4a4_gemm", nv.FORMAT_MXFP4, *xq.addresses(), None, *wq.addresses(), None, M, N, K, y, code,
                  ws, ws.n)
            _intact(y, ws)
            _call(nv, "nvfp4_w4a4_gemm", nv.FORMAT_NVFP4, nvx[0].data_ptr(), nvs[0].data_ptr(), one.data_ptr(),
                  nvx[1].data_ptr(), nvs[1].data_ptr(), one.data_ptr(), M, N, K, y, code, ws, ws.n)
            _intact(y, ws)
            for t, xcode in ((x, nv.OUT_FP32), (x.bfloat16(), nv.OUT_BF16)):
                _call(nv, "nvfp4_mx_linear", t.data_ptr(), xcode, K, M, N, K, *wq.addresses(), y, code, lin, lin.n)
                _intact(y, lin)


@pytest.mark.parametrize("M,N,K", [(1, 32, 32), (5, 64, 96), (100, 288, 160), (333, 1056, 512)])
def test_backward(nv, M, N, K):
    g = torch.Generator("cuda").manual_seed(M)
    xq = nv.mx_quantize(torch.randn(M, K, device="cuda", generator=g), rowwise=False, colwise=True).col
    wq = nv.mx_quantize(torch.randn(N, K, device="cuda", generator=g), rowwise=False, colwise=True).col
    dy = torch.randn(M, N, device="cuda", generator=g)
    for es, code in ((4, nv.OUT_FP32), (2, nv.OUT_BF16)):
        dx, dw = Guarded(M * K * es), Guarded(N * K * es)
        ws = Guarded(nv.nvfp4_mx_linear_backward_workspace_bytes(M, N, K), fill=0)
        _call(nv, "nvfp4_mx_linear_backward", dy.data_ptr(), nv.OUT_FP32, N, M, N, K, *xq.addresses(), *wq.addresses(),
              dx, code, dw, code, ws, ws.n)
        _intact(dx, dw, ws)


@pytest.mark.parametrize("tail", [0, 1])
@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("T,V,k,pad", [(1, 1, 1, 0), (3, 9, 4, 0), (5, 1001, 20, 6), (2, 50001, 700, 3), (160, 60001, 16, 7),
                                       (310, 50000, 30, 0)])
def test_distillation(nv, T, V, k, pad, dtype, tail):
    g = torch.Generator("cuda").manual_seed(V)
    es, code = (2, nv.OUT_BF16) if dtype == bf16 else (4, nv.OUT_FP32)
    z = torch.randn(T, V, device="cuda", generator=g).to(dtype)
    val, idx = torch.topk(torch.randn(T, V, device="cuda", generator=g), k)
    val = torch.log_softmax(val, 1) - 0.5
    w = torch.ones(T, device="cuda")
    w[T // 2] = 0.0
    ld = V + pad
    for with_dz in (True, False):
        loss, ws = Guarded(4 * T), Guarded(256, fill=0)
        dz = Guarded(T * ld * es) if with_dz else None
        _call(nv, "nvfp4_distill_topk", z.data_ptr(), code, T, V, V, idx.data_ptr(), 8, val.data_ptr(), nv.OUT_FP32, k, 1.0,
              tail, w.data_ptr(), None, 0, loss, dz, ld, ws, ws.n)
        _intact(loss, dz, ws)
        if with_dz and pad:
            assert bool((dz.view(u8, (T, ld * es))[:, V * es:] == 0xA5).all())
