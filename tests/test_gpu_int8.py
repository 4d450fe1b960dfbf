"""8-bit integers: quantiser, product and layer against 64-bit definitions."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _quant64(x):
    """(codes, amax), float64."""
    x = x.double()
    amax = x.abs().amax(1, keepdim=True)
    return torch.where(amax > 0, torch.round(x * 127 / amax), 0.0), amax


@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 48), (129, 4096), (40, 18944), (2, 131072), (5000, 176)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantise(nv, rows, cols, dtype):
    g = _gen(rows + cols)
    x = torch.randn(rows, cols + 16, device="cuda", generator=g)
    # magnitudes over the whole range; the last rows are integers over an amax of 127 or 254, ties among them
    x *= torch.exp2(torch.randint(-120, 120, (rows, 1), device="cuda", generator=g).float())
    x[-1] = torch.randint(-253, 254, (cols + 16,), device="cuda", generator=g).float()
    x[-1, 0] = 254
    x = x.to(dtype)[:, :cols] if rows > 1 else x.to(dtype)[:, :cols].contiguous()
    q = nv.int8_quantize(x)
    codes, amax = _quant64(x)
    assert torch.equal(q.codes.double(), codes)
    assert ((q.scales.double() - amax[:, 0] / 127).abs() <= 2.0 ** -24 * amax[:, 0] / 127).all()


def test_rows_without_a_scale(nv):
    for dtype in (BF, F32):
        x = torch.ones(5, 32, device="cuda")
        x[1], x[2, 3], x[3, 4] = 0, float("nan"), -float("inf")
        x[4] = 2.0 ** -130            # subnormal: the reciprocal leaves FP32
        x = x.to(dtype)
        q = nv.int8_quantize(x)
        assert q.codes[0].tolist() == [127] * 32 and q.codes[1:4].abs().max() == 0 and q.codes[4].tolist() == [127] * 32
        assert q.scales[1] == 0 and q.scales[2].isnan() and q.scales[3].isnan()
        y = nv.int8_linear(x, nv.int8_quantize(torch.ones(3, 32, device="cuda")))
        assert (y[1] == 0).all() and y[2:4].isnan().all() and not y[0].isnan().any()


SIZES = [  # M, N, K
    (1, 1, 16), (1, 300, 3584), (2, 129, 48), (16, 640, 18944), (17, 257, 400), (33, 1000, 1040), (64, 128, 128),
    (100, 3584, 4096), (128, 96, 2000), (129, 77, 272), (200, 20000, 144), (500, 300, 6000), (777, 1055, 800), (2048, 512, 512),
    (300, 10000, 256),
]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype,out", [(BF, BF), (F32, F32)])
def test_layer(nv, M, N, K, dtype, out):
    g = _gen(M + N + K)
    x = torch.randn(M, K + 8, device="cuda", generator=g).to(dtype)[:, :K]
    if M == 1:
        x = x.contiguous()
    w = nv.int8_quantize((torch.randn(N, K, device="cuda", generator=g) * 0.05).to(dtype))
    ws = nv.new_workspace(nv.nvfp4_int8_linear_workspace_bytes(M, N, K))
    y = nv.int8_linear(x, w, out_dtype=out, workspace=ws)
    codes, amax = _quant64(x)
    sums = codes @ w.codes.double().t()
    assert sums.abs().max() < 2 ** 24       # exact in FP32, whatever the order
    want = sums * (amax / 127) * w.scales.double()
    # the token's scale and two products are rounded, then the result
    assert ((y.double() - want).abs() <= (3 * 2.0 ** -24 + HALF_STEP[out]) * 1.01 * want.abs()).all()
    # the quantiser and the product apart, bit for bit
    assert torch.equal(nv.int8_gemm(nv.int8_quantize(x), w, out_dtype=out, workspace=ws), y)
    assert nv.nvfp4_get_device_status(ws) == nv.OK


@pytest.mark.parametrize("M", [1, 40, 100, 300])
def test_largest_sums(nv, M):
    """All products 127^2, or of -128: sums beyond 2^24 are FP32 sums of exact terms, an instruction adds 16."""
    N, K = 260, 131072 if M < 300 else 8192
    a = torch.full((M, K), 127, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), 127, dtype=torch.int8, device="cuda")
    w[1], w[2, ::2] = -128, -127
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    y = nv.int8_gemm(nv.Int8Matrix(a, one(M)), nv.Int8Matrix(w, one(N))).double()
    # every addition is off by a step (2^-23) of the sum at most
    tol = 127 * 128 * K * (K / 16 + 8) * 2.0 ** -23
    assert (y[:, 0] - 127 * 127 * K).abs().max() <= tol and (y[:, 1] + 127 * 128 * K).abs().max() <= tol
    assert (y[:, 2] == 0).all() and (y[:, 3:] == y[:, :1]).all()


@pytest.mark.parametrize("M,N,K", [(1, 500, 3584), (1, 18944, 3584), (4, 300, 4096), (16, 300, 1024), (3, 200, 18944)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_ties(nv, M, N, K, dtype):
    """A largest magnitude of 254 / 64 makes ties of all odd multiples of 1 / 64: also where the product's kernel
    quantises the tokens itself (few of them), whose warps part at ties."""
    g = _gen(M + K)
    x = torch.randint(-200, 201, (M, K), device="cuda", generator=g).float() / 64
    x[:, 5] = 254 / 64
    x[:, ::3] = 0.3
    w = nv.int8_quantize(torch.randn(N, K, device="cuda", generator=g))
    x = x.to(dtype)
    a = nv.int8_quantize(x)
    assert torch.equal(a.codes.double(), _quant64(x)[0])
    for _ in range(3):
        assert torch.equal(nv.int8_linear(x, w), nv.int8_gemm(a, w))


def test_layers_behind_one_another(nv):
    """Launches overlap: each call's tokens are what the call before has just written."""
    g = _gen(7)
    for M, K in ((1, 1024), (8, 2048), (40, 512), (300, 512)):
        ws_ = [nv.int8_quantize(torch.randn(K, K, device="cuda", generator=g) / K ** 0.5) for _ in range(3)]
        x = torch.randn(M, K, device="cuda", generator=g)
        space = nv.new_workspace(nv.nvfp4_int8_linear_workspace_bytes(M, K, K))
        want, t = [], x
        for i in range(12):
            t = nv.int8_linear(t, ws_[i % 3])
            torch.cuda.synchronize()
            want.append(t)
        buf = [x.clone(), torch.empty_like(x)]
        torch.cuda.synchronize()
        for i in range(12):
            a, b = buf[i % 2], buf[1 - i % 2]
            nv._call("nvfp4_int8_linear", a.data_ptr(), nv.OUT_FP32, K, M, K, K, ws_[i % 3].codes.data_ptr(),
                     ws_[i % 3].scales.data_ptr(), b.data_ptr(), nv.OUT_FP32, space.data_ptr(), space.numel(),
                     nv._raw_stream())
        assert torch.equal(buf[0], want[11]) and torch.equal(buf[1], want[10])
        assert nv.nvfp4_get_device_status(space) == nv.OK


@pytest.mark.parametrize("M,N,K", [(1, 18944, 3584), (10, 3584, 18944), (40, 18944, 3584), (100, 18944, 3584)])
def test_weights_that_come_from_memory(nv, M, N, K):
    """Weights beyond L2 in turn: stages land late and out of order."""
    g = _gen(M)
    w = [nv.int8_quantize(torch.randn(N, K, device="cuda", generator=g)) for _ in range(4)]
    x = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    a = nv.int8_quantize(x)
    codes = a.codes.double()
    want = [(codes @ q.codes.double().t()) * a.scales.double()[:, None] * q.scales.double() for q in w]
    ws = nv.new_workspace(nv.nvfp4_int8_linear_workspace_bytes(M, N, K))
    for _ in range(5):
        ys = [nv.int8_linear(x, q, workspace=ws) for q in w]
        for y, r in zip(ys, want):
            # sums are exact; two products are rounded
            assert ((y.double() - r).abs() <= 3.1 * 2.0 ** -24 * r.abs()).all()
