"""W4A4 product and MX layer on the GPU against 64-bit products of the decoded operands.

Tolerance (fixed before the first run): products of two codes and their scales are exact in FP32, so the error is that
of an FP32 sum of K terms in some order: |err| <= (K + 64) 2^-23 sum_k |a||w| per element, plus two roundings for the
tensor scales (inside the 64).  A bf16 output is the rounding of the same FP32 result, bit for bit.
"""
import numpy as np
import pytest
import torch

from tests import fp4_reference as ref

pytestmark = pytest.mark.gpu


def _operand(nv, fmt, rows, cols, seed, span=6):
    """Random codes and scales; returns (operand, float64 values without the tensor scale, tensor scale)."""
    g = torch.Generator().manual_seed(seed)
    packed = torch.randint(0, 256, (rows, cols // 2), dtype=torch.uint8, generator=g)
    grid = ref.GRID[ref.unpack(packed.numpy()) & 7] * np.where(ref.unpack(packed.numpy()) & 8, -1.0, 1.0)
    if fmt == "mx":
        byte = torch.randint(127 - span, 128 + span, (rows, cols // 32), dtype=torch.uint8, generator=g)
        s = np.exp2(byte.numpy().astype(np.float64) - 127)
        op = nv.MxOperand.from_row_major(packed.cuda(), byte.cuda())
        return op, (grid.reshape(rows, -1, 32) * s[..., None]).reshape(rows, cols), 1.0
    byte = torch.randint(0, 127, (rows, cols // 16), dtype=torch.uint8, generator=g)
    s = byte.view(torch.float8_e4m3fn).to(torch.float64).numpy()
    ts = 0.37 + seed % 5
    op = nv.Nvfp4Operand.from_row_major(packed.cuda(), byte.cuda(), torch.tensor([ts], dtype=torch.float32).cuda())
    return op, (grid.reshape(rows, -1, 16) * s[..., None]).reshape(rows, cols), float(np.float32(ts))


def _check_product(y, a, w, scale, K):
    want = (a @ w.T) * scale
    bound = (K + 64) * 2.0 ** -23 * (np.abs(a) @ np.abs(w).T) * abs(scale) + 1e-38
    err = np.abs(ref.to64(y) - want)
    assert y.dtype == torch.float32 and (err <= bound).all(), (err / bound).max()


SHAPES = [
    # M, N, K
    (16, 128, 256), (1, 128, 256), (1, 1, 32), (3, 7, 64), (16, 100, 96), (5, 129, 160), (8, 300, 288), (16, 256, 512),
    (2, 1000, 3584), (16, 130, 18944), (17, 128, 128), (32, 200, 1056), (33, 256, 256), (64, 136, 2048),
    (65, 128, 256), (100, 77, 544), (128, 384, 1024), (129, 128, 256), (200, 513, 800), (256, 256, 512),
    (257, 255, 1088), (300, 40, 4096), (511, 1024, 96), (700, 700, 704), (1024, 2048, 512), (31, 4001, 640),
]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(nv, fmt, M, N, K):
    a, a64, sa = _operand(nv, fmt, M, K, M + K)
    w, w64, sw = _operand(nv, fmt, N, K, N + 3 * K)
    y = nv.w4a4_gemm(a, w)
    _check_product(y, a64, w64, sa * sw, K)
    yb = nv.w4a4_gemm(a, w, out_dtype=torch.bfloat16)
    assert torch.equal(yb, y.to(torch.bfloat16))
    assert torch.equal(y, nv.w4a4_gemm(a, w))


@pytest.mark.parametrize("M", [1, 16, 48, 130, 400])
def test_every_code_and_scale(nv, M):
    """One-hot rows of A pick single elements of W: every code under every E8M0 exponent that FP32 can hold."""
    N, K = 256, 512
    g = torch.Generator().manual_seed(M)
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, generator=g)
    byte = torch.randint(0, 253, (N, K // 32), dtype=torch.uint8, generator=g)
    w = nv.MxOperand.from_row_major(codes.cuda(), byte.cuda())
    w64 = ref.mx_values(ref.unpack(codes.numpy()), byte.numpy())
    pick = torch.randint(0, K, (M,), generator=g)
    x = torch.zeros(M, K)
    x[torch.arange(M), pick] = 1.0
    y = nv.mx_linear(x.cuda(), w)
    want = w64[:, pick.numpy()].T
    normal = np.abs(want) >= 2.0 ** -126          # below, the tensor core may flush
    assert np.array_equal(ref.to64(y)[normal], want[normal])
    assert (np.abs(ref.to64(y) - want) <= 2.0 ** -126).all()


def test_a_nan_block_reaches_its_row_only(nv):
    for M in (4, 40, 300):
        x = torch.randn(M, 512, generator=torch.Generator().manual_seed(M)).cuda()
        w, w64, _ = _operand(nv, "mx", 200, 512, 7)
        clean = nv.mx_linear(x, w)
        x[2, 100] = float("nan")
        y = nv.mx_linear(x, w)
        assert torch.isnan(y[2]).all()
        keep = torch.arange(M) != 2
        assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(1, 512, 3584), (7, 300, 1024), (16, 1000, 512), (20, 130, 96), (130, 256, 2048),
                                   (600, 384, 544)])
def test_linear(nv, M, N, K, dtype):
    g = torch.Generator().manual_seed(M)
    big = torch.randn(M, K + 64, generator=g).to(dtype).cuda()
    w = nv.mx_quantize((torch.randn(N, K, generator=g) * 0.02).cuda()).row
    w64 = ref.to64(w.dequantize())
    for x in (big[:, 32:32 + K], big[:, :K].contiguous()):
        y = nv.mx_linear(x, w)
        _check_product(y, ref.mx_round(ref.to64(x)), w64, 1.0, K)
        assert torch.equal(y, nv.w4a4_gemm(nv.mx_quantize(x).row, w))
        assert torch.equal(nv.mx_linear(x, w, out_dtype=torch.bfloat16), y.to(torch.bfloat16))


def test_linear_many_times_with_one_workspace_and_stream(nv):
    g = torch.Generator().manual_seed(1)
    w = nv.mx_quantize(torch.randn(640, 512, generator=g).cuda()).row
    xs = [torch.randn(m, 512, generator=g).cuda() for m in (1, 40, 3, 200, 16)]
    alone = [nv.mx_linear(x, w) for x in xs]
    ws = nv.new_workspace(max(nv.nvfp4_mx_linear_workspace_bytes(x.shape[0], 640, 512) for x in xs))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(20):
            got = [nv.mx_linear(x, w, workspace=ws) for x in xs]
        assert nv.nvfp4_get_device_status(ws) == nv.OK
    s.synchronize()
    for a, b in zip(alone, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(1, 32, 32), (5, 64, 96), (32, 128, 256), (100, 288, 160), (333, 1056, 512),
                                   (640, 512, 1024)])
def test_backward(nv, M, N, K, dtype):
    g = torch.Generator().manual_seed(M + N)
    x = torch.randn(M, K, generator=g).to(dtype).cuda()
    w = (torch.randn(N, K, generator=g) * 0.02).to(dtype).cuda()
    dy = (torch.randn(M, N + 32, generator=g) * 1e-3).to(dtype).cuda()[:, :N]
    xq, wq = nv.mx_quantize(x, colwise=True), nv.mx_quantize(w, colwise=True)
    dx, dw = nv.mx_linear_backward(dy, xq.col, wq.col)
    cols = lambda t: ref.mx_round(np.ascontiguousarray(ref.pad_rows(ref.to64(t)).T))  # noqa: E731
    _check_product(dx, ref.mx_round(ref.to64(dy)), cols(w), 1.0, N)
    _check_product(dw, cols(dy), cols(x), 1.0, (M + 31) // 32 * 32)
    only_x, none = nv.mx_linear_backward(dy, None, wq.col, dx_dtype=torch.bfloat16)
    none2, only_w = nv.mx_linear_backward(dy, xq.col, None, dw_dtype=torch.bfloat16)
    assert none is None and none2 is None
    assert torch.equal(only_x, dx.bfloat16()) and torch.equal(only_w, dw.bfloat16())


def test_backward_against_differences(nv):
    """Inputs that MXFP4 holds exactly in both directions (grid values with a 4 in every block): the layer is then
    the bilinear L = <dY, X W^T> itself, and L(X + D) - L(X) = <dX, D> has no error but the FP32 sums'."""
    M, N, K = 96, 160, 224
    rng = np.random.default_rng(5)

    def exact(rows, cols):
        v = rng.choice(ref.GRID[:7], (rows, cols)) * rng.choice([-1.0, 1.0], (rows, cols))
        i, j = np.meshgrid(np.arange(rows), np.arange(cols), indexing="ij")
        v[(i + j) % 32 == 0] = 4.0
        assert np.array_equal(ref.mx_round(v), v) and np.array_equal(ref.mx_round(np.ascontiguousarray(v.T)).T, v)
        return v

    x, w, dy = exact(M, K), exact(N, K), exact(M, N)
    dev = lambda v: torch.from_numpy(v).to(torch.bfloat16).cuda()  # noqa: E731
    xq, wq = nv.mx_quantize(dev(x), colwise=True), nv.mx_quantize(dev(w), colwise=True)
    dx, dw = nv.mx_linear_backward(dev(dy), xq.col, wq.col)
    L = lambda a, b: (dy * (a @ b.T)).sum()  # noqa: E731
    for seed in range(4):
        r = np.random.default_rng(seed)
        D, E = r.standard_normal((M, K)), r.standard_normal((N, K))
        bx = (N + 64) * 2.0 ** -23 * (np.abs(D) * (np.abs(dy) @ np.abs(w))).sum()
        bw = (M + 64) * 2.0 ** -23 * (np.abs(E) * (np.abs(dy).T @ np.abs(x))).sum()
        assert abs(L(x + D, w) - L(x, w) - (ref.to64(dx) * D).sum()) <= bx + 1e-7
        assert abs(L(x, w + E) - L(x, w) - (ref.to64(dw) * E).sum()) <= bw + 1e-7


def test_nvfp4_weight_and_activation(nv):
    """The library's own NVFP4 quantiser feeds the product: same result as its dequantised matrices give."""
    g = torch.Generator().manual_seed(3)
    for M in (3, 96, 260):
        x = nv.quantize(torch.randn(M, 1024, generator=g).bfloat16().cuda())
        w = nv.quantize((torch.randn(384, 1024, generator=g) * 0.02).bfloat16().cuda())
        y = nv.w4a4_gemm(nv.Nvfp4Operand.from_weight(x), nv.Nvfp4Operand.from_weight(w))
        one = torch.ones(1, device="cuda")
        a64 = ref.to64(nv.dequantize(nv.QuantizedWeight(x.codes, x.scales, one)))
        w64 = ref.to64(nv.dequantize(nv.QuantizedWeight(w.codes, w.scales, one)))
        _check_product(y, a64, w64, float(x.tensor_scale) * float(w.tensor_scale), 1024)


def test_tensor_scales_whose_product_underflows(nv):
    """A row of A with a single non-zero code gives exact FP32 sums; 2^-80 and 2^-60 are applied one after the
    other, so nothing is lost but what FP32's subnormal spacing (2^-149) cannot hold."""
    w, w64, _ = _operand(nv, "nv", 128, 256, 2)
    w.tensor_scale.fill_(2.0 ** -60)
    codes = np.zeros((8, 256), np.uint8)
    codes[np.arange(8), 30 * np.arange(8)] = 7                                          # 6.0
    byte = torch.full((8, 16), 0x7E, dtype=torch.uint8)                                 # 448
    a = nv.Nvfp4Operand.from_row_major(torch.from_numpy(ref.pack(codes)).cuda(), byte.cuda(),
                                       torch.tensor([2.0 ** -80], device="cuda"))
    y = nv.w4a4_gemm(a, w)
    want = 6.0 * 448.0 * w64[:, 30 * np.arange(8)].T * 2.0 ** -140
    assert (np.abs(ref.to64(y) - want) <= 2.0 ** -149).all() and (np.abs(want) > 2.0 ** -140).any()


def test_large_outputs_beyond_32_bits(nv):
    M, N, K = 40000, 65536, 32
    a, a64, _ = _operand(nv, "mx", M, K, 1)
    w, w64, _ = _operand(nv, "mx", N, K, 2)
    y = nv.w4a4_gemm(a, w, out_dtype=torch.bfloat16)
    for rows, cols in ((slice(0, 70), slice(0, 300)), (slice(M - 70, M), slice(N - 300, N))):
        want = a64[rows] @ w64[cols].T
        assert (np.abs(ref.to64(y[rows, cols]) - want) <= 2.0 ** -8 * np.abs(want) + 1e-5).all()


def test_refusals(nv):
    a, _, _ = _operand(nv, "mx", 16, 64, 1)
    w, _, _ = _operand(nv, "mx", 32, 64, 2)
    n, _, _ = _operand(nv, "nv", 32, 64, 2)
    k, _, _ = _operand(nv, "mx", 32, 96, 2)
    x = torch.zeros(16, 64, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: nv.w4a4_gemm(a, n), lambda: nv.w4a4_gemm(a, k),
                 lambda: nv.w4a4_gemm(a, w, out_dtype=torch.float16), lambda: nv.mx_linear(x, n),
                 lambda: nv.mx_linear(x, k), lambda: nv.mx_linear(x.half(), w), lambda: nv.mx_linear(x.t(), w),
                 lambda: nv.mx_linear_backward(x, None, None), lambda: nv.mx_linear_backward(x, a, w)):
        with pytest.raises(ValueError):
            call()
    small = torch.zeros(128, dtype=torch.uint8, device="cuda")
    for call in (lambda: nv.w4a4_gemm(a, w, workspace=small), lambda: nv.mx_linear(x, w, workspace=small)):
        with pytest.raises(nv.NVFP4Error) as e:
            call()
        assert e.value.status == nv.ERR_WORKSPACE
    with pytest.raises(nv.NVFP4Error) as e:
        nv.mx_linear(torch.zeros(16, 80, dtype=torch.bfloat16, device="cuda")[:, 4:68], w)
    assert e.value.status == nv.ERR_ALIGNMENT


LONG = [(70, 130, 4128), (129, 513, 8192), (300, 520, 18944), (1000, 1030, 4352), (260, 3584, 6144), (65, 4000, 16384)]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M,N,K", LONG)
def test_long_contractions_of_few_tiles(nv, fmt, M, N, K):
    a, a64, sa = _operand(nv, fmt, M, K, M + K)
    w, w64, sw = _operand(nv, fmt, N, K, N + 3 * K)
    y = nv.w4a4_gemm(a, w)
    _check_product(y, a64, w64, sa * sw, K)
    assert torch.equal(nv.w4a4_gemm(a, w, out_dtype=torch.bfloat16), y.to(torch.bfloat16))


@pytest.mark.parametrize("K", [32, 96, 512])
@pytest.mark.parametrize("M,N", [(2048, 8192), (5000, 5408), (300, 40000), (16384, 2312), (1111, 12345)])
def test_many_tiles_of_short_contractions(nv, M, N, K):
    """Tiles that follow one another quickly: every element of both output types against the definition, in FP64 on
    the device (the operands' values come from the dequantiser, which has its own test)."""
    g = torch.Generator("cuda").manual_seed(M)
    a = nv.mx_quantize(torch.randn(M, K, device="cuda", generator=g)).row
    w = nv.mx_quantize(torch.randn(N, K, device="cuda", generator=g)).row
    a64, w64 = a.dequantize().double(), w.dequantize().double()
    want, bound = a64 @ w64.t(), (K + 64) * 2.0 ** -23 * (a64.abs() @ w64.abs().t()) + 1e-38
    y = nv.w4a4_gemm(a, w)
    assert ((y.double() - want).abs() <= bound).all()
    assert torch.equal(nv.w4a4_gemm(a, w, out_dtype=torch.bfloat16), y.bfloat16())


def test_one_workspace_for_calls_of_all_sizes(nv):
    """The counters are at zero after every call, whatever its size, and results do not depend on the calls before."""
    sizes = [(300, 520, 18944), (3, 512, 4096), (129, 513, 8192), (64, 256, 512), (700, 700, 704), (1, 128, 8192)]
    g = torch.Generator().manual_seed(2)
    xs = [torch.randn(m, k, generator=g).bfloat16().cuda() for m, n, k in sizes]
    ws_ = [nv.mx_quantize(torch.randn(n, k, generator=g).cuda()).row for m, n, k in sizes]
    alone = [nv.mx_linear(x, w) for x, w in zip(xs, ws_)]
    ws = nv.new_workspace(max(nv.nvfp4_mx_linear_workspace_bytes(*s) for s in sizes))
    for r in range(6):
        for i in (range(6) if r % 2 else reversed(range(6))):
            assert torch.equal(nv.mx_linear(xs[i], ws_[i], workspace=ws), alone[i])
            assert not ws[:256 + 4 * 8192].any()
    assert nv.nvfp4_get_device_status(ws) == nv.OK


def test_large_product(nv):
    """2048 x 3584 x 18944 on sampled rows and columns."""
    M, N, K = 2048, 3584, 18944
    a, a64, sa = _operand(nv, "nv", M, K, 1)
    w, w64, sw = _operand(nv, "nv", N, K, 2)
    y = nv.w4a4_gemm(a, w)
    rows = np.random.default_rng(0).choice(M, 200, replace=False)
    cols = np.random.default_rng(1).choice(N, 300, replace=False)
    _check_product(y[torch.from_numpy(rows).cuda()][:, torch.from_numpy(cols).cuda()], a64[rows], w64[cols], sa * sw, K)
    assert torch.equal(y, nv.w4a4_gemm(a, w))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M", [2, 3, 5, 9, 15, 16])
@pytest.mark.parametrize("N,K", [(257, 3616), (129, 96), (40, 32), (1500, 992)])
def test_few_tokens(nv, M, N, K, dtype):
    """One kernel or two by the work a CTA has: the same bits either way, and as the quantiser's codes give."""
    g = torch.Generator().manual_seed(100 * M + K)
    x = (torch.randn(M, K, generator=g) * torch.exp2(torch.randint(-9, 9, (M, 1), generator=g).float())).to(dtype).cuda()
    x[M // 2] = 0
    w = nv.mx_quantize((torch.randn(N, K, generator=g) * 0.1).cuda()).row
    y = nv.mx_linear(x, w)
    _check_product(y, ref.mx_round(ref.to64(x)), ref.to64(w.dequantize()), 1.0, K)
    assert torch.equal(y, nv.w4a4_gemm(nv.mx_quantize(x).row, w))
    x[M - 1, K - 1] = float("inf")
    bad = nv.mx_linear(x, w)
    assert torch.isnan(bad[M - 1]).all() and torch.equal(bad[:M - 1], y[:M - 1])
