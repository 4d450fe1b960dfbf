"""The 8-bit layer over the range of its scales and sums, against 64 bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF: 2.0 ** -8, F32: 2.0 ** -24}
LARGEST = torch.finfo(F32).max


@pytest.mark.parametrize("M,N,K", [(1, 300, 4096), (1, 200, 18944), (9, 129, 1024), (30, 300, 400), (100, 257, 2000),
                                   (300, 1000, 800), (700, 520, 512)])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (F32, F32)])
def test_scales_far_apart(nv, M, N, K, dtype, out):
    """Tokens near the largest number with weights far below 1, and the reverse: no product on the way overflows."""
    g = torch.Generator("cuda").manual_seed(M + N)
    up = torch.linspace(-100, 125, M, device="cuda").round() if M > 1 else torch.full((1,), 125.0, device="cuda")
    x = torch.randn(M, K, device="cuda", generator=g).clamp_(-3.9, 3.9)
    x = (x.double() * torch.exp2(up.double())[:, None]).to(F32).to(dtype)
    down = torch.linspace(-110, 20, N, device="cuda").round()
    w = nv.int8_quantize((torch.randn(N, K, device="cuda", generator=g).double() * torch.exp2(down.double())[:, None]).to(F32))
    y = nv.int8_linear(x, w, out_dtype=out)
    amax = x.double().abs().amax(1, keepdim=True)
    sums = torch.round(x.double() * 127 / amax) @ w.codes.double().t()
    assert sums.abs().max() < 2 ** 24       # exact in FP32, whatever the order
    want = sums * (amax / 127) * w.scales.double()
    # the token's scale and two products are rounded, then the result; below the normal numbers steps are 2^-149 in FP32,
    # where a scale's is multiplied by the sum and the other scale
    sub = 2.0 ** -149 * (1 + 2 * sums.abs() * w.scales.double()) + (2.0 ** -133 if out is BF else 0)
    tol = (3 * 2.0 ** -24 + HALF_STEP[out]) * 1.01 * want.abs() + sub
    fits = want.abs() < LARGEST * (1 - 2.0 ** -6)
    assert (fits & (want.abs() > 2.0 ** 100)).any()
    assert ((y.double() - want).abs() <= tol)[fits].all()
    over = want.abs() > LARGEST * (1 + 2.0 ** -6)
    assert (y[over].double() == torch.sign(want[over]) * torch.inf).all()
    assert torch.equal(nv.int8_gemm(nv.int8_quantize(x), w, out_dtype=out), y)


@pytest.mark.parametrize("M,K", [(1, 1024), (100, 1024), (1, 18944), (16, 18944), (40, 18944), (100, 18944), (200, 18944),
                                 (600, 18944), (1, 131072), (100, 131072)])
@pytest.mark.parametrize("how", ["random", "negative", "127 x 126", "123 x 125"])
def test_sums_of_one_sign(nv, M, K, how):
    """Against 64-bit integers.  An instruction adds 16 products to a running sum in 2^e .. 2^(e + 1).  Each product loses
    what lies below 2^(e - 25), and the sum is rounded to the nearest step, 2^(e - 23): 16 / 4 + 1 / 2 steps at most.
    (600 rows of 123 x 125, K = 18944: by this 93 instructions lose 112, 546 lose 48 and 273 lose 16, together 40992; 40896
    were measured.)  Running sums grow evenly, random ones within 5 %, so n instructions are off by 4.5 (n + 1) / 2 steps of
    the whole, and a sum whose K is shared out by 8 roundings more.  A stage of 128 left out would be 128 / K of it, which
    is above that."""
    g = torch.Generator("cuda").manual_seed(K + M)
    N = 260
    if how in ("random", "negative"):
        a, w = (torch.randint(0, 128, (n, K), device="cuda", generator=g, dtype=torch.int8) for n in (M, N))
        a = -a if how == "negative" else a
    else:
        a, w = (torch.full((n, K), v, device="cuda", dtype=torch.int8) for n, v in zip((M, N), map(int, how.split(" x "))))
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    y = nv.int8_gemm(nv.Int8Matrix(a, one(M)), nv.Int8Matrix(w, one(N))).double()
    want = a.double() @ w.double().t()      # below 2^53: exact
    n = K / 16 / (8 if K > 2 ** 16 else 1)      # three tiles of outputs: eight CTAs share K
    steps = 0 if 127 ** 2 * K < 2 ** 24 else 1.05 * (4.5 * (n + 1) / 2 + 8)
    assert steps * 2.0 ** -23 < 128 / K
    assert ((y - want).abs() <= steps * 2.0 ** -23 * want.abs()).all()


@pytest.mark.parametrize("power", [-140, -100, -61, -59, 0, 60, 103])
@pytest.mark.parametrize("cols", [512, 8192, 24576])
def test_ties_of_full_mantissas(nv, cols, power):
    """A largest magnitude of 254 c, c of 16 bits, makes ties of all odd multiples of c, whose products with 127 have more
    bits than FP32; among them their neighbours, a step of FP32 to either side."""
    g = torch.Generator("cuda").manual_seed(cols + power)
    rows = 40
    c = torch.randint(2 ** 14, 2 ** 15, (rows, 1), device="cuda", generator=g).float() * 2 + 1
    x = (torch.randint(0, 127, (rows, cols), device="cuda", generator=g).float() * 2 + 1) * c
    x[:, ::3] = torch.nextafter(x[:, ::3], torch.full_like(x[:, ::3], torch.inf))
    x[:, 1::3] = torch.nextafter(x[:, 1::3], torch.zeros_like(x[:, 1::3]))
    x *= torch.randint(0, 2, x.shape, device="cuda", generator=g).float() * 2 - 1
    x[:, 7] = 254 * c[:, 0]
    x[:, 16] = 0
    x = (x.double() * 2.0 ** power).to(F32)     # exact, except below the normal numbers
    amax = x.double().abs().amax(1, keepdim=True)
    # 31 bits over 24: in 64 bits ties stay ties and their neighbours do not become any
    want = torch.round(127 * x.double() / amax)
    q = nv.int8_quantize(x)
    assert torch.equal(q.codes.double(), want)
    assert ((q.scales.double() - amax[:, 0] / 127).abs() <= 2.0 ** -24 * amax[:, 0] / 127 + 2.0 ** -150).all()
    if cols <= 512:     # tokens quantised by the product itself
        w = nv.int8_quantize(torch.randn(300, cols, device="cuda", generator=g))
        for m in (1, 9):
            assert torch.equal(nv.int8_linear(x[:m], w), nv.int8_gemm(nv.int8_quantize(x[:m]), w))
