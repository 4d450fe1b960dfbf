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
