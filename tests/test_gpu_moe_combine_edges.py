"""The weighted sum at the edges of what it takes."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("N", [2 ** 24 - 1, 2 ** 24 - 2, 65535 * 256 + 1, 65535 * 256 - 1, 2 ** 24])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_widest_rows(nv, dtype, N):
    """A row in more pieces than a grid has places for."""
    g = torch.Generator("cuda").manual_seed(1)
    y = torch.randn(2, N, device="cuda", generator=g).to(dtype)
    plan = nv.moe_plan(torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"), 2)
    w = torch.tensor([[0.25, 2.0]], device="cuda")
    want = 0.25 * y[1].double() + 2 * y[0].double()     # choice 0's row is the second expert's
    out = nv.moe_combine(y, w, plan)[0]
    # powers of two: one addition is rounded, then the result
    tol = 2.0 ** -24 * want.abs() + (2.0 ** -8 * 1.01 * want.abs() if dtype is BF else 0)
    assert ((out.double() - want).abs() <= tol).all()
    dy, dw = nv.moe_combine_backward(y[:1].contiguous(), y, w, plan)
    assert torch.equal(dy[1], (0.25 * y[0].float()).to(dtype)) and torch.equal(dy[0], (2 * y[0].float()).to(dtype))
    prod = y[0].double() * y[1].double()
    # 256 threads' sums of N / 256 terms and a tree
    assert (dw[0, 0].double() - prod.sum()).abs() <= prod.abs().sum() * (N / 256 + 16) * 2.0 ** -24
