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


@pytest.mark.parametrize("N", [7, 8, 264])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_weights_without_an_expert(nv, dtype, N):
    """Whatever such a weight is, it adds nothing; only a NaN shows."""
    inf, nan = float("inf"), float("nan")
    ex = torch.tensor([[0, -1], [-1, 1], [-1, -1], [1, 0], [-1, 0]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[1.0, inf], [-inf, 2.0], [inf, -inf], [3e38, 0.0], [nan, 1.0]], device="cuda")
    plan = nv.moe_plan(ex, 2)
    y = torch.ones(10, N, device="cuda", dtype=dtype)
    y[3] = 0
    base = torch.full((5, N), 0.5, device="cuda", dtype=dtype)
    pos = plan.position.tolist()
    for b, add in ((None, 0.0), (base, 0.5)):
        out = nv.moe_combine(y, w, plan, base=b).double()
        for t in range(5):
            want = add + sum(w[t, j].double() * y[pos[t][j], 0].double() for j in range(2) if pos[t][j] >= 0)
            if w[t].isnan().any():
                assert out[t].isnan().all()
            else:       # sums of two terms, rounded to FP32 and to the result's type
                assert ((out[t] - want).abs() <= 2.0 ** -7 * abs(want)).all()
    dy, dw = nv.moe_combine_backward(base, y, w, plan)
    assert dw[0, 1] == 0 and dw[1, 0] == 0 and (dw[2] == 0).all() and dw[4, 0] == 0
