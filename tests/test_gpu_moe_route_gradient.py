"""The router's gradient where its terms nearly cancel: one weight close to 1, gradients of the weights with a common
offset.  Against 64 bits, entry by entry."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def _score(z, scoring, renorm, idx):
    """The taken scores and the sum of the others' (64 bits)."""
    if renorm:
        ln = torch.nn.functional.logsigmoid(z) if scoring == "sigmoid" else z
        return torch.softmax(ln.gather(1, idx), 1), torch.zeros_like(z[:, :1])
    if scoring == "sigmoid":
        return torch.sigmoid(z.gather(1, idx)), None
    p = torch.softmax(z, 1)
    return p.gather(1, idx), p.scatter(1, idx, 0.0).sum(1, keepdim=True)


@pytest.mark.parametrize("offset", [0.0, 100.0, -3e4])
@pytest.mark.parametrize("E,k", [(4, 4), (40, 1), (40, 2), (256, 8), (1000, 32)])
@pytest.mark.parametrize("scoring,renorm,bias", [("softmax", True, False), ("softmax", False, False), ("softmax", False, True),
                                                 ("sigmoid", True, True), ("sigmoid", False, False), ("softmax", True, True)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradient_of_peaked_rows(nv, dtype, scoring, renorm, bias, E, k, offset):
    g = torch.Generator("cuda").manual_seed(E + k)
    T, scale = 60, 2.5
    z = torch.randn(T, E, device="cuda", generator=g)
    # the largest logit from 0 to 30 above the others, in some rows two of them
    top = torch.randint(0, E, (T, 2), device="cuda", generator=g)
    peak = torch.linspace(0, 30, T, device="cuda")[:, None]
    if scoring == "sigmoid":
        z = z - peak        # scores far below 1, their ratios as far apart
    z.scatter_(1, top[:, :1], 2 + (peak if scoring == "softmax" else 0 * peak))
    z[::3].scatter_(1, top[::3, 1:], z[::3].amax(1, keepdim=True))
    z = z.to(dtype)
    b = torch.randperm(E, device="cuda", generator=g).float() * 2 if bias else None
    dw = torch.randn(T, k, device="cuda", generator=g) + offset
    r = nv.moe_route(z, k, scoring=scoring, renormalise=renorm, bias=b, scale=scale)
    dz = nv.moe_route_backward(dw, z, r)

    idx, z64, d = r.experts.long(), z.double(), dw.double()
    u, others = _score(z64, scoring, renorm, idx)
    # relative error of a weight: the difference to the largest logit is rounded at the logits' size, which the
    # exponential makes relative; two exponentials and two additions' trees of 4 steps each, a division, the scale
    weight = 2.0 ** -24 * (4 * z64.abs().max().item() + 4 * 4 + 12 + 4)
    if others is None:      # own scores: w dw sigmoid(-z)
        taken = scale * u * d * torch.sigmoid(-z64.gather(1, idx))
        size = taken.abs()
        want = torch.zeros_like(z64).scatter(1, idx, taken)
        tol = torch.zeros_like(z64).scatter(1, idx, size * (weight + 12 * 2.0 ** -24))
    else:
        gap = d[:, :, None] - d[:, None, :]
        taken = scale * u * ((u[:, None, :] * gap).sum(2) + others * d)
        size = scale * u * ((u[:, None, :] * gap.abs()).sum(2) + others * d.abs())
        if scoring == "sigmoid":
            s = torch.sigmoid(-z64.gather(1, idx))
            taken, size = taken * s, size * s
        want, most = torch.zeros_like(z64), torch.zeros_like(z64)
        if not renorm:
            p = torch.softmax(z64, 1)
            want, most = -p * scale * (u * d).sum(1, keepdim=True), p * scale * (u * d).abs().sum(1, keepdim=True)
        want, most = want.scatter(1, idx, taken), most.scatter(1, idx, size)
        # two weights (three with the sum of the others) are involved; k fused additions, E / 32 + 5 of the scores; the
        # difference, division, products and the sigmoid's six roundings
        tol = most * (3 * weight + (k + E / 32 + 5 + 12) * 2.0 ** -24)
    # below the smallest normal number a step is 2^-149 in FP32 (bf16: 2^-133), a few of them for the factors
    tiny = 2.0 ** -130 if dtype is BF else 2.0 ** -140
    err = (dz.double() - want).abs()
    assert (err <= tol + HALF_STEP[dtype] * 1.01 * want.abs() + tiny).all(), (err / (tol + HALF_STEP[dtype] * want.abs() + tiny)).max()
    if renorm and k == 1:
        assert (dz == 0).all()
    if renorm and scoring == "softmax" and dtype is F32:
        # what one logit gains the others lose: of the order of the entries' errors, not of dw
        assert (dz.double().sum(1).abs() <= 2 * tol.sum(1) + 1e-38).all()


def test_gradients_that_are_not_finite(nv):
    """A NaN in dw of a used slot makes the row's gradient NaN, one of an unused slot does nothing."""
    inf, nan = float("inf"), float("nan")
    z = torch.tensor([[1.0, 2.0, 0.0, -1.0], [1.0, -inf, 0.5, -inf], [1.0, 2.0, 0.0, -1.0], [5.0, 1.0, 0.0, 2.0]], device="cuda")
    dw = torch.tensor([[1.0, nan, 2.0], [1.0, 2.0, nan], [1.0, 2.0, 3.0], [nan, 1.0, 1.0]], device="cuda")
    for renorm in (True, False):
        r = nv.moe_route(z, 3, renormalise=renorm)
        assert r.experts[1].tolist() == [0, 2, -1]
        dz = nv.moe_route_backward(dw, z, r)
        assert dz[0].isnan().all() and dz[3].isnan().all() and dz[1:3].isfinite().all()
        assert dz[1, 1] == 0 and dz[1, 3] == 0
    one = nv.moe_route(z, 1)
    dz = nv.moe_route_backward(torch.full((4, 1), nan, device="cuda"), z, one)
    assert dz.isnan().all()
