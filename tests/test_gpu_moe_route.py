"""Routing, grouping, the router's gradient, and the weighted sum with its gradient, against 64-bit definitions."""
import pytest
import torch

from tests import moe_reference as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _same_plan(plan, experts):
    offsets, order, position = ref.plan(experts.cpu(), plan.E)
    assert torch.equal(plan.offsets.cpu(), offsets)
    assert torch.equal(plan.order.cpu(), order)
    assert torch.equal(plan.position.cpu(), position)


def _weight_tolerance(z, E):
    """FP32: the difference to the largest logit (rounded: half a step of the logits' size, which the exponential makes
    relative), two exponentials, E additions at most in a tree, a division, the scale."""
    size = torch.where(torch.isfinite(z), z.abs(), 0.0).max().item()
    return 2.0 ** -24 * (4 * size + 4 * 4 + 12 + 4)


CASES = [  # T, E, k, dtype, scoring, renormalise, bias, scale
    (1, 1, 1, F32, "softmax", True, False, 1.0), (1, 64, 6, BF, "softmax", True, False, 1.0),
    (3, 5, 5, F32, "softmax", False, False, 2.5), (40, 33, 32, BF, "softmax", True, False, 1.0),
    (130, 128, 8, BF, "softmax", False, False, 1.0), (257, 256, 8, F32, "sigmoid", True, True, 2.5),
    (100, 500, 3, F32, "sigmoid", False, False, 1.0), (70, 1024, 10, BF, "softmax", True, False, 0.5),
    (64, 100, 4, F32, "softmax", True, True, 1.0), (3000, 60, 4, BF, "softmax", True, False, 1.0),
]


@pytest.mark.parametrize("T,E,k,dtype,scoring,renorm,bias,scale", CASES)
def test_route(nv, T, E, k, dtype, scoring, renorm, bias, scale):
    g = _gen(T + E)
    wide = torch.randn(T, E + 3, device="cuda", generator=g).mul_(2).to(dtype)
    # rows with a stride, a base 16-byte aligned
    z = wide[:, :E] if T > 1 else wide[:, :E].contiguous()
    b = None
    if bias:
        # scores plus bias are apart by more than their rounding: the bias orders the experts in steps above the scores
        b = torch.randperm(E, device="cuda", generator=g).float() * 2
    r = nv.moe_route(z, k, scoring=scoring, renormalise=renorm, bias=b, scale=scale)
    w, ex = ref.route(z.cpu(), k, scoring, renorm, None if b is None else b.cpu(), scale)
    assert torch.equal(r.experts.cpu(), ex)
    _same_plan(r.plan, ex)
    assert ((r.weights.cpu().double() - w).abs() <= _weight_tolerance(z.float(), E) * w.abs() + 1e-38).all()

    # the gradient against the formula by automatic differentiation in 64 bits
    dw = torch.randn(T, k, device="cuda", generator=g)
    dz = nv.moe_route_backward(dw, z, r)
    z64 = z.double().requires_grad_()
    idx = r.experts.long()
    if renorm:
        ln = torch.nn.functional.logsigmoid(z64) if scoring == "sigmoid" else z64
        w64 = torch.softmax(ln.gather(1, idx), 1) * scale
    else:
        w64 = (torch.sigmoid(z64) if scoring == "sigmoid" else torch.softmax(z64, 1)).gather(1, idx) * scale
    want, = torch.autograd.grad((w64 * dw.double()).sum(), z64)
    # terms of size w |dw| are subtracted; each has the weights' error and k additions
    size = scale * dw.abs().double().amax(1, keepdim=True)
    tol = size * (3 * _weight_tolerance(z.float(), E) + 40 * 2.0 ** -24) + HALF_STEP[dtype] * want.abs()
    assert dz.dtype == dtype and ((dz.double() - want).abs() <= tol).all()


def test_router_gradient_by_differences(nv):
    """A step along a direction changes <dw, weights> by <dz, direction>, to second order in the step."""
    g = _gen(9)
    T, E, k, h = 50, 40, 4, 2.0 ** -7
    z = torch.randn(T, E, device="cuda", generator=g)
    dw = torch.randn(T, k, device="cuda", generator=g)
    r = nv.moe_route(z, k)
    # a direction over the chosen experts, so that the choice stays
    d = torch.zeros_like(z).scatter_(1, r.experts.long(), torch.randn(T, k, device="cuda", generator=g))
    move = lambda s: torch.softmax((z + s * d).double().gather(1, r.experts.long()), 1)  # noqa: E731
    dz = nv.moe_route_backward(dw, z, r)
    slope = ((move(h) - move(-h)) * dw).sum(1) / (2 * h)
    # third derivative of a softmax along d: below 8 |d|^3
    third = 8 * d.abs().amax(1).double() ** 3 * dw.abs().sum(1)
    assert ((slope - (dz * d).double().sum(1)).abs() <= h * h / 6 * third + 1e-4).all()


def test_rows_that_leave_little(nv):
    inf, nan = float("inf"), float("nan")
    z = torch.tensor([[-inf] * 6, [-inf, 1.0, -inf, -inf, 2.0, -inf], [0.0, -0.0, 0.0, 0.0, -0.0, 0.0],
                      [1.0, nan, 3.0, 0.0, 2.0, -inf], [-3e38, -inf, -3.4e38, -inf, -inf, -inf], [-200.0, -300.0] + [-inf] * 4],
                     device="cuda")
    r = nv.moe_route(z, 3)
    w, ex = r.weights.cpu(), r.experts.cpu()
    assert ex.tolist() == [[-1, -1, -1], [4, 1, -1], [0, 1, 2], [2, 4, 0], [0, 2, -1], [0, 1, -1]]
    assert w[0].tolist() == [0, 0, 0] and w[1, 2] == 0 and w[3].isnan().all()
    assert torch.allclose(w[2], torch.full((3,), 1 / 3)) and w[4].tolist() == [1, 0, 0]
    # e^-100 = 3.7e-44 is a subnormal number, steps of 2^-149 apart
    assert w[5, 0] == 1 and abs(w[5, 1].double() - torch.tensor(-100.0).double().exp()) <= 2.0 ** -148 and w[5, 2] == 0
    _same_plan(r.plan, ex)
    dz = nv.moe_route_backward(torch.ones(6, 3, device="cuda"), z, r)
    assert dz[:3].abs().max() < 1e-6 and dz[3].isnan().all() and dz[4:].abs().max() < 1e-40
    # far below zero sigmoids underflow, their ratios do not
    s = nv.moe_route(torch.tensor([[-200.0, -201.0, -500.0]], device="cuda"), 2, scoring="sigmoid")
    assert torch.allclose(s.weights.double(), torch.softmax(torch.tensor([[-200.0, -201.0]], device="cuda").double(), 1))
    # a bias of -inf shuts an expert out
    b = torch.tensor([-inf, 0, 0], device="cuda")
    assert nv.moe_route(torch.tensor([[9.0, 1.0, 0.0]], device="cuda"), 3, bias=b).experts.tolist() == [[1, 2, -1]]


@pytest.mark.parametrize("E", [40, 64, 100, 128, 256, 300, 512, 1024])
@pytest.mark.parametrize("k", [1, 6, 8, 16, 17, 32])
def test_orders_of_experts(nv, E, k):
    """Logits in ascending and descending order (the best in few lanes), equal ones, few distinct ones, and a largest
    value that 31 to 34 experts share: the choice is that of a stable sort."""
    g = _gen(E + k)
    up = torch.arange(E, device="cuda", dtype=F32)
    rows = [up, -up, torch.zeros_like(up), up // 3, -(up // 5), up % 7]
    for n in (31, 32, 33, 34):
        row = torch.randn(E, device="cuda", generator=g).clamp_(max=2.0)
        row[torch.randperm(E, device="cuda", generator=g)[:n]] = 3.0
        rows.append(row)
    z = torch.cat([torch.stack(rows), torch.randn(40, E, device="cuda", generator=g).mul_(3).round_()])
    want = torch.argsort(z, dim=1, descending=True, stable=True)[:, :k].int()
    r = nv.moe_route(z, k)
    assert torch.equal(r.experts, want)
    _same_plan(r.plan, want)
    assert torch.equal(nv.moe_route(z, k, scoring="sigmoid", bias=-z.new_full((E,), float("inf"))).experts,
                       torch.full_like(want, -1))


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 128), (7, 3, 2), (1000, 1, 5), (700, 4, 1000), (5000, 8, 60),
                                   (40000, 2, 17)])
@pytest.mark.parametrize("how", ["random", "one", "twice", "dropped"])
def test_plan(nv, T, k, E, how):
    g = _gen(T + k)
    ex = torch.randint(0, E, (T, k), device="cuda", generator=g, dtype=torch.int32)
    if how == "one":
        ex[:] = E - 1
    elif how == "twice":
        ex[:] = ex[:, :1]           # a token's choices are all the same expert
    elif how == "dropped":
        ex[torch.rand(T, k, device="cuda", generator=g) < 0.4] = -1
    _same_plan(nv.moe_plan(ex, E), ex)


def test_plan_beyond_the_last_expert(nv):
    ex = torch.tensor([[0, 7], [2, 3], [-5, 1]], dtype=torch.int32, device="cuda")
    ws = nv.new_workspace(256)
    plan = nv.moe_plan(ex, 3, workspace=ws)
    _same_plan(plan, torch.where(ex >= 3, -1, ex))
    assert nv.nvfp4_get_device_status(ws) == nv.ERR_INDEX
    assert nv.nvfp4_get_device_status(ws) == nv.OK
    nv.moe_plan(ex, 8, workspace=ws)
    assert nv.nvfp4_get_device_status(ws) == nv.OK


@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (3, 2, 7), (16, 8, 4096), (100, 5, 264), (33, 32, 72), (1000, 3, 130)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_combine(nv, T, k, N, dtype):
    g = _gen(T * k + N)
    E = 9
    ex = torch.randint(-1, E, (T, k), device="cuda", generator=g, dtype=torch.int32)
    plan = nv.moe_plan(ex, E)
    pos = plan.position
    rows = int(plan.offsets[-1])
    y = torch.randn(T * k, N, device="cuda", generator=g).to(dtype)
    y[rows:] = float("nan")         # behind the last row: not read
    w = torch.rand(T, k, device="cuda", generator=g)
    base = torch.randn(T, N, device="cuda", generator=g).to(dtype)
    for weights, b, odt in ((w, None, dtype), (w, base, dtype), (None, None, BF), (None, None, F32)):
        out = nv.moe_combine(y, weights, plan, base=b, out_dtype=odt)
        want, size = ref.combine(y, weights, pos, b)
        # a product and an addition a slot, and the rounding of the result
        assert ((out.double() - want).abs() <= size * (k + 1) * 2.0 ** -24 + HALF_STEP[odt] * want.abs() * 1.01).all()
    dout = torch.randn(T, N, device="cuda", generator=g).to(dtype)
    dy, dw = nv.moe_combine_backward(dout, y, w, plan)
    have = pos >= 0
    token = torch.arange(T, device="cuda")[:, None].expand(T, k)
    want = w[have][:, None].double() * dout[token[have]].double()
    assert ((dy[pos[have].long()].double() - want).abs() <= HALF_STEP[dtype] * 1.01 * want.abs() + 1e-40).all()
    prod = dout[token[have]].double() * y[pos[have].long()].double()
    err = (dw[have].double() - prod.sum(1)).abs()
    assert (err <= prod.abs().sum(1) * (N / 256 + 16) * 2.0 ** -24 + 1e-38).all() and (dw[~have] == 0).all()
    assert nv.moe_combine_backward(dout, None, w, plan, need_dweights=False)[1] is None
    # y itself may take dy
    one, two = y.clone(), nv.moe_combine_backward(dout, y, w, plan)
    nv._call("nvfp4_moe_combine_backward", dout.data_ptr(), one.data_ptr(), nv._DTYPE_CODE[dtype], w.data_ptr(),
             plan.buffer.data_ptr(), plan.nbytes, T, k, E, N, one.data_ptr(), dw.data_ptr(), nv._raw_stream())
    assert torch.equal(one[:rows], two[0][:rows]) and torch.equal(dw, two[1]) and one[rows:].isnan().all()


def test_combine_keeps_what_is_not_finite(nv):
    ex = torch.tensor([[0, -1], [-1, -1], [1, 0]], dtype=torch.int32, device="cuda")
    plan = nv.moe_plan(ex, 2)
    w = torch.tensor([[1.0, float("nan")], [0.0, 0.0], [2.0, 1.0]], device="cuda")
    out = nv.moe_combine(torch.ones(6, 8, device="cuda"), w, plan)
    assert out[0].isnan().all() and (out[1] == 0).all() and (out[2] == 3).all()
