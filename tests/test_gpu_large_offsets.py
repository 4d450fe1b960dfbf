"""Outputs of more than 2^32 elements and plans of the most slots: offsets of rows far back."""
import pytest
import torch

from tests import moe_reference as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def memory():
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    yield
    torch.cuda.empty_cache()


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


@pytest.mark.parametrize("T,k,E", [(500000, 8, 60), (1 << 21, 8, 1024), (1 << 24, 1, 3)])
def test_plan_of_many_slots(nv, T, k, E):
    ex = torch.randint(-1, E, (T, k), device="cuda", generator=_gen(1), dtype=torch.int32)
    plan = nv.moe_plan(ex, E)
    flat = ex.reshape(-1)
    key = torch.where(flat < 0, E, flat)
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=E + 1)
    rows = int(counts[:E].sum())
    assert torch.equal(plan.offsets, torch.cat((counts.new_zeros(1), counts[:E].cumsum(0))).int())
    assert torch.equal(plan.order[:rows], order[:rows].int()) and (plan.order[rows:] == -1).all()
    where = torch.full((T * k,), -1, dtype=torch.int32, device="cuda")
    where[order[:rows]] = torch.arange(rows, device="cuda", dtype=torch.int32)
    assert torch.equal(plan.position.reshape(-1), where)


def test_experts_and_sum_of_many_rows(nv):
    T, k, E, N, K = 140000, 8, 3, 4096, 64
    g = _gen(2)
    plan = nv.moe_plan(torch.randint(0, E, (T, k), device="cuda", generator=g, dtype=torch.int32), E)
    x = torch.randn(T, K, device="cuda", generator=g).to(BF)
    w = torch.randn(E, N, K, device="cuda", generator=g) / 8
    y = nv.moe_linear(x, nv.moe_quantize_weights(w).row, plan, out_dtype=BF)
    assert y.numel() > 1 << 32
    weights = torch.rand(T, k, device="cuda", generator=g)
    out = nv.moe_combine(y, weights, plan)
    dout = torch.randn(T, N, device="cuda", generator=g).to(BF)
    dy, dw = nv.moe_combine_backward(dout, y, weights, plan)
    at, order = plan.offsets.tolist(), plan.order
    for e in range(E):
        wr = ref.mx_round(w[e])
        for r in (at[e], (at[e] + at[e + 1]) // 2, at[e + 1] - 1):
            slot = int(order[r])
            t, j = slot // k, slot % k
            want = ref.mx_round(x[t:t + 1]) @ wr.t()
            # 64 terms, then bf16
            size = ref.mx_round(x[t:t + 1]).abs() @ wr.abs().t()
            assert ((y[r].double() - want).abs() <= 2.0 ** -8 * want.abs() + 80 * 2.0 ** -23 * size).all()
            assert torch.equal(dy[r], (weights[t, j] * dout[t].float()).to(BF))
            prod = dout[t].double() * y[r].double()
            assert (dw[t, j] - prod.sum()).abs() <= prod.abs().sum() * 32 * 2.0 ** -24
    for t in (0, T // 2, T - 1):
        rows = y[plan.position[t].long()].double() * weights[t, :, None].double()
        assert ((out[t].double() - rows.sum(0)).abs() <= 2.0 ** -8 * rows.sum(0).abs() + 10 * 2.0 ** -24 * rows.abs().sum(0)).all()


def test_int8_of_many_tokens(nv):
    M, N, K = 70000, 65600, 64
    g = _gen(3)
    x = torch.randn(M, K, device="cuda", generator=g).to(BF)
    w = nv.int8_quantize(torch.randn(N, K, device="cuda", generator=g))
    y = nv.int8_linear(x, w, out_dtype=BF)
    assert y.numel() > 1 << 32
    a = nv.int8_quantize(x)
    for rows in (slice(0, 2), slice(M // 2, M // 2 + 2), slice(M - 2, M)):
        want = (a.codes[rows].double() @ w.codes.double().t()) * a.scales[rows, None].double() * w.scales.double()
        assert ((y[rows].double() - want).abs() <= (2.0 ** -8 + 3 * 2.0 ** -24) * 1.01 * want.abs()).all()
