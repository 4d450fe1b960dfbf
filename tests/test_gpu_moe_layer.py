"""The layer grouped by expert (quantisers, product, backward pass) against 64-bit definitions."""
import pytest
import torch

from tests import moe_reference as ref

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HALF_STEP = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def _gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def _close(got, a, b):
    """got against a @ b^T (64 bits): FP32 sums whose terms are exact; every addition is off by a step (2^-23) of the
    running sum at most, which the sum of the magnitudes bounds; an instruction adds 64 terms at a time."""
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    tol = size * (a.shape[1] / 64 + 64 + 8) * 2.0 ** -23 + HALF_STEP[got.dtype] * 1.01 * want.abs()
    bad = want.isnan()
    assert torch.equal(got.isnan(), bad)
    err = (got.double() - want).abs()
    assert (err[~bad] <= tol[~bad]).all(), (err / tol)[~bad].max()


def _experts(T, k, E, how, g):
    ex = torch.randint(0, E, (T, k), device="cuda", generator=g, dtype=torch.int32)
    if how == "one":
        ex[:] = E // 2
    elif how == "dropped":
        ex[torch.rand(T, k, device="cuda", generator=g) < 0.4] = -1
    elif how == "none":
        ex[:] = -1
    return ex


LAYERS = [  # T, k, E, N, K
    (1, 1, 1, 1, 32), (1, 8, 128, 384, 512), (5, 2, 3, 100, 96), (64, 4, 60, 257, 416), (90, 3, 8, 130, 1024),
    (120, 2, 7, 264, 160), (300, 2, 4, 264, 256), (700, 1, 3, 520, 800), (2000, 4, 8, 512, 288), (33, 1, 1, 640, 2048),
]


@pytest.mark.parametrize("T,k,E,N,K", LAYERS)
@pytest.mark.parametrize("how", ["random", "one", "dropped"])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (F32, F32)])
def test_layer(nv, T, k, E, N, K, how, dtype, out):
    g = _gen(T + N + K)
    ex = _experts(T, k, E, how, g)
    plan = nv.moe_plan(ex, E)
    w = (torch.randn(E, N, K, device="cuda", generator=g) * 0.05).to(dtype)
    x = torch.randn(T, K + 8, device="cuda", generator=g).to(dtype)[:, :K]     # rows with a stride
    wq = nv.moe_quantize_weights(w).row
    ws = nv.new_workspace(nv.nvfp4_moe_linear_workspace_bytes(T, k, E, N, K))
    y = nv.moe_linear(x, wq, plan, out_dtype=out, workspace=ws)
    at, order = plan.offsets.tolist(), plan.order.long()
    xr = ref.mx_round(x)
    for e in range(E):
        if at[e + 1] > at[e]:
            _close(y[at[e]:at[e + 1]], xr[order[at[e]:at[e + 1]] // k], ref.mx_round(w[e]))
    rows = at[-1]
    # the same from the quantiser and the product, bit for bit, and from sorted rows
    q = nv.moe_quantize(x, plan)
    assert torch.equal(nv.moe_gemm(q.row, wq, plan, out_dtype=out, workspace=ws)[:rows], y[:rows])
    xs = torch.full((T * k, K), float("nan"), dtype=dtype, device="cuda")
    xs[:rows] = x[order[:rows] // k]
    assert torch.equal(nv.moe_linear(xs, wq, plan, out_dtype=out, sorted_rows=True, workspace=ws)[:rows], y[:rows])
    assert nv.nvfp4_get_device_status(ws) == nv.OK


def test_rows_behind_the_last_one_are_left(nv):
    g = _gen(1)
    for T, k, E, N, K in [(9, 2, 4, 96, 64), (700, 2, 4, 264, 96)]:
        ex = _experts(T, k, E, "dropped", g)
        plan = nv.moe_plan(ex, E)
        rows = int(plan.offsets[-1])
        wq = nv.moe_quantize_weights(torch.randn(E, N, K, device="cuda", generator=g)).row
        q = nv.moe_quantize(torch.randn(T, K, device="cuda", generator=g), plan).row
        ws = nv.new_workspace(nv.nvfp4_moe_gemm_workspace_bytes(T, k, E, N, K))
        y = torch.full((T * k, N), 7.5, device="cuda")
        nv._call("nvfp4_moe_gemm", *q.addresses(), *wq.addresses(), plan.buffer.data_ptr(), plan.nbytes, T, k, E, N, K,
                 y.data_ptr(), nv.OUT_FP32, ws.data_ptr(), ws.numel(), nv._raw_stream())
        assert 0 < rows < T * k and (y[rows:] == 7.5).all() and torch.equal(
            y[:rows], nv.moe_gemm(q, wq, plan)[:rows])


def test_no_rows_at_all(nv):
    g = _gen(2)
    T, k, E, N, K = 40, 2, 3, 96, 64
    plan = nv.moe_plan(_experts(T, k, E, "none", g), E)
    wq = nv.moe_quantize_weights(torch.randn(E, N, K, device="cuda", generator=g), colwise=True)
    nv.moe_linear(torch.randn(T, K, device="cuda", generator=g), wq.row, plan)
    x = nv.moe_quantize(torch.randn(T, K, device="cuda", generator=g), plan, colwise=True)
    _, dw = nv.moe_linear_backward(torch.randn(T * k, N, device="cuda", generator=g), x.col, wq.col, plan)
    assert (dw == 0).all()


def test_values_that_are_not_finite_stay_in_their_rows(nv):
    """A NaN in a token's row reaches that token's rows of Y only, also where it shares a tile with others."""
    g = _gen(3)
    for T in (20, 900):
        k, E, N, K = 2, 3, 72, 128
        ex = _experts(T, k, E, "random", g)
        plan = nv.moe_plan(ex, E)
        x = torch.randn(T, K, device="cuda", generator=g)
        x[5, 40], x[11, 3] = float("nan"), float("inf")
        y = nv.moe_linear(x, nv.moe_quantize_weights(torch.randn(E, N, K, device="cuda", generator=g)).row, plan)
        token = plan.order.long() // k
        assert torch.equal(y.isnan().all(1), (token == 5) | (token == 11)) and torch.equal(y.isnan().any(1), y.isnan().all(1))


@pytest.mark.parametrize("T,k,E,N,K", [(1, 1, 2, 32, 32), (40, 2, 5, 96, 160), (333, 2, 7, 1056, 800), (900, 1, 3, 512, 288),
                                       (2000, 4, 6, 288, 512)])
@pytest.mark.parametrize("how", ["random", "one", "dropped"])
@pytest.mark.parametrize("dtype,out", [(BF, BF), (F32, F32)])
def test_backward(nv, T, k, E, N, K, how, dtype, out):
    g = _gen(T + N)
    ex = _experts(T, k, E, how, g)
    plan = nv.moe_plan(ex, E)
    rows = int(plan.offsets[-1])
    x = torch.randn(T, K, device="cuda", generator=g).to(dtype)
    w = (torch.randn(E, N, K, device="cuda", generator=g) * 0.05).to(dtype)
    dy = torch.randn(T * k, N + 8, device="cuda", generator=g).to(dtype)[:, :N]
    dy[rows:] = float("nan")        # not read
    xq, wq = nv.moe_quantize(x, plan, colwise=True), nv.moe_quantize_weights(w, colwise=True)
    # both directions of the quantiser give the same rows as one
    y = nv.moe_gemm(xq.row, wq.row, plan, out_dtype=out)
    assert torch.equal(y[:rows], nv.moe_linear(x, wq.row, plan, out_dtype=out)[:rows])
    ws = nv.new_workspace(nv.nvfp4_moe_linear_backward_workspace_bytes(T, k, E, N, K))
    dx, dw = nv.moe_linear_backward(dy, xq.col, wq.col, plan, dx_dtype=out, dw_dtype=out, workspace=ws)
    at, order = plan.offsets.tolist(), plan.order.long()
    for e in range(E):
        a, b = at[e], at[e + 1]
        if a == b:
            assert (dw[e] == 0).all()
            continue
        _close(dx[a:b], ref.mx_round(dy[a:b]), ref.mx_round_rows(w[e]).t())
        _close(dw[e], ref.mx_round_rows(dy[a:b]).t(), ref.mx_round_rows(x[order[a:b] // k]).t())
    only = nv.moe_linear_backward(dy, None, wq.col, plan, dx_dtype=out, workspace=ws)
    assert only[1] is None and torch.equal(only[0][:rows], dx[:rows])
    only = nv.moe_linear_backward(dy, xq.col, None, plan, dw_dtype=out, workspace=ws)
    assert only[0] is None and torch.equal(only[1], dw)
    assert nv.nvfp4_get_device_status(ws) == nv.OK


def test_weights_quantised_as_each_alone(nv):
    g = _gen(4)
    for dtype in (BF, F32):
        w = torch.randn(3, 200, 160, device="cuda", generator=g).to(dtype)
        q = nv.moe_quantize_weights(w, colwise=True)
        for e in range(3):
            one = nv.mx_quantize(w[e], colwise=True)
            assert torch.equal(q.row.codes[e], one.row.codes) and torch.equal(q.row.scales[e], one.row.scales)
            assert torch.equal(q.col.codes[e], one.col.codes) and torch.equal(q.col.scales[e], one.col.scales)
            assert torch.equal(q.row.expert(e).dequantize(), one.row.dequantize())


@pytest.mark.parametrize("T,k,E", [(1, 2, 4), (30, 2, 5), (400, 2, 4)])
def test_layers_behind_one_another(nv, T, k, E):
    """Launches overlap: each call's rows are what the call before has just written, its output goes where that read,
    and every other call's plan has just been made."""
    g = _gen(T)
    K, R = 512, T * k
    ex = _experts(T, k, E, "random", g)
    ws_ = [nv.moe_quantize_weights(torch.randn(E, K, K, device="cuda", generator=g) / K ** 0.5).row for _ in range(3)]
    x = torch.randn(R, K, device="cuda", generator=g)
    plan = nv.moe_plan(ex, E)
    space = nv.new_workspace(nv.nvfp4_moe_linear_workspace_bytes(T, k, E, K, K))
    want, t = [], x
    for i in range(12):
        t = nv.moe_linear(t, ws_[i % 3], plan, sorted_rows=True)
        torch.cuda.synchronize()
        want.append(t)
    for _ in range(3):
        buf = [x.clone(), torch.empty_like(x)]
        torch.cuda.synchronize()
        for i in range(12):
            a, b = buf[i % 2], buf[1 - i % 2]
            if i % 2:
                plan = nv.moe_plan(ex, E)
            nv._call("nvfp4_moe_linear", a.data_ptr(), nv.OUT_FP32, K, 1, *ws_[i % 3].addresses(), plan.buffer.data_ptr(),
                     plan.nbytes, T, k, E, K, K, b.data_ptr(), nv.OUT_FP32, space.data_ptr(), space.numel(),
                     nv._raw_stream())
        assert torch.equal(buf[0], want[11]) and torch.equal(buf[1], want[10])
    assert nv.nvfp4_get_device_status(space) == nv.OK
