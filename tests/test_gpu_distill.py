"""Distillation loss and gradient on the GPU against the 64-bit definition.

Tolerances (fixed before the first run).  All statistics are FP32.  An exponent argument z log2(e)/tau - lse2 carries
a rounding error of at most 2^-23 (|z2| + |lse2|) and the base-2 logarithm and exponential about 2^-22 each, so q has
a relative error of at most r = 2^-21 (4 + max |z| / tau) (max over finite logits of the row), and so have the p.  Then
  |d loss| <= w tau^2 r sum_j p_j (4 + |log p_j| + |log q_j|)   (+ the rest class's term with 1 - sum p: k 2^-23),
  |d dz_v| <= |c| [r (q_v P + p_v) + q_v / q_r (r p_r + k 2^-23)];
a bf16 gradient adds half a unit in the last place, 2^-8 of its magnitude.
"""
import numpy as np
import pytest
import torch

from tests import fp4_reference as ref

pytestmark = pytest.mark.gpu


def _case(T, V, k, dtype, seed, tail=False, tau=1.0, tdtype=torch.float32, spread=3.0, ld=None):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, V, generator=g) * spread
    t = z + torch.randn(T, V, generator=g)
    if tail:
        t = torch.log_softmax(t / tau, 1)
    val, idx = torch.topk(t, k, dim=1)
    perm = torch.argsort(torch.rand(T, k, generator=g), 1)  # entries in no order
    val, idx = val.gather(1, perm), idx.gather(1, perm)
    if ld is not None:
        buf = torch.full((T, ld), float("nan"))
        buf[:, :V] = z
        zg = buf.to(dtype).cuda()[:, :V]
    else:
        zg = z.to(dtype).cuda()
    return zg, idx.cuda(), val.to(tdtype).cuda()


def _tol(z, idx, t, tau, tail, w, g):
    """(loss tolerance (T,), dz tolerance (T, V)) as derived above."""
    T, V = z.shape
    k = idx.shape[1]
    lt, dt = np.zeros(T), np.zeros((T, V))
    for r in range(T):
        wr = 1.0 if w is None else w[r]
        gr = 1.0 if g is None else g[r if len(g) == T else 0]
        used = [j for j in range(k) if 0 <= idx[r, j] < V]
        if wr == 0 or not used:
            continue
        if not tail and (t[r, used] == -np.inf).all():
            continue                     # loss and gradient exactly 0
        zz = z[r] / tau
        fin = zz[np.isfinite(zz)]
        if not fin.size:
            continue
        with np.errstate(all="ignore"):
            tt = t[r, used] if tail else t[r, used] / tau
            big = np.abs(fin).max() + (0 if tail else np.abs(tt[np.isfinite(tt)]).max(initial=0))
            rr = 2.0 ** -21 * (4 + big)
            lq = zz - (fin.max() + np.log(np.exp(fin - fin.max()).sum()))
            q = np.exp(lq)
            lp = tt if tail else tt - (tt.max() + np.log(np.exp(tt - tt.max()).sum()))
            p = np.exp(lp)
            S = idx[r, used]
            pv = np.zeros(V)
            pv[S] = p
            rest = max(0.0, 1 - p.sum()) if tail else 0.0
            m = p > 0
            lt[r] = abs(wr) * tau * tau * rr * (p[m] * (4 + np.abs(lp[m]) + np.abs(lq[S][m]))).sum()
            d = rr * (q * (p.sum() + rest) + pv)
            if tail:
                other = np.ones(V, bool)
                other[S] = False
                qr = q[other].sum()
                if qr > 0:
                    slack = rr * rest + k * 2.0 ** -23
                    d[other] += q[other] / qr * slack
                    lt[r] += abs(wr) * tau * tau * slack * (4 + abs(np.log(max(rest, 1e-30))) + abs(np.log(qr)))
            dt[r] = abs(gr * wr) * tau * d
    return lt, dt


def _check(nv, z, idx, val, tau=1.0, tail=False, w=None, g=None, **kw):
    z64, i64, t64 = ref.to64(z), idx.cpu().numpy().astype(np.int64), ref.to64(val)
    w64 = None if w is None else ref.to64(w)
    g64 = None if g is None else ref.to64(g).reshape(-1)
    loss, dz = nv.distill_topk_loss_grad(z, idx, val, temperature=tau, tail=tail, row_weight=w, grad_loss=g, **kw)
    only = nv.distill_topk_loss(z, idx, val, temperature=tau, tail=tail, row_weight=w)
    back = nv.distill_topk_grad(z, idx, val, grad_loss=g, temperature=tau, tail=tail, row_weight=w)
    assert loss.dtype == torch.float32 and dz.dtype == z.dtype
    same = lambda a, b: torch.equal(torch.nan_to_num(a.float(), 7.5), torch.nan_to_num(b.float(), 7.5))  # noqa: E731
    assert same(loss, only) and same(dz, back)      # the same results whichever outputs are asked for
    rl, rd = ref.distill(z64, i64, t64, tau, tail, w64, g64)
    lt, dt = _tol(z64, i64, t64, tau, tail, w64, g64)
    gl, gd = ref.to64(loss), ref.to64(dz)
    assert np.array_equal(np.isfinite(gl), np.isfinite(rl)) and np.array_equal(np.isnan(gl), np.isnan(rl))
    fin = np.isfinite(rl)
    assert (np.abs(gl - rl)[fin] <= lt[fin] + 1e-37).all(), np.max((np.abs(gl - rl) / (lt + 1e-37))[fin])
    assert np.array_equal(np.isnan(gd), np.isnan(rd))
    ok = ~np.isnan(rd)
    if z.dtype == torch.bfloat16:
        dt = dt + 2.0 ** -8 * np.abs(np.nan_to_num(rd))
    assert (np.abs(gd - rd)[ok] <= dt[ok] + 1e-37).all(), np.max((np.abs(gd - rd) / (dt + 1e-37))[ok])
    return loss, dz


SIZES = [(1, 1, 1), (1, 2, 1), (2, 7, 3), (3, 8, 8), (2, 9, 4), (5, 31, 5), (3, 1000, 17), (2, 4097, 64),
         (7, 20001, 300), (400, 2053, 33), (2, 50001, 1024), (3, 131072, 100)]


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,V,k", SIZES)
def test_sizes(nv, T, V, k, dtype, tail):
    _check(nv, *_case(T, V, k, dtype, T + V + k, tail), tail=tail)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("tau", [0.5, 1.0, 3.0])
@pytest.mark.parametrize("tdtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
def test_types_and_temperature(nv, tail, tau, tdtype, itype):
    z, idx, val = _case(6, 3001, 40, torch.bfloat16, 11, tail, tau, tdtype)
    w = torch.tensor([1.0, 0.0, 0.25, 2.0, -1.0, 1e-3], device="cuda")
    g = torch.linspace(-1, 2, 6, device="cuda")
    _check(nv, z, idx.to(itype), val, tau, tail, w, g)
    _check(nv, z, idx.to(itype), val, tau, tail, w, torch.tensor([0.125], device="cuda"))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ld", [2003, 2008, 2051])
def test_strides_in_place_and_stream(nv, dtype, ld):
    z, idx, val = _case(9, 2001, 20, dtype, ld, ld=ld)
    loss, dz = _check(nv, z, idx, val)
    out = torch.empty(9, 2100, dtype=dtype, device="cuda")[:, 5:2006] if dtype == torch.float32 else \
        torch.empty(9, 2100, dtype=dtype, device="cuda")[:, 8:2009]
    if out.data_ptr() % 16 == 0:
        l2, d2 = nv.distill_topk_loss_grad(z, idx, val, out=out)
        assert d2 is out and torch.equal(d2, dz) and torch.equal(l2, loss)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        zc = z.clone()   # contiguous: other row alignments, so another order of summation
        l3, d3 = nv.distill_topk_loss_grad(zc, idx, val, out=zc)
    s.synchronize()
    loss, dz = _check(nv, z.contiguous(), idx, val)
    assert torch.equal(d3, dz) and torch.equal(l3, loss) and d3 is zc


def test_in_place_rows_of_odd_length(nv):
    for T, V in ((300, 999), (3, 150001)):
        z, idx, val = _case(T, V, 12, torch.bfloat16, 77)
        loss, dz = nv.distill_topk_loss_grad(z, idx, val)
        zc = z.clone()
        l2, d2 = nv.distill_topk_loss_grad(zc, idx, val, out=zc)
        assert torch.equal(loss, l2) and torch.equal(dz, d2)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_masked_rows_slots_and_logits(nv, dtype, tail):
    T, V, k = 10, 1500, 24
    z, idx, val = _case(T, V, k, dtype, 21, tail)
    nan, inf = float("nan"), float("inf")
    w = torch.ones(T, device="cuda")
    idx[0, 5:] = -1                      # few slots used
    val[0, 5:] = nan                     # unused values are not looked at
    idx[1] = -1                          # none used
    z[1, ::3] = nan
    w[2] = 0.0                           # weight 0: the logits are not looked at
    z[2, ::2] = inf
    z[2, 1::2] = nan
    val[3] = -inf                        # no mass at all
    val[4, 1:] = -inf                    # one entry has it all
    z[5, :700] = -inf                    # masked logits, some of them named
    low = torch.finfo(dtype).min
    z[6, 100:1400] = low
    z[7, 3] = nan
    z[8, 7] = inf
    z[9] = -inf
    loss, dz = _check(nv, z, idx, val, tail=tail, w=w)
    for r in (1, 2) + (() if tail else (3,)):
        assert loss[r] == 0 and not dz[r].any()
    for r in (7, 8, 9):
        assert torch.isnan(loss[r]) and torch.isnan(dz[r]).all()


def test_whole_vocabulary_named_has_no_rest(nv):
    z, idx, val = _case(4, 64, 64, torch.float32, 31, True)
    loss, _ = _check(nv, z, idx, val, tail=True)
    assert torch.isfinite(loss).all()


def test_student_that_rules_out_the_rest(nv):
    # the unnamed logits are 100 below: q_r = 1 - sum would have no digit
    z, idx, val = _case(3, 5000, 10, torch.float32, 41, True)
    keep = torch.zeros(3, 5000, dtype=torch.bool, device="cuda").scatter_(1, idx, True)
    z = torch.where(keep, z, z - 100.0)
    _check(nv, z, idx, val, tail=True)


def test_indices_beyond_the_vocabulary_are_reported(nv):
    z, idx, val = _case(3, 100, 4, torch.float32, 51)
    idx[1, 2] = 100
    idx[2, 0] = 1 << 40
    ws = nv.new_workspace(256)
    _check(nv, z, idx, val)
    assert nv.nvfp4_get_device_status(ws) == nv.OK
    nv.distill_topk_loss(z, idx, val, workspace=ws)
    assert nv.nvfp4_get_device_status(ws) == nv.ERR_INDEX
    assert nv.nvfp4_get_device_status(ws) == nv.OK
    assert "range" in nv.status_string(nv.ERR_INDEX)


@pytest.mark.parametrize("tail", [False, True])
def test_gradient_against_differences(nv, tail):
    """<dz, d> against central differences of the 64-bit loss: the quotient's own error is O(h^2) of the third
    derivative (<= tau^-1, |d| = 1) plus 2^-52 loss / h; dz's is its tolerance."""
    T, V, k, tau = 4, 300, 20, 1.5
    z, idx, val = _case(T, V, k, torch.float32, 61, tail, tau)
    _, dz = nv.distill_topk_loss_grad(z, idx, val, temperature=tau, tail=tail)
    z64, i64, t64 = ref.to64(z), idx.cpu().numpy(), ref.to64(val)
    _, dt = _tol(z64, i64, t64, tau, tail, None, None)
    rng = np.random.default_rng(0)
    h = 1e-4
    for _ in range(5):
        d = rng.standard_normal((T, V))
        d /= np.linalg.norm(d, axis=1, keepdims=True)
        up = ref.distill_loss(z64 + h * d, i64, t64, tau=tau, tail=tail)
        dn = ref.distill_loss(z64 - h * d, i64, t64, tau=tau, tail=tail)
        quotient = (up - dn) / (2 * h)
        got = (ref.to64(dz) * d).sum(1)
        assert (np.abs(got - quotient) <= (dt * np.abs(d)).sum(1) + 10 * h * h + 1e-11).all()


def test_largest_rows(nv):
    for dtype, V in ((torch.float32, 409568), (torch.bfloat16, 819136)):
        z, idx, val = _case(2, V, 50, dtype, 71, True)
        _check(nv, z, idx, val, tail=True)


def test_offsets_beyond_32_bits(nv):
    T, V, k = 20000, 120001, 8
    z = torch.zeros(T, V, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator("cuda").manual_seed(3)
    z[-3:] = torch.randn(3, V, device="cuda", generator=g).bfloat16()
    val, idx = torch.topk(torch.randn(T, 512, device="cuda", generator=g), k, dim=1)
    loss, dz = nv.distill_topk_loss_grad(z, idx, val)
    rl, rd = ref.distill(ref.to64(z[-3:]), idx[-3:].cpu().numpy(), ref.to64(val[-3:]))
    assert np.allclose(ref.to64(loss[-3:]), rl, rtol=1e-5)
    assert (np.abs(ref.to64(dz[-3:]) - rd) <= 2.0 ** -7 * np.abs(rd) + 1e-12).all()


def test_results_do_not_depend_on_scheduling(nv):
    z, idx, val = _case(64, 40000, 64, torch.bfloat16, 81, True)
    first = nv.distill_topk_loss_grad(z, idx, val, tail=True)
    for _ in range(5):
        again = nv.distill_topk_loss_grad(z, idx, val, tail=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_refusals(nv):
    z, idx, val = _case(2, 64, 4, torch.float32, 91)
    for bad in (dict(z=z.half()), dict(z=z.t()), dict(z=z.cpu()), dict(index=idx.float()), dict(teacher=val[:, :3]),
                dict(teacher=val.half())):
        kw = dict(z=z, index=idx, teacher=val) | bad
        with pytest.raises(ValueError):
            nv.distill_topk_loss_grad(**kw)
    with pytest.raises(ValueError):
        nv.distill_topk_loss(z, idx, val, row_weight=torch.ones(3, device="cuda"))
    with pytest.raises(ValueError):
        nv.distill_topk_loss_grad(z, idx, val, out=torch.empty(2, 64, dtype=torch.bfloat16, device="cuda"))
    for tau in (0.0, -1.0, float("nan"), float("inf"), 1e-40):
        with pytest.raises(nv.NVFP4Error) as e:
            nv.distill_topk_loss(z, idx, val, temperature=tau)
        assert e.value.status == nv.ERR_INVALID_ARG
    wide = torch.zeros(1, 409572, device="cuda")
    with pytest.raises(nv.NVFP4Error) as e:
        nv.distill_topk_loss(wide, idx[:1], val[:1])
    assert e.value.status == nv.ERR_SHAPE
    many = torch.zeros(2, 1025, dtype=torch.int32, device="cuda")
    with pytest.raises(nv.NVFP4Error) as e:
        nv.distill_topk_loss(z, many, many.float())
    assert e.value.status == nv.ERR_SHAPE
    with pytest.raises(nv.NVFP4Error) as e:
        nv.distill_topk_loss(z, idx, val, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == nv.ERR_WORKSPACE


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype,V,k", [(torch.bfloat16, 60001, 40), (torch.bfloat16, 150001, 64),
                                       (torch.float32, 40003, 300), (torch.float32, 131072, 992),
                                       (torch.float32, 25001, 1), (torch.bfloat16, 140000, 1000)])
def test_many_long_rows(nv, dtype, V, k, tail):
    """As many rows as SMs and more, rows longer than an SM's shared memory among them; masked rows, empty rows and
    unusual logits on the way.  Sampled rows against the definition, the others against the same rows alone."""
    T = 333
    z, idx, val = _case(T, V, k, dtype, V + k, tail)
    nan, inf = float("nan"), float("inf")
    w = torch.linspace(0.5, 2, T, device="cuda")
    w[::7] = 0.0
    z[7] = nan                                  # weight 0
    idx[8] = -1
    z[9, 5] = nan
    z[10, 17:V - 40] = -inf
    z[11] = torch.finfo(dtype).min
    z[12] = -inf
    if k > 1:
        idx[13, 1:] = -1
        val[13, 1:] = nan
        val[15, 1:] = -inf
    g = torch.linspace(-1, 1, T, device="cuda")
    loss, dz = nv.distill_topk_loss_grad(z, idx, val, tail=tail, row_weight=w, grad_loss=g)
    assert torch.equal(torch.nan_to_num(loss, 3.0),
                       torch.nan_to_num(nv.distill_topk_loss(z, idx, val, tail=tail, row_weight=w), 3.0))
    zc = z.clone()
    l2, d2 = nv.distill_topk_loss_grad(zc, idx, val, tail=tail, row_weight=w, grad_loss=g, out=zc)
    same = lambda a, b: torch.equal(torch.nan_to_num(a, 3.0), torch.nan_to_num(b, 3.0))  # noqa: E731
    assert same(l2, loss) and same(d2, dz)
    rows = [0, 1, 7, 8, 9, 10, 11, 12, 13, 15, 100, 153, 154, 305, 306, 331, 332]
    z64, i64, t64 = ref.to64(z[rows]), idx[rows].cpu().numpy(), ref.to64(val[rows])
    w64, g64 = ref.to64(w[rows]), ref.to64(g[rows])
    rl, rd = ref.distill(z64, i64, t64, 1.0, tail, w64, g64)
    lt, dt = _tol(z64, i64, t64, 1.0, tail, w64, g64)
    gl, gd = ref.to64(loss[rows]), ref.to64(dz[rows])
    assert np.array_equal(np.isnan(gl), np.isnan(rl)) and np.array_equal(np.isinf(gl), np.isinf(rl))
    fin = np.isfinite(rl)
    assert (np.abs(gl - rl)[fin] <= lt[fin] + 1e-37).all()
    assert np.array_equal(np.isnan(gd), np.isnan(rd))
    ok = ~np.isnan(rd)
    if dtype == torch.bfloat16:
        dt = dt + 2.0 ** -8 * np.abs(np.nan_to_num(rd))
    assert (np.abs(gd - rd)[ok] <= dt[ok] + 1e-37).all()


def test_many_long_rows_of_odd_stride(nv):
    z, idx, val = _case(200, 70001, 30, torch.bfloat16, 5, True, ld=70013)
    out = torch.empty(200, 70005, dtype=torch.bfloat16, device="cuda")[:, :70001]
    loss, dz = nv.distill_topk_loss_grad(z, idx, val, tail=True, out=out)
    rows = [0, 1, 2, 3, 5, 151, 152, 199]
    z64, i64, t64 = ref.to64(z[rows]), idx[rows].cpu().numpy(), ref.to64(val[rows])
    rl, rd = ref.distill(z64, i64, t64, 1.0, True)
    lt, dt = _tol(z64, i64, t64, 1.0, True, None, None)
    assert (np.abs(ref.to64(loss[rows]) - rl) <= lt).all()
    assert (np.abs(ref.to64(dz[rows]) - rd) <= dt + 2.0 ** -8 * np.abs(rd) + 1e-37).all()


@pytest.mark.parametrize("T,V,k", [(300, 60001, 64), (40, 32000, 8), (17, 999, 300)])
@pytest.mark.parametrize("tail", [False, True])
def test_loss_to_the_last_digits(nv, T, V, k, tail):
    """FP32 logits, loss alone: a logarithm is off by 2^-23 of its size at most, a share and a probability by 2^-21
    (sums of V terms over threads included), the rest's 1 - sum p by k 2^-24."""
    z, idx, val = _case(T, V, k, torch.float32, 77, tail=tail)
    loss, dz = nv.distill_topk_loss_grad(z, idx, val, tail=tail)
    z64, i64, t64 = ref.to64(z), idx.cpu().numpy().astype(np.int64), ref.to64(val)
    rl, rd = ref.distill(z64, i64, t64, 1.0, tail, None, None)
    lq = z64 - z64.max(1, keepdims=True)
    lq -= np.log(np.exp(lq).sum(1, keepdims=True))
    named = np.take_along_axis(lq, i64, 1)
    lp = t64 if tail else t64 - t64.max(1, keepdims=True)
    if not tail:
        lp = lp - np.log(np.exp(lp).sum(1, keepdims=True))
    p = np.exp(lp)
    tol = (p * (2.0 ** -23 * (np.abs(lp) + np.abs(named)) + 2.0 ** -21)).sum(1)
    if tail:
        pr, qr = 1 - p.sum(1), 1 - np.exp(named).sum(1)
        tol += pr * 2.0 ** -21 + (k * 2.0 ** -24) * (1 + np.abs(np.log(pr / qr)))
    assert (np.abs(ref.to64(loss) - rl) <= tol).all()
    # and the gradient as a whole (Euclidean norm): 2^-22 of its own
    d = ref.to64(dz) - rd
    assert np.sqrt((d * d).sum()) <= 2.0 ** -22 * np.sqrt((rd * rd).sum())


@pytest.mark.parametrize("offset", [0.0, 2700.0, -2900.0, 1.0e4, -1.0e6])
@pytest.mark.parametrize("T,V", [(5, 3001), (160, 50003)])
@pytest.mark.parametrize("tail", [False, True])
def test_logits_far_from_zero(nv, offset, T, V, tail):
    """A softmax does not see an offset.  Multiples of 1/16 keep their differences exactly beside it, so nothing may
    be lost: shares within 2^-19, logarithms within 2^-20 of a row's spread."""
    z, idx, val = _case(T, V, 20, torch.float32, 5, tail=tail)
    z = torch.round(z * 16) / 16
    z64 = ref.to64(z)
    loss, dz = nv.distill_topk_loss_grad(z + offset, idx, val, tail=tail)
    i64, t64 = idx.cpu().numpy().astype(np.int64), ref.to64(val)
    rl, rd = ref.distill(z64, i64, t64, 1.0, tail, None, None)
    q = np.exp(z64 - z64.max(1, keepdims=True))
    q /= q.sum(1, keepdims=True)
    p = np.exp(t64 if tail else t64 - t64.max(1, keepdims=True))
    p = p if tail else p / p.sum(1, keepdims=True)
    tol = 2.0 ** -19 * q
    np.put_along_axis(tol, i64, np.take_along_axis(tol, i64, 1) + 2.0 ** -19 * p, 1)
    rest = 2.0 ** -19 * np.maximum(0, 1 - p.sum(1, keepdims=True)) + 20 * 2.0 ** -23 if tail else 0.0
    qr = 1 - np.take_along_axis(q, i64, 1).sum(1, keepdims=True)
    assert (np.abs(ref.to64(dz) - rd) <= tol + rest * q / qr).all()
    spread = np.ptp(z64, axis=1) + np.abs(t64).max(1)
    assert (np.abs(ref.to64(loss) - rl) <= 2.0 ** -20 * (4 + spread)).all()
