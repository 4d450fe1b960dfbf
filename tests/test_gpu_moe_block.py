"""A mixture-of-experts block as a program runs it: router, experts in 4 bits, a shared expert in 8 bits, the weighted sum,
and the backward pass of all but the shared expert, against 64-bit definitions; in CUDA graphs; on several streams."""
import pytest
import torch

from tests import moe_reference as ref
from tests.test_gpu_graph_fp4 import _replays

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


class Block:
    """out = shared(x) + sum over the k best experts of w_j * (W2_e relu(W1_e x))."""

    def __init__(self, nv, T, K, H, E, k, seed):
        g = torch.Generator("cuda").manual_seed(seed)
        self.nv, self.k, self.E = nv, k, E
        self.router = torch.randn(E, K, device="cuda", generator=g) / K ** 0.5
        self.w1 = torch.randn(E, H, K, device="cuda", generator=g) / K ** 0.5
        self.w2 = torch.randn(E, K, H, device="cuda", generator=g) / H ** 0.5
        self.shared = nv.int8_quantize(torch.randn(K, K, device="cuda", generator=g) / K ** 0.5)
        need = [nv.nvfp4_moe_gemm_workspace_bytes(T, k, E, H, K), nv.nvfp4_int8_linear_workspace_bytes(T, K, K),
                nv.nvfp4_moe_linear_workspace_bytes(T, k, E, H, K), nv.nvfp4_moe_linear_workspace_bytes(T, k, E, K, H),
                nv.nvfp4_moe_linear_backward_workspace_bytes(T, k, E, H, K),
                nv.nvfp4_moe_linear_backward_workspace_bytes(T, k, E, K, H)]
        self.ws = nv.new_workspace(max(need))
        self.q1, self.q2 = (nv.moe_quantize_weights(w, colwise=True) for w in (self.w1, self.w2))

    def serve(self, x):
        nv, ws = self.nv, self.ws
        r = nv.moe_route((x.float() @ self.router.t()), self.k)
        h = nv.moe_linear(x, self.q1.row, r.plan, workspace=ws).relu()
        y = nv.moe_linear(h, self.q2.row, r.plan, sorted_rows=True, workspace=ws)
        base = nv.int8_linear(x, self.shared, workspace=ws)
        return nv.moe_combine(y, r.weights, r.plan, base=base)

    def step(self, x, dout):
        """(out, gradients of the router's logits, of x through the experts, of both weights)."""
        nv, ws = self.nv, self.ws
        z = x.float() @ self.router.t()
        r = nv.moe_route(z, self.k)
        x1 = nv.moe_quantize(x, r.plan, colwise=True)
        h = nv.moe_gemm(x1.row, self.q1.row, r.plan, workspace=ws).relu()
        x2 = nv.moe_quantize(h, r.plan, colwise=True, sorted_rows=True)
        y = nv.moe_gemm(x2.row, self.q2.row, r.plan, workspace=ws)
        out = nv.moe_combine(y, r.weights, r.plan, base=nv.int8_linear(x, self.shared, workspace=ws))
        dy, dw = nv.moe_combine_backward(dout, y, r.weights, r.plan)
        dz = nv.moe_route_backward(dw, z, r)
        dh, dw2 = nv.moe_linear_backward(dy, x2.col, self.q2.col, r.plan, workspace=ws)
        dx, dw1 = nv.moe_linear_backward(dh * (h > 0), x1.col, self.q1.col, r.plan, workspace=ws)
        return out, dz, nv.moe_combine(dx, None, r.plan), dw1, dw2


@pytest.mark.parametrize("T,K,H,E,k", [(1, 256, 128, 8, 2), (40, 256, 288, 5, 3), (700, 512, 256, 4, 2)])
def test_block(nv, T, K, H, E, k):
    b = Block(nv, T, K, H, E, k, T)
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(T, K, device="cuda", generator=g).bfloat16()
    dout = torch.randn(T, K, device="cuda", generator=g)
    out, dz, dx, dw1, dw2 = b.step(x, dout)
    assert torch.equal(b.serve(x), out)
    # in 64 bits.  The quantisers between the products see values that differ by the FP32 sums' last digits, so near the
    # grid's borders a few of h, dy and dh take the other neighbour: 0.2 % of the largest value covers a code of each sum
    # (half a step of 1/4 relative to one of H >= 128 terms) and a relative error of 1e-4 beside it would show a wrong row.
    z = x.float() @ b.router.t()
    r = nv.moe_route(z, k)
    at, order = r.plan.offsets.tolist(), r.plan.order.long()
    pos, w = r.plan.position.long(), r.weights.double()
    xr = ref.mx_round(x)
    y = torch.zeros(T * k, K, dtype=torch.float64, device="cuda")
    h = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
    for e in range(E):
        rows = slice(at[e], at[e + 1])
        h[rows] = (xr[order[rows] // k] @ ref.mx_round(b.w1[e]).t()).relu()
        if at[e + 1] > at[e]:
            y[rows] = ref.mx_round(h[rows].float()) @ ref.mx_round(b.w2[e]).t()
    q = torch.round(x.double() * 127 / x.double().abs().amax(1, keepdim=True))
    base = (q @ b.shared.codes.double().t()) * (x.double().abs().amax(1, keepdim=True) / 127) * b.shared.scales.double()
    want = base + (w[:, :, None] * y[pos]).sum(1)
    near = lambda got, ref_, tol: (got.double() - ref_).abs().max() <= tol * ref_.abs().max()  # noqa: E731
    assert near(out, want, 2e-3)
    dy = torch.zeros_like(y)
    dy[pos.reshape(-1)] = (w[:, :, None] * dout.double()[:, None, :]).reshape(T * k, K)
    dwt = (dout.double()[:, None, :] * y[pos]).sum(2)
    u = w * (dwt - (w * dwt).sum(1, keepdim=True))
    # besides, weights (off by 2^-23 of 1) times dw are subtracted from one another in FP32: with a weight next to 1 the
    # difference is as small as their roundings, 4 of 2^-23 |dw| at most
    want = torch.zeros(T, E, dtype=torch.float64, device="cuda").scatter_(1, r.experts.long(), u)
    assert (dz.double() - want).abs().max() <= 5e-3 * want.abs().max() + 2.0 ** -21 * dwt.abs().max()
    dxr = torch.zeros(T * k, K, dtype=torch.float64, device="cuda")
    for e in range(E):
        rows = slice(at[e], at[e + 1])
        if at[e + 1] == at[e]:
            assert (dw1[e] == 0).all() and (dw2[e] == 0).all()
            continue
        dyf, hf = dy[rows].float(), h[rows].float()
        dh = (ref.mx_round(dyf) @ ref.mx_round_rows(b.w2[e])) * (hf > 0)
        assert near(dw2[e], ref.mx_round_rows(dyf).t() @ ref.mx_round_rows(hf), 5e-3)
        assert near(dw1[e], ref.mx_round_rows(dh.float()).t() @ ref.mx_round_rows(x[order[rows] // k]), 5e-3)
        dxr[rows] = ref.mx_round(dh.float()) @ ref.mx_round_rows(b.w1[e])
    assert near(dx, dxr[pos].sum(1), 5e-3)
    assert nv.nvfp4_get_device_status(b.ws) == nv.OK


@pytest.mark.parametrize("T", [1, 50, 600])
def test_captured(nv, T):
    K, H, E, k = 256, 160, 6, 2
    b = Block(nv, T, K, H, E, k, 3)
    g = torch.Generator("cuda").manual_seed(2)
    x = torch.randn(T, K, device="cuda", generator=g).bfloat16()
    dout = torch.randn(T, K, device="cuda", generator=g)
    _replays(lambda: (b.serve(x),) + b.step(x, dout), [x, dout],
             lambda i: [torch.randn(T, K, device="cuda", generator=g).bfloat16(), torch.randn(T, K, device="cuda", generator=g)])
    assert nv.nvfp4_get_device_status(b.ws) == nv.OK


@pytest.mark.parametrize("T", [1, 30, 300])
def test_blocks_on_three_streams(nv, T):
    """Launches of several streams share the SMs; each result is the one of the call alone."""
    K, H, E, k = 512, 256, 8, 2
    blocks = [Block(nv, T, K, H, E, k, s) for s in range(3)]
    x = torch.randn(T, K, device="cuda", generator=torch.Generator("cuda").manual_seed(4)).bfloat16()
    alone = [b.serve(x) for b in blocks]
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    got = [[] for _ in blocks]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(blocks[i].serve(x))
    torch.cuda.synchronize()
    for b, want, ys in zip(blocks, alone, got):
        assert nv.nvfp4_get_device_status(b.ws) == nv.OK
        for y in ys:
            assert torch.equal(y, want)


def test_combine_gradient_by_differences(nv):
    """The weighted sum is linear in the rows and in the weights: steps change it by what the gradients say."""
    g = torch.Generator("cuda").manual_seed(6)
    T, k, E, N = 30, 4, 7, 96
    plan = nv.moe_plan(torch.randint(-1, E, (T, k), device="cuda", generator=g, dtype=torch.int32), E)
    draw = lambda *s: torch.randint(-8, 9, s, device="cuda", generator=g).float() / 8  # noqa: E731
    y, w, dout = draw(T * k, N), draw(T, k), draw(T, N)
    dy, dw = nv.moe_combine_backward(dout, y, w, plan)
    rows = int(plan.offsets[-1])
    step_y, step_w = draw(T * k, N), draw(T, k)
    # multiples of 1/64 below 2^12: every sum is exact
    change = lambda a, b: ((nv.moe_combine(a, b, plan) - nv.moe_combine(y, w, plan)).double() * dout.double()).sum()  # noqa: E731
    assert change(y + step_y, w) == (dy[:rows].double() * step_y[:rows].double()).sum()
    assert change(y, w + step_w) == (dw.double() * step_w.double()).sum()
