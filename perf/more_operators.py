"""Cases of the mixture-of-experts operators and of the 8-bit integer layer, with their plain forms.

Each case is a call (or the few calls in a row) that a user of the library makes: routing tokens to experts, the layer
grouped by expert on MXFP4 operands from one token up to a prefill batch, a training step of it, the weighted sum back to
the tokens with its gradient, and the layer whose weights and activations are 8-bit integers.  `own` chooses between the
library's kernels and elementary torch operations in 32 bits; `exact` is the definition in 64 bits.

The dense layers have the sizes of the Qwen2.5 projections that the benchmark and the tests use; experts have generic ones.
"""
import math

import torch

own = False

BLOCK = 32


# ---------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # routing of a decode step of four sequences: latency only
        dict(name="route_4x64", op="route", T=4, E=64, k=6, dtype="bf16", renormalise=True, grad=False),
        # routing of a training batch over many experts, with the gradient of the router's logits
        dict(name="route_16384x256", op="route", T=16384, E=256, k=8, dtype="fp32", renormalise=True, grad=True),
        # one token through its 8 of 128 experts
        dict(name="experts_1x8of128", op="experts", T=1, k=8, E=128, N=1536, K=4096, dtype="bf16", out="bf16"),
        # 64 concurrent sequences, 60 experts of odd width: a few ragged rows each, every expert's weights are read
        dict(name="experts_64x4of60", op="experts", T=64, k=4, E=60, N=2600, K=3584, dtype="bf16", out="fp32"),
        # prefill of 8192 tokens over 128 experts
        dict(name="experts_8192x8of128", op="experts", T=8192, k=8, E=128, N=1536, K=4096, dtype="bf16", out="bf16"),
        # a training step: plan, quantisers, forward, dX back at the tokens, dW of every expert
        dict(name="train_4096x4of32", op="train", T=4096, k=4, E=32, N=2048, K=2048, dtype="bf16", out="bf16", dw="fp32"),
        # a small one with an odd number of tokens, FP32 activations and gradients, few and ragged rows
        dict(name="train_333x2of7", op="train", T=333, k=2, E=7, N=1056, K=800, dtype="fp32", out="fp32", dw="fp32"),
        # the weighted sum of a decode step, added to the shared expert's output
        dict(name="combine_16x8", op="combine", T=16, k=8, E=64, N=4096, dtype="bf16", base=True, grad=False),
        # the weighted sum of a training batch and its gradients
        dict(name="combine_8192x8", op="combine", T=8192, k=8, E=128, N=4096, dtype="bf16", base=False, grad=True),
        # one token through the 7B up projection in 8 bits
        dict(name="int8_1_up", op="int8", M=1, N=18944, K=3584, dtype="bf16", out="bf16"),
        # a ragged batch of 100 tokens through the 7B down projection
        dict(name="int8_100_down", op="int8", M=100, N=3584, K=18944, dtype="bf16", out="fp32"),
        # prefill of 8192 tokens through the 7B up projection
        dict(name="int8_8192_up", op="int8", M=8192, N=18944, K=3584, dtype="bf16", out="bf16"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "train", "combine", "int8", "int8"])
    mult = lambda lo, hi: 32 * max(1, _log_uniform(rng, lo / 32, hi / 32))  # noqa: E731
    if op == "route":
        E = _log_uniform(rng, 4, 512)
        return dict(op=op, T=_log_uniform(rng, 1, 12000), E=E, k=rng.randint(1, min(E, 10)),
                    dtype=rng.choice(["bf16", "fp32"]), renormalise=rng.random() < 0.7, grad=rng.random() < 0.5)
    E = _log_uniform(rng, 2, 128)
    k = rng.randint(1, min(E, 8))
    if op == "experts":
        return dict(op=op, T=_log_uniform(rng, 1, 8192), k=k, E=E, K=mult(64, 4096),
                    N=rng.choice([_log_uniform(rng, 100, 1536), mult(128, 1536)]), dtype=rng.choice(["bf16", "fp32"]),
                    out=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "train":
        return dict(op=op, T=_log_uniform(rng, 16, 4096), k=min(k, 4), E=min(E, 32), N=mult(128, 2048), K=mult(128, 2048),
                    dtype=rng.choice(["bf16", "fp32"]), out=rng.choice(["bf16", "bf16", "fp32"]),
                    dw=rng.choice(["bf16", "fp32"]))
    if op == "combine":
        return dict(op=op, T=_log_uniform(rng, 1, 8192), k=k, E=E, N=rng.choice([_log_uniform(rng, 100, 4096), mult(128, 4096)]),
                    dtype=rng.choice(["bf16", "bf16", "fp32"]) if k <= 4 else "bf16", base=rng.random() < 0.5,
                    grad=rng.random() < 0.5)
    return dict(op=op, M=_log_uniform(rng, 1, 8192), N=rng.choice([_log_uniform(rng, 100, 18944), mult(128, 18944)]),
                K=mult(64, 3584), dtype=rng.choice(["bf16", "bf16", "fp32"]), out=rng.choice(["bf16", "bf16", "fp32"]))


_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 29)
    return g


def _activations(M, K, dtype, g):
    """N(0, 1) with a few strong channels, as hidden states have."""
    x = torch.randn(M, K, device="cuda", generator=g)
    strong = torch.randint(0, K, (max(1, K // 256),), device="cuda", generator=g)
    x[:, strong] *= 20.0
    return x.to(_DT[dtype])


def _logits(T, E, g):
    """Router logits: some experts are asked for more often than others."""
    return torch.randn(T, E, device="cuda", generator=g) * 1.5 + torch.randn(E, device="cuda", generator=g) * 0.7


def _experts(case, g):
    return torch.topk(_logits(case["T"], case["E"], g), case["k"], dim=1).indices.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    op, s = case["op"], dict(case)
    if op == "int8":
        s["x"] = _activations(case["M"], case["K"], case["dtype"], g)
        s["w_codes"], s["w_scales"] = _int8_plain(torch.randn(case["N"], case["K"], device="cuda", generator=g) * 0.02)
        s["workspace"] = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
        return s
    T, E, k = case["T"], case["E"], case["k"]
    if op == "route":
        s["logits"] = _logits(T, E, g).to(_DT[case["dtype"]])
        if case["grad"]:
            s["dweights"] = torch.randn(T, k, device="cuda", generator=g) * 1e-2
        return s
    s["experts"] = _experts(case, g)
    if op == "combine":
        N = case["N"]
        s["y"] = torch.randn(T * k, N, device="cuda", generator=g).to(_DT[case["dtype"]])
        s["weights"] = torch.softmax(torch.randn(T, k, device="cuda", generator=g), 1)
        s["base"] = torch.randn(T, N, device="cuda", generator=g).to(_DT[case["dtype"]]) if case["base"] else None
        if case["grad"]:
            s["dout"] = (torch.randn(T, N, device="cuda", generator=g) * 1e-3).to(_DT[case["dtype"]])
        return s
    N, K = case["N"], case["K"]
    s["x"] = _activations(T, K, case["dtype"], g)
    s["workspace"] = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    if op == "experts":
        packed = [_pack(*_mx_plain(torch.randn(N, K, device="cuda", generator=g) * 0.02)) for _ in range(E)]
        s["w_codes"], s["w_scales"] = torch.stack([c for c, _ in packed]), torch.stack([t for _, t in packed])
        return s
    s["w"] = (torch.randn(E, N, K, device="cuda", generator=g) * 0.02).to(_DT[case["dtype"]])
    # gradients at the experts' outputs, in the experts' order: small, some rows without any
    dy = torch.randn(T * k, N, device="cuda", generator=g) * 1e-3
    s["dy"] = (dy * (torch.rand(T * k, 1, device="cuda", generator=g) > 0.1)).to(_DT[case["dtype"]])
    return s


# ---------------------------------------------------------------------------------------------------- plain forms
_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _e2m1_round(v):
    """Nearest E2M1 magnitude of v >= 0, ties to the even code, at most 6."""
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0))
    return torch.clamp(torch.round(v / step) * step, max=6.0)


def _mx_plain(x):
    """(grid values, E8M0 bytes) of x quantised in blocks of 32 along the last axis."""
    x = x.float().reshape(x.shape[0], -1, BLOCK)
    byte = torch.clamp(((x.abs().amax(2).view(torch.int32) >> 23) & 255) - 2, min=0)
    v = torch.ldexp(x, (127 - byte)[..., None])
    return torch.copysign(_e2m1_round(v.abs()), x).reshape(x.shape[0], -1), byte.to(torch.uint8)


def _mx_values(x):
    grid, byte = _mx_plain(x)
    return torch.ldexp(grid.reshape(grid.shape[0], -1, BLOCK), (byte.int() - 127)[..., None]).reshape(grid.shape)


def _mx_values_cols(x):
    """The same along the first axis (zero rows appended to a multiple of 32)."""
    M = x.shape[0]
    xt = torch.nn.functional.pad(x, (0, 0, 0, -M % BLOCK)).t().contiguous()
    return _mx_values(xt)[:, :M].t()


def _pack(grid, scale_bytes):
    """Codes (rows x cols/2, even element in the low nibble) and scale bytes in tiles of 128 rows x 4 blocks: byte
    16 (r % 32) + 4 (r % 128 / 32) + j % 4 of tile (r / 128, j / 4), padding zero."""
    mags = torch.tensor(_GRID, device=grid.device)
    code = torch.bucketize(grid.abs(), mags).to(torch.uint8) | (torch.signbit(grid).to(torch.uint8) << 3)
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    rows, nb = scale_bytes.shape
    pad = torch.nn.functional.pad(scale_bytes, (0, -nb % 4, 0, -rows % 128))
    rt, kt = pad.shape[0] // 128, pad.shape[1] // 4
    return codes.contiguous(), pad.reshape(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).contiguous().reshape(-1)


def _mx_decode(codes, tiles):
    rows, cols = codes.shape[0], codes.shape[1] * 2
    nb = cols // BLOCK
    rt, kt = -(-rows // 128), -(-nb // 4)
    sb = tiles.reshape(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)[:rows, :nb]
    lut = torch.tensor(_GRID + tuple(-v for v in _GRID), device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), 2).reshape(rows, nb, BLOCK)
    return torch.ldexp(lut[c.int()], (sb.int() - 127)[..., None]).reshape(rows, cols)


def _int8_plain(x):
    """Codes and scales of the rows of x: amax / 127 a step, round to nearest even (ties are decided in 64 bits)."""
    amax = x.abs().amax(1).double()
    ratio = torch.where(amax > 0, 127.0 / amax, 0.0)[:, None]
    codes = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    for r in range(0, x.shape[0], 4096):
        p = x[r:r + 4096].double()
        codes[r:r + 4096] = torch.round(torch.where(ratio[r:r + 4096] > 0, p * 127.0 / amax[r:r + 4096, None], 0.0)).to(torch.int8)
    return codes, (amax.float() / 127.0)


def _group(experts, E):
    """Slots (t, j) in the order of their experts, the first slots first; the rows' beginnings of each expert; where the
    row of each slot is."""
    flat = experts.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    counts = (flat[None, :] == torch.arange(E, device=flat.device)[:, None]).sum(1)
    offsets = torch.cat((counts.new_zeros(1), torch.cumsum(counts, 0)))
    position = torch.empty_like(order)
    position[order] = torch.arange(order.numel(), device=flat.device)
    return order, offsets, position.reshape(experts.shape)


def _plain_route(s):
    z = s["logits"].float()
    vals, idx = torch.sort(z, dim=1, descending=True, stable=True)
    vals, idx = vals[:, :s["k"]], idx[:, :s["k"]]
    e = torch.exp(z - z.amax(1, keepdim=True))
    ek = torch.gather(e, 1, idx)
    w = ek / (ek if s["renormalise"] else e).sum(1, keepdim=True)
    order, offsets, _ = _group(idx, s["E"])
    out = {"weights": w, "experts": idx.to(torch.int32), "order": order.to(torch.int32), "offsets": offsets.to(torch.int32)}
    if s["grad"]:
        dw = s["dweights"]
        dot = (w * dw).sum(1, keepdim=True)
        if s["renormalise"]:
            dz = torch.zeros_like(z).scatter_(1, idx, w * (dw - dot))
        else:
            p = e / e.sum(1, keepdim=True)
            dz = (p * -dot).scatter_add_(1, idx, w * dw)
        out["dlogits"] = dz.to(s["logits"].dtype)
    return out


def _plain_combine(s):
    _, _, pos = _group(s["experts"], s["E"])
    T, k = pos.shape
    out = torch.zeros(T, s["N"], device=pos.device) if s["base"] is None else s["base"].float()
    for j in range(k):
        out = out + s["weights"][:, j:j + 1] * s["y"][pos[:, j]].float()
    res = {"out": out.to(s["y"].dtype)}
    if s["grad"]:
        do = s["dout"].float()
        dy = torch.empty_like(s["y"])
        dw = torch.empty(T, k, device=pos.device)
        for j in range(k):
            dy[pos[:, j]] = (s["weights"][:, j:j + 1] * do).to(dy.dtype)
            dw[:, j] = (do * s["y"][pos[:, j]].float()).sum(1)
        res.update(dy=dy, dweights=dw)
    return res


def _plain_experts(s):
    order, offsets, _ = _group(s["experts"], s["E"])
    xq = _mx_values(s["x"])
    y = torch.empty(order.numel(), s["N"], dtype=_DT[s["out"]], device=xq.device)
    at = offsets.tolist()
    for e in range(s["E"]):
        if at[e + 1] > at[e]:
            rows = order[at[e]:at[e + 1]] // s["k"]
            y[at[e]:at[e + 1]] = (xq[rows] @ _mx_decode(s["w_codes"][e], s["w_scales"][e]).t()).to(y.dtype)
    return {"y": y}


def _plain_train(s):
    order, offsets, pos = _group(s["experts"], s["E"])
    xq, dyq = _mx_values(s["x"]), _mx_values(s["dy"])
    R, (E, N, K) = order.numel(), s["w"].shape
    y = torch.empty(R, N, dtype=_DT[s["out"]], device=xq.device)
    dx = torch.empty(R, K, device=xq.device)
    dw = torch.zeros(E, N, K, dtype=_DT[s["dw"]], device=xq.device)
    at = offsets.tolist()
    for e in range(E):
        a, b = at[e], at[e + 1]
        if b > a:
            rows = order[a:b] // s["k"]
            y[a:b] = (xq[rows] @ _mx_values(s["w"][e]).t()).to(y.dtype)
            dx[a:b] = dyq[a:b] @ _mx_values_cols(s["w"][e])
            dw[e] = (_mx_values_cols(s["dy"][a:b]).t() @ _mx_values_cols(s["x"][rows])).to(dw.dtype)
    return {"y": y, "dx": dx[pos].sum(1).to(_DT[s["out"]]), "dw": dw}


def _plain_int8(s):
    q, sx = _int8_plain(s["x"])
    y = q.float() @ s["w_codes"].float().t()
    return {"y": (y * sx[:, None] * s["w_scales"][None, :]).to(_DT[s["out"]])}


# ---------------------------------------------------------------------------------------------------- one pass
_PLAIN = {"route": _plain_route, "combine": _plain_combine, "experts": _plain_experts, "train": _plain_train,
          "int8": _plain_int8}


def run(s):
    return _run_own(s) if own else _PLAIN[s["op"]](s)


def _run_own(s):
    from nvfp4_weight_only_02_gb300 import binding as nv
    op = s["op"]
    if op == "int8":
        w = nv.Int8Matrix(s["w_codes"], s["w_scales"])
        ws = _workspace(s, nv.nvfp4_int8_linear_workspace_bytes(s["M"], s["N"], s["K"]))
        return {"y": nv.int8_linear(s["x"], w, out_dtype=_DT[s["out"]], workspace=ws)}
    if op == "route":
        r = nv.moe_route(s["logits"], s["k"], renormalise=s["renormalise"])
        out = {"weights": r.weights, "experts": r.experts, "order": r.plan.order, "offsets": r.plan.offsets}
        if s["grad"]:
            out["dlogits"] = nv.moe_route_backward(s["dweights"], s["logits"], r)
        return out
    plan = nv.moe_plan(s["experts"], s["E"])
    if op == "combine":
        out = {"out": nv.moe_combine(s["y"], s["weights"], plan, base=s["base"])}
        if s["grad"]:
            out["dy"], out["dweights"] = nv.moe_combine_backward(s["dout"], s["y"], s["weights"], plan)
        return out
    if op == "experts":
        w = nv.MxExperts(s["w_codes"], s["w_scales"])
        ws = _workspace(s, nv.nvfp4_moe_linear_workspace_bytes(s["T"], s["k"], s["E"], s["N"], s["K"]))
        return {"y": nv.moe_linear(s["x"], w, plan, out_dtype=_DT[s["out"]], workspace=ws)}
    N, K = s["N"], s["K"]
    ws = _workspace(s, nv.nvfp4_moe_linear_backward_workspace_bytes(s["T"], s["k"], s["E"], N, K))
    x, w = nv.moe_quantize(s["x"], plan, colwise=True), nv.moe_quantize_weights(s["w"], colwise=True)
    y = nv.moe_gemm(x.row, w.row, plan, out_dtype=_DT[s["out"]], workspace=ws)
    dx, dw = nv.moe_linear_backward(s["dy"], x.col, w.col, plan, dw_dtype=_DT[s["dw"]], workspace=ws)
    return {"y": y, "dx": nv.moe_combine(dx, None, plan, out_dtype=_DT[s["out"]]), "dw": dw}


def _workspace(s, need):
    """The layer's workspace, kept between calls as a program keeps it; made larger when a call needs more."""
    if s["workspace"].numel() < need:
        s["workspace"] = torch.zeros(need, dtype=torch.uint8, device="cuda")
    return s["workspace"]


# ---------------------------------------------------------------------------------------------------- 64 bits
def _exact_mx(x):
    """Definition: shared exponent floor(log2 amax) - 2 (at least -127), nearest grid value by comparing with the
    midpoints, ties to the even code."""
    b = x.double().reshape(x.shape[0], -1, BLOCK)
    amax = b.abs().amax(2, keepdim=True)
    _, e = torch.frexp(amax)
    e = torch.where(amax > 0, (e - 1 - 2).double(), -127.0).clamp(min=-127.0)
    a = b.abs() / torch.exp2(e)
    r = torch.zeros_like(a)
    for mid, up, tie_up in ((0.25, 0.5, False), (0.75, 0.5, True), (1.25, 0.5, False), (1.75, 0.5, True),
                            (2.5, 1.0, False), (3.5, 1.0, True), (5.0, 2.0, False)):
        r += up * ((a >= mid) if tie_up else (a > mid))
    return (torch.sign(b) * r * torch.exp2(e)).reshape(x.shape)


def _exact_mx_cols(x):
    pad = torch.zeros(-x.shape[0] % BLOCK, x.shape[1], device=x.device, dtype=x.dtype)
    return _exact_mx(torch.cat((x, pad)).t().contiguous())[:, :x.shape[0]].t()


def _exact_decode(codes, tiles):
    rows, cols = codes.shape[0], 2 * codes.shape[1]
    c = torch.empty(rows, cols, dtype=torch.int64, device=codes.device)
    c[:, 0::2], c[:, 1::2] = (codes & 15).long(), (codes >> 4).long()
    mag = c & 7
    v = torch.where(mag < 2, mag * 0.5, (1 + 0.5 * (mag & 1)) * torch.exp2((mag >> 1).double() - 1))
    v = torch.where(c > 7, -v, v).double()
    r = torch.arange(rows, device=codes.device)[:, None]
    j = torch.arange(cols // BLOCK, device=codes.device)[None, :]
    kt = -(-(cols // BLOCK) // 4)
    byte = tiles[((r // 128) * kt + j // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + j % 4].long()
    return (v.reshape(rows, -1, BLOCK) * torch.exp2(byte.double() - 127)[..., None]).reshape(rows, cols)


def _slots(experts, E):
    """Per expert, its slots in ascending order."""
    flat = experts.reshape(-1)
    return [torch.nonzero(flat == e)[:, 0] for e in range(E)]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "int8":
        x = s["x"].double()
        amax = x.abs().amax(1, keepdim=True)
        q = torch.where(amax > 0, torch.round(127.0 * x / amax), 0.0)
        y = (q @ s["w_codes"].double().t()) * (amax / 127.0) * s["w_scales"].double()
        return {"y": y}
    if op == "route":
        return _exact_route(s)
    k, slots = case["k"], _slots(s["experts"], case["E"])
    order = torch.cat(slots)
    row = torch.empty_like(order)
    row[order] = torch.arange(order.numel(), device=order.device)
    row = row.reshape(case["T"], k)
    if op == "combine":
        return _exact_combine(s, row)
    if op == "experts":
        x = _exact_mx(s["x"])
        return {"y": torch.cat([x[i // k] @ _exact_decode(s["w_codes"][e], s["w_scales"][e]).t()
                                for e, i in enumerate(slots) if i.numel()])}
    x, dy = _exact_mx(s["x"]), _exact_mx(s["dy"])
    y, dx, dw, a = [], [], [], 0
    for e, i in enumerate(slots):
        b = a + i.numel()
        y.append(x[i // k] @ _exact_mx(s["w"][e]).t())
        dx.append(dy[a:b] @ _exact_mx_cols(s["w"][e]))
        dw.append(_exact_mx_cols(s["dy"][a:b]).t() @ _exact_mx_cols(s["x"][i // k]) if b > a
                  else torch.zeros(case["N"], case["K"], dtype=torch.float64, device=x.device))
        a = b
    return {"y": torch.cat(y), "dx": torch.cat(dx)[row].sum(1), "dw": torch.stack(dw)}


def _exact_route(s):
    z = s["logits"].double()
    T, E = z.shape
    k = s["k"]
    left = z.clone()
    idx = torch.empty(T, k, dtype=torch.int64, device=z.device)
    for j in range(k):
        best = left.amax(1, keepdim=True)
        idx[:, j] = torch.where(left == best, torch.arange(E, device=z.device), E).amin(1)
        left.scatter_(1, idx[:, j:j + 1], -math.inf)
    chosen = torch.zeros_like(z, dtype=torch.bool).scatter_(1, idx, True)
    p = torch.softmax(torch.where(chosen, z, -math.inf) if s["renormalise"] else z, 1)
    slots = _slots(idx, E)
    counts = torch.tensor([0] + [i.numel() for i in slots], device=z.device)
    out = {"weights": torch.gather(p, 1, idx), "experts": idx.to(torch.int32), "order": torch.cat(slots).to(torch.int32),
           "offsets": torch.cumsum(counts, 0).to(torch.int32)}
    if s["grad"]:
        up = torch.zeros_like(z).scatter_(1, idx, s["dweights"].double())
        out["dlogits"] = p * (up - (p * up).sum(1, keepdim=True))
    return out


def _exact_combine(s, row):
    T, k = row.shape
    out = torch.zeros(T, s["N"], dtype=torch.float64, device=row.device)
    if s["base"] is not None:
        out += s["base"]
    w = s["weights"].double()
    dy = torch.zeros(s["y"].shape, dtype=torch.float64, device=row.device) if s["grad"] else None
    dws = []
    for j in range(k):
        out.addcmul_(w[:, j, None], s["y"][row[:, j]].double())
        if s["grad"]:
            dy[row[:, j]] = w[:, j, None] * s["dout"].double()
            dws.append((s["dout"].double() * s["y"][row[:, j]].double()).sum(1))
    res = {"out": out}
    if s["grad"]:
        res.update(dy=dy, dweights=torch.stack(dws, 1))
    return res


# ---------------------------------------------------------------------------------------------------- work
def work(case):
    """Bytes: every input and output once, the weights of as many experts as can be asked for (what a training step
    quantises on its way counts once, as its 16- or 32-bit input).  Operations: multiplications and additions of the
    products; per element for the others."""
    op = case["op"]
    size = {"bf16": 2, "fp32": 4}
    d = size[case["dtype"]]
    if op == "int8":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * d + N * K + 4 * N + M * N * size[case["out"]], "flops": 2.0 * M * N * K}
    T, k, E = case["T"], case["k"], case["E"]
    R = T * k
    if op == "route":
        return {"bytes": T * E * d * (2 if case["grad"] else 1) + R * (12 + (4 if case["grad"] else 0)) + 4 * (E + 1),
                "flops": T * E * (6.0 if case["grad"] else 4.0)}
    N = case["N"]
    if op == "combine":
        b = R * N * d + T * N * d * (2 if case["base"] else 1) + R * 8
        if case["grad"]:
            b += T * N * d + R * N * d + R * 4
        return {"bytes": b, "flops": R * N * (5.0 if case["grad"] else 2.0)}
    K = case["K"]
    if op == "experts":
        return {"bytes": T * K * d + min(E, R) * N * K * 17 / 32 + R * N * size[case["out"]] + R * 4,
                "flops": 2.0 * R * N * K}
    o = size[case["out"]]
    return {"bytes": T * K * d + E * N * K * (d + size[case["dw"]]) + R * N * (d + o) + T * K * o + R * 4,
            "flops": 6.0 * R * N * K}
