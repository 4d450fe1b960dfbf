"""Cases of the 4-bit activation and distillation operators, with their plain forms.

Each case is a call that a user of the library makes: quantising activations to MXFP4, the W4A4 layer for one token up to
a prefill batch, one training step of such a layer, and the distillation loss against a teacher's top logits.  `own`
chooses between the library's kernels and elementary torch operations in 32 bits; `exact` is the definition in 64 bits.

Layer sizes are the Qwen2.5 projections that the benchmark and the tests use, or generic ones.
"""
import math

import torch

own = False

BLOCK = 32


# ---------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # a decode step's activations on their way into a 4-bit layer: latency only
        dict(name="quant_8x3584", op="quant", rows=8, cols=3584, dtype="bf16", both=False),
        # a training batch's activations, quantised along both axes (forward product and weight gradient)
        dict(name="quant_both_16384x3584", op="quant", rows=16384, cols=3584, dtype="bf16", both=True),
        # one token through the 7B up projection
        dict(name="linear_1_up", op="linear", M=1, N=18944, K=3584, dtype="bf16", out="bf16"),
        # 16 concurrent sequences through the 7B down projection (long contraction, few weight rows)
        dict(name="linear_16_down", op="linear", M=16, N=3584, K=18944, dtype="bf16", out="bf16"),
        # a ragged batch of 200 tokens through the 32B up projection
        dict(name="linear_200_up32", op="linear", M=200, N=27648, K=5120, dtype="bf16", out="bf16"),
        # prefill of 16384 tokens through the 7B up projection
        dict(name="linear_16384_up", op="linear", M=16384, N=18944, K=3584, dtype="bf16", out="bf16"),
        # the product on the library's NVFP4 format (blocks of 16, tensor scales): 2048 tokens, 7B down projection
        dict(name="nvfp4_gemm_2048_down", op="nvfp4_gemm", M=2048, N=3584, K=18944, out="bf16"),
        # one training step of the 7B up projection: both operands quantised, forward, dX and dW
        dict(name="train_4096_up", op="train", M=4096, N=18944, K=3584, dtype="bf16", out="bf16", dw="fp32"),
        # a small layer, an odd number of tokens, FP32 activations and gradients
        dict(name="train_777_small", op="train", M=777, N=1056, K=2048, dtype="fp32", out="fp32", dw="fp32"),
        # distillation of a few answer tokens, small vocabulary
        dict(name="distill_4x32000", op="distill", T=4, V=32000, k=8, dtype="bf16", tail=False, tau=1.0, grad=True,
             weights=False, index="int64", teacher="bf16"),
        # a training batch: loss and gradient, teacher's log-probabilities with the remaining mass as one more class
        dict(name="distill_4096x131072", op="distill", T=4096, V=131072, k=64, dtype="bf16", tail=True, tau=1.0, grad=True,
             weights=True, index="int64", teacher="fp32"),
        # evaluation (loss only) of FP32 logits, odd vocabulary
        dict(name="distill_eval_513x50001", op="distill", T=513, V=50001, k=100, dtype="fp32", tail=False, tau=2.0,
             grad=False, weights=True, index="int32", teacher="fp32"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "nvfp4_gemm", "train", "distill", "distill"])
    mult = lambda lo, hi: 32 * max(1, _log_uniform(rng, lo / 32, hi / 32))  # noqa: E731
    if op == "quant":
        return dict(op=op, rows=_log_uniform(rng, 1, 16384), cols=mult(64, 18944), dtype=rng.choice(["bf16", "fp32"]),
                    both=rng.random() < 0.5)
    if op == "linear":
        return dict(op=op, M=_log_uniform(rng, 1, 16384), N=rng.choice([_log_uniform(rng, 100, 18944), mult(128, 18944)]),
                    K=mult(64, 3584), dtype=rng.choice(["bf16", "fp32"]), out=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "nvfp4_gemm":
        return dict(op=op, M=_log_uniform(rng, 1, 4096), N=_log_uniform(rng, 100, 18944), K=mult(64, 8192),
                    out=rng.choice(["bf16", "bf16", "fp32"]))
    if op == "train":
        return dict(op=op, M=_log_uniform(rng, 16, 4096), N=mult(128, 8192), K=mult(128, 4096),
                    dtype=rng.choice(["bf16", "fp32"]), out=rng.choice(["bf16", "bf16", "fp32"]),
                    dw=rng.choice(["bf16", "fp32"]))
    T = _log_uniform(rng, 1, 2048)
    V = _log_uniform(rng, 1000, 131072)
    return dict(op=op, T=T, V=V, k=_log_uniform(rng, 1, 512), dtype=rng.choice(["bf16", "bf16", "fp32"]),
                tail=rng.random() < 0.5, tau=rng.choice([1.0, 1.0, 2.0, 0.7]), grad=rng.random() < 0.7,
                weights=rng.random() < 0.5, index=rng.choice(["int64", "int32"]), teacher=rng.choice(["fp32", "bf16"]))


_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    return g


def _activations(M, K, dtype, g):
    """N(0, 1) with a few strong channels, as hidden states have."""
    x = torch.randn(M, K, device="cuda", generator=g)
    strong = torch.randint(0, K, (max(1, K // 256),), device="cuda", generator=g)
    x[:, strong] *= 20.0
    return x.to(_DT[dtype])


def _weights(N, K, g):
    return torch.randn(N, K, device="cuda", generator=g) * 0.02


def _gradient(M, N, dtype, g):
    """Small, with the rows of masked tokens zero."""
    dy = torch.randn(M, N, device="cuda", generator=g) * 1e-3
    dy *= (torch.rand(M, 1, device="cuda", generator=g) > 0.1)
    return dy.to(_DT[dtype])


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case)
    if op == "quant":
        s["x"] = _activations(case["rows"], case["cols"], case["dtype"], g)
    elif op == "linear":
        s["x"] = _activations(case["M"], case["K"], case["dtype"], g)
        s["w_codes"], s["w_scales"] = _pack(*_mx_plain(_weights(case["N"], case["K"], g)))
        s["workspace"] = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    elif op == "nvfp4_gemm":
        for n, v in (("a", _activations(case["M"], case["K"], "bf16", g).float()),
                     ("w", _weights(case["N"], case["K"], g).to(torch.bfloat16).float())):
            grid, scale, ts = _nvfp4_plain(v)
            s[n + "_codes"], s[n + "_scales"] = _pack(grid, scale.to(torch.float8_e4m3fn).view(torch.uint8))
            s[n + "_ts"] = ts
        s["workspace"] = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    elif op == "train":
        s["x"] = _activations(case["M"], case["K"], case["dtype"], g)
        s["w"] = _weights(case["N"], case["K"], g).to(_DT[case["dtype"]])
        s["dy"] = _gradient(case["M"], case["N"], case["dtype"], g)
        s["workspace"] = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    else:
        _prepare_distill(s, case, g)
    return s


def _prepare_distill(s, case, g):
    T, V, k = case["T"], case["V"], min(case["k"], case["V"])
    z = torch.randn(T, V, device="cuda", generator=g) * 2.5
    t = torch.randn(T, V, device="cuda", generator=g).add_(z)
    if case["tail"]:
        t -= torch.logsumexp(t / case["tau"], 1, keepdim=True) * case["tau"]
        t /= case["tau"]
    val, idx = torch.topk(t, k, dim=1)
    del t
    # every tenth row has fewer entries than slots: nucleus-filtered teachers leave some unused
    some = (torch.rand(T, 1, device="cuda", generator=g) < 0.1) & (torch.arange(k, device="cuda")[None, :] >= max(1, k // 2))
    idx = torch.where(some, torch.full_like(idx, -1), idx)
    s["z"] = z.to(_DT[case["dtype"]])
    s["idx"] = idx.to(torch.int32 if case["index"] == "int32" else torch.int64)
    s["val"] = val.to(_DT[case["teacher"]])
    # prompt tokens carry no loss
    s["weight"] = (torch.rand(T, device="cuda", generator=g) > 0.15).float() / T if case["weights"] else None


# ---------------------------------------------------------------------------------------------------- plain forms
_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _e2m1_round(v):
    """Nearest E2M1 magnitude of v >= 0, ties to the even code, at most 6."""
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0))
    return torch.clamp(torch.round(v / step) * step, max=6.0)


def _mx_plain(x):
    """(grid values, E8M0 bytes) of x quantised in blocks of 32 along the last axis."""
    x = x.float().reshape(x.shape[0], -1, BLOCK)
    amax = x.abs().amax(2)
    byte = torch.clamp(((amax.view(torch.int32) >> 23) & 255) - 2, min=0)
    v = torch.ldexp(x, (127 - byte)[..., None])
    grid = torch.copysign(_e2m1_round(v.abs()), x)
    return grid.reshape(x.shape[0], -1), byte.to(torch.uint8)


def _mx_values(x):
    grid, byte = _mx_plain(x)
    return torch.ldexp(grid.reshape(grid.shape[0], -1, BLOCK), (byte.int() - 127)[..., None]).reshape(grid.shape)


def _mx_values_cols(x):
    """The same along the first axis (zero rows appended to a multiple of 32)."""
    M = x.shape[0]
    pad = -M % BLOCK
    xt = torch.nn.functional.pad(x, (0, 0, 0, pad)).t().contiguous()
    return _mx_values(xt)[:, :M].t()


def _nvfp4_plain(x):
    """(grid values, E4M3 scales, tensor scale) of x in blocks of 16."""
    ts = (x.abs().max() / 2688.0).reshape(1)
    b = x.reshape(x.shape[0], -1, 16)
    sc = torch.clamp(b.abs().amax(2) / (6 * ts), max=448.0).to(torch.float8_e4m3fn).float()
    eff = (sc * ts)[..., None]
    v = torch.where(eff > 0, b / eff, torch.zeros_like(b))
    return torch.copysign(_e2m1_round(v.abs()), b).reshape(x.shape), sc, ts


def _pack(grid, scale_bytes):
    """Codes (rows x cols/2, even element in the low nibble) and scale bytes in tiles of 128 rows x 4 blocks: byte
    16 (r % 32) + 4 (r % 128 / 32) + j % 4 of tile (r / 128, j / 4), padding zero."""
    mags = torch.tensor(_GRID, device=grid.device)
    code = torch.bucketize(grid.abs(), mags).to(torch.uint8) | (torch.signbit(grid).to(torch.uint8) << 3)
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    rows, nb = scale_bytes.shape
    pad = torch.nn.functional.pad(scale_bytes, (0, -nb % 4, 0, -rows % 128))
    rt, kt = pad.shape[0] // 128, pad.shape[1] // 4
    tiles = pad.reshape(rt, 4, 32, kt, 4).permute(0, 3, 2, 1, 4).contiguous().reshape(-1)
    return codes.contiguous(), tiles


def _unpack(codes, tiles, per_block):
    """(signed grid values, scale bytes rows x blocks) of packed operands."""
    rows, cols = codes.shape[0], codes.shape[1] * 2
    nb = cols // per_block
    rt, kt = -(-rows // 128), -(-nb // 4)
    sb = tiles.reshape(rt, kt, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, kt * 4)[:rows, :nb]
    lut = torch.tensor(_GRID + tuple(-v for v in _GRID), device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), 2).reshape(rows, cols)
    return lut[c.int()], sb


def _mx_decode(codes, tiles):
    grid, sb = _unpack(codes, tiles, BLOCK)
    return torch.ldexp(grid.reshape(grid.shape[0], -1, BLOCK), (sb.int() - 127)[..., None]).reshape(grid.shape)


def _nvfp4_decode(codes, tiles):
    grid, sb = _unpack(codes, tiles, 16)
    return (grid.reshape(grid.shape[0], -1, 16) * sb.view(torch.float8_e4m3fn).float()[..., None]).reshape(grid.shape)


def _plain_distill(s):
    z = s["z"].float() / s["tau"]
    T, V = z.shape
    used = s["idx"] >= 0
    idx = torch.where(used, s["idx"], torch.zeros_like(s["idx"])).long()
    t = s["val"].float()
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    lse = m + torch.log(total)
    logq = torch.gather(z, 1, idx) - lse
    if s["tail"]:
        logp = torch.where(used, t, -math.inf)
        p = torch.exp(logp)
        # unused slots point at entry 0, so members are counted, not overwritten
        member = torch.zeros(T, V, dtype=torch.int32, device=z.device).scatter_add_(1, idx, used.int()) > 0
        rest_p = torch.clamp(1 - p.sum(1, keepdim=True), min=0)
        rest_q = torch.where(member, 0.0, e).sum(1, keepdim=True) / total
        rest = torch.where(rest_p > 0, rest_p * (torch.log(rest_p) - torch.log(rest_q)), 0.0)
    else:
        tt = torch.where(used, t / s["tau"], -math.inf)
        logp = tt - torch.logsumexp(tt, 1, keepdim=True)
        p = torch.exp(logp)
    terms = torch.where(used & (p > 0), p * (logp - logq), 0.0)
    loss = terms.sum(1)
    mass = p.sum(1, keepdim=True)
    if s["tail"]:
        loss = loss + rest[:, 0]
        mass = mass + rest_p
    w = s["weight"] if s["weight"] is not None else torch.ones(T, device=z.device)
    out = {"loss": torch.where(w != 0, loss * w * s["tau"] ** 2, 0.0)}
    if s["grad"]:
        q = e / total
        dz = q * mass
        if s["tail"]:
            dz = torch.where(member, dz, q * (mass - rest_p / rest_q))
        dz.scatter_add_(1, idx, torch.where(used, -p, 0.0))
        dz = torch.where((w != 0)[:, None], dz * (w * s["tau"])[:, None], 0.0)
        out["dz"] = dz.to(s["z"].dtype)
    return out


# ---------------------------------------------------------------------------------------------------- one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_plain(s):
    op = s["op"]
    if op == "quant":
        out = {"rows": _mx_values(s["x"]).to(torch.bfloat16)}
        if s["both"]:
            out["cols"] = _mx_values_cols(s["x"]).to(torch.bfloat16).contiguous()
        return out
    if op == "linear":
        return {"y": (_mx_values(s["x"]) @ _mx_decode(s["w_codes"], s["w_scales"]).t()).to(_DT[s["out"]])}
    if op == "nvfp4_gemm":
        y = _nvfp4_decode(s["a_codes"], s["a_scales"]) @ _nvfp4_decode(s["w_codes"], s["w_scales"]).t()
        return {"y": (y * (s["a_ts"] * s["w_ts"])).to(_DT[s["out"]])}
    if op == "train":
        y = _mx_values(s["x"]) @ _mx_values(s["w"]).t()
        dx = _mx_values(s["dy"]) @ _mx_values_cols(s["w"])
        dw = _mx_values_cols(s["dy"]).t() @ _mx_values_cols(s["x"])
        return {"y": y.to(_DT[s["out"]]), "dx": dx.to(_DT[s["out"]]), "dw": dw.to(_DT[s["dw"]])}
    return _plain_distill(s)


def _run_own(s):
    from nvfp4_weight_only_02_gb300 import binding as nv
    op = s["op"]
    if op == "quant":
        q = nv.mx_quantize(s["x"], colwise=s["both"], values=True)
        return {"rows": q.values, "cols": q.values_t} if s["both"] else {"rows": q.values}
    if op == "linear":
        w = nv.MxOperand(s["w_codes"], s["w_scales"])
        ws = _workspace(s, nv.nvfp4_mx_linear_workspace_bytes(s["M"], s["N"], s["K"]))
        return {"y": nv.mx_linear(s["x"], w, out_dtype=_DT[s["out"]], workspace=ws)}
    if op == "nvfp4_gemm":
        a = nv.Nvfp4Operand(s["a_codes"], s["a_scales"], s["a_ts"])
        w = nv.Nvfp4Operand(s["w_codes"], s["w_scales"], s["w_ts"])
        ws = _workspace(s, nv.nvfp4_w4a4_workspace_bytes(s["M"], s["N"], s["K"]))
        return {"y": nv.w4a4_gemm(a, w, out_dtype=_DT[s["out"]], workspace=ws)}
    if op == "train":
        ws = _workspace(s, max(nv.nvfp4_w4a4_workspace_bytes(s["M"], s["N"], s["K"]),
                               nv.nvfp4_mx_linear_backward_workspace_bytes(s["M"], s["N"], s["K"])))
        x, w = nv.mx_quantize(s["x"], colwise=True), nv.mx_quantize(s["w"], colwise=True)
        y = nv.w4a4_gemm(x.row, w.row, out_dtype=_DT[s["out"]], workspace=ws)
        dx, dw = nv.mx_linear_backward(s["dy"], x.col, w.col, dx_dtype=_DT[s["out"]], dw_dtype=_DT[s["dw"]], workspace=ws)
        return {"y": y, "dx": dx, "dw": dw}
    if s["grad"]:
        loss, dz = nv.distill_topk_loss_grad(s["z"], s["idx"], s["val"], temperature=s["tau"], tail=s["tail"],
                                             row_weight=s["weight"])
        return {"loss": loss, "dz": dz}
    return {"loss": nv.distill_topk_loss(s["z"], s["idx"], s["val"], temperature=s["tau"], tail=s["tail"],
                                         row_weight=s["weight"])}


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


def _exact_decode(codes, tiles, per_block):
    rows, cols = codes.shape[0], 2 * codes.shape[1]
    c = torch.empty(rows, cols, dtype=torch.int64, device=codes.device)
    c[:, 0::2], c[:, 1::2] = (codes & 15).long(), (codes >> 4).long()
    mag = c & 7
    v = torch.where(mag < 2, mag * 0.5, (1 + 0.5 * (mag & 1)) * torch.exp2((mag >> 1).double() - 1))
    v = torch.where(c > 7, -v, v).double()
    r = torch.arange(rows, device=codes.device)[:, None]
    j = torch.arange(cols // per_block, device=codes.device)[None, :]
    kt = -(-(cols // per_block) // 4)
    byte = tiles[((r // 128) * kt + j // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + j % 4].long()
    if per_block == BLOCK:
        scale = torch.exp2(byte.double() - 127)
    else:
        scale = torch.where(byte >> 3 > 0, (8 + (byte & 7)).double() * torch.exp2((byte >> 3).double() - 10),
                            (byte & 7).double() * 2.0 ** -9)
    return (v.reshape(rows, -1, per_block) * scale[..., None]).reshape(rows, cols)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        out = {"rows": _exact_mx(s["x"])}
        if case["both"]:
            out["cols"] = _exact_mx_cols(s["x"]).contiguous()
        return out
    if op == "linear":
        return {"y": _exact_mx(s["x"]) @ _exact_decode(s["w_codes"], s["w_scales"], BLOCK).t()}
    if op == "nvfp4_gemm":
        y = _exact_decode(s["a_codes"], s["a_scales"], 16) @ _exact_decode(s["w_codes"], s["w_scales"], 16).t()
        return {"y": y * (s["a_ts"].double() * s["w_ts"].double())}
    if op == "train":
        return {"y": _exact_mx(s["x"]) @ _exact_mx(s["w"]).t(), "dx": _exact_mx(s["dy"]) @ _exact_mx_cols(s["w"]),
                "dw": _exact_mx_cols(s["dy"]).t() @ _exact_mx_cols(s["x"])}
    return _exact_distill(s)


def _exact_distill(s):
    T, V = s["z"].shape
    losses, grads = [], []
    for at in range(0, T, 512):
        rows = slice(at, min(T, at + 512))
        zt = s["z"][rows].double() / s["tau"]
        n = zt.shape[0]
        idx = s["idx"][rows].long()
        ok = idx >= 0
        spot = torch.where(ok, idx, V)  # unused slots go to a column of their own
        t = s["val"][rows].double()
        logq = torch.log_softmax(zt, 1)
        teach = torch.full((n, V + 1), -math.inf, dtype=torch.float64, device=zt.device)
        teach.scatter_(1, spot, t if s["tail"] else t / s["tau"])
        inside = torch.zeros(n, V + 1, dtype=torch.bool, device=zt.device).scatter_(1, spot, True)[:, :V]
        teach = teach[:, :V]
        p = torch.exp(teach) if s["tail"] else torch.softmax(teach, 1)
        q = torch.exp(logq)
        loss = torch.where(p > 0, p * (torch.log(p) - logq), 0.0).sum(1)
        dz = q * p.sum(1, keepdim=True) - p
        if s["tail"]:
            pr = torch.clamp(1 - p.sum(1, keepdim=True), min=0)
            qr = torch.where(inside, 0.0, q).sum(1, keepdim=True)
            loss += torch.where(pr > 0, pr * (torch.log(pr) - torch.log(qr)), 0.0)[:, 0]
            dz = dz + torch.where(inside, q * pr, q * pr - pr * q / qr)
        w = s["weight"][rows].double() if s["weight"] is not None else torch.ones(n, dtype=torch.float64, device=zt.device)
        losses.append(w * s["tau"] ** 2 * loss)
        if s["grad"]:
            grads.append(dz * (w * s["tau"])[:, None])
    out = {"loss": torch.cat(losses)}
    if s["grad"]:
        out["dz"] = torch.cat(grads)
    return out


# ---------------------------------------------------------------------------------------------------- work
def work(case):
    """Bytes: every input and output once (codes and scales of quantised data count as outputs where they are the
    operator's own).  Operations: multiplications and additions of the products; per element for the others."""
    op = case["op"]
    size = {"bf16": 2, "fp32": 4}
    if op == "quant":
        n = case["rows"] * case["cols"]
        dirs = 2 if case["both"] else 1
        return {"bytes": n * (size[case["dtype"]] + dirs * (17 / 32 + 2)), "flops": n * dirs * 4}
    if op in ("linear", "nvfp4_gemm"):
        M, N, K = case["M"], case["N"], case["K"]
        if op == "linear":
            b = M * K * size[case["dtype"]] + N * K * 17 / 32
        else:
            b = (M + N) * K * 9 / 16
        return {"bytes": b + M * N * size[case["out"]], "flops": 2.0 * M * N * K}
    if op == "train":
        M, N, K = case["M"], case["N"], case["K"]
        d, o = size[case["dtype"]], size[case["out"]]
        return {"bytes": (M * K + N * K + M * N) * d + (M * N + M * K) * o + N * K * size[case["dw"]],
                "flops": 6.0 * M * N * K}
    T, V = case["T"], case["V"]
    k = min(case["k"], V)
    b = T * V * size[case["dtype"]] * (2 if case["grad"] else 1)
    b += T * k * ((8 if case["index"] == "int64" else 4) + size[case["teacher"]]) + T * 4 * (2 if case["weights"] else 1)
    return {"bytes": b, "flops": T * V * (8.0 if case["grad"] else 4.0)}
