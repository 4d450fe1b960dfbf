"""Plain 64-bit definitions of the mixture-of-experts operators (torch, any device), written from include/nvfp4.h."""
import torch

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def mx_round(x):
    """x (rows, cols), cols a multiple of 32, as its MXFP4 codes stand for it, float64."""
    b = x.double().reshape(x.shape[0], -1, 32)
    bad = ~torch.isfinite(b).all(2, keepdim=True)
    b = torch.where(bad, 0.0, b)
    amax = b.abs().amax(2, keepdim=True)
    e = torch.where(amax > 0, torch.frexp(amax)[1] - 3, -127).clamp(min=-127).double()
    a = b.abs() / torch.exp2(e)
    r = torch.zeros_like(a)
    for i in range(7):
        mid = (GRID[i] + GRID[i + 1]) / 2
        r += (GRID[i + 1] - GRID[i]) * ((a > mid) | ((a == mid) & (i % 2 == 1)))
    v = torch.sign(b) * r * torch.exp2(e)
    return torch.where(bad, torch.nan, v).reshape(x.shape)


def mx_round_rows(x):
    """The same with the blocks of 32 along the first axis; missing rows are zeros."""
    pad = torch.zeros(-x.shape[0] % 32, x.shape[1], dtype=x.dtype, device=x.device)
    return mx_round(torch.cat((x, pad)).t().contiguous())[:, :x.shape[0]].t()


def group(experts, E):
    """Rows of each expert as lists of slots, in ascending order."""
    flat = experts.reshape(-1).tolist()
    return [[s for s, e in enumerate(flat) if e == x] for x in range(E)]


def plan(experts, E):
    """(offsets, order with -1 behind the last row, position)."""
    slots = group(experts, E)
    n = experts.numel()
    order = [s for g in slots for s in g]
    offsets = [0]
    for g in slots:
        offsets.append(offsets[-1] + len(g))
    position = [-1] * n
    for r, s in enumerate(order):
        position[s] = r
    i = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return i(offsets), i(order + [-1] * (n - len(order))), i(position).reshape(experts.shape)


def route(z, k, scoring, renormalise, bias, scale):
    """(weights float64, experts) token by token."""
    T, E = z.shape
    w, ex = torch.zeros(T, k, dtype=torch.float64), torch.full((T, k), -1, dtype=torch.int32)
    for t in range(T):
        row = z[t].double()
        bad = bool(torch.isnan(row).any()) or (scoring == "softmax" and bool((row == torch.inf).any()))
        s = torch.sigmoid(row) if scoring == "sigmoid" else torch.softmax(torch.where(torch.isnan(row), -torch.inf, row), 0)
        choose = row if bias is None else s + bias.double()
        usable = [e for e in range(E) if row[e] > -torch.inf and choose[e] > -torch.inf]
        best = sorted(usable, key=lambda e: (-float(choose[e]), e))[:k]
        if best:
            taken = s[best]
            if renormalise:
                ln = torch.nn.functional.logsigmoid(row[best]) if scoring == "sigmoid" else row[best]
                taken = torch.softmax(ln, 0)
            w[t, :len(best)] = taken * scale
            ex[t, :len(best)] = torch.tensor(best, dtype=torch.int32)
        if bad:
            w[t] = torch.nan
    return w, ex


def combine(y, weights, position, base):
    T, k = position.shape
    out = torch.zeros(T, y.shape[1], dtype=torch.float64, device=y.device) if base is None else base.double()
    size = out.abs()
    for j in range(k):
        have = (position[:, j] >= 0)[:, None]
        rows = y[position[:, j].clamp(min=0).long()].double()
        w = torch.ones(T, 1, dtype=torch.float64, device=y.device) if weights is None else weights[:, j:j + 1].double()
        out = out + torch.where(have, w * rows, 0.0)
        size = size + torch.where(have, (w * rows).abs(), 0.0)
    return out, size
