"""Plain 64-bit definitions of the 4-bit activation operators and of the distillation loss (CPU, numpy).

Written from the definitions in include/nvfp4.h; shares no code with the library.
"""
import numpy as np
import torch

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def to64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def mx_encode(x):
    """x (rows, cols) float64 -> (codes (rows, cols) uint8, bytes (rows, cols/32) uint8), blocks along cols."""
    rows, cols = x.shape
    b = x.reshape(rows, cols // 32, 32)
    bad = ~np.isfinite(b).all(2)
    safe = np.where(bad[..., None], 0.0, b)
    amax = np.abs(safe).max(2)
    _, e = np.frexp(amax)                       # amax = f 2^e, f in [1/2, 1)
    byte = np.where(amax > 0, np.maximum(e - 1 - 2 + 127, 0), 0)
    mag = np.abs(safe) / np.exp2(byte - 127.0)[..., None]
    mid = (GRID[1:] + GRID[:-1]) / 2
    code = np.zeros(mag.shape, np.int64)
    for i, m in enumerate(mid):                 # tie to the even code
        code += (mag > m) | ((mag == m) & (i % 2 == 1))
    code |= np.signbit(safe) * 8
    code[bad] = 0
    byte = np.where(bad, 255, byte)
    return code.reshape(rows, cols).astype(np.uint8), byte.astype(np.uint8)


def mx_values(codes, byte):
    v = np.where(codes & 8, -1.0, 1.0) * GRID[codes & 7]
    s = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127))
    return (v.reshape(codes.shape[0], -1, 32) * s[..., None]).reshape(codes.shape)


def mx_round(x):
    return mx_values(*mx_encode(x))


def pack(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def unpack(packed):
    out = np.empty((packed.shape[0], packed.shape[1] * 2), np.uint8)
    out[:, 0::2], out[:, 1::2] = packed & 15, packed >> 4
    return out


def tile(byte):
    """Row-major scale bytes -> the documented tiles, index by index."""
    rows, nb = byte.shape
    kt = -(-nb // 4)
    out = np.zeros(-(-rows // 128) * kt * 512, np.uint8)
    r, j = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    out[((r // 128) * kt + j // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + j % 4] = byte
    return out


def pad_rows(x):
    return np.concatenate([x, np.zeros((-x.shape[0] % 32, x.shape[1]))])


def distill(z, idx, t, tau=1.0, tail=False, w=None, g=None):
    """(loss (T,), dz (T, V)) in float64, row by row, from the definition."""
    T, V = z.shape
    loss, dz = np.zeros(T), np.zeros((T, V))
    for r in range(T):
        wr = 1.0 if w is None else w[r]
        gr = 1.0 if g is None else g[r if len(g) == T else 0]
        used = [j for j in range(idx.shape[1]) if 0 <= idx[r, j] < V]
        if wr == 0 or not used:
            continue
        S, tv = idx[r, used], t[r, used]
        if not tail and (tv == -np.inf).all():
            continue
        with np.errstate(all="ignore"):
            zz = z[r] / tau
            m = zz.max()
            e = np.exp(zz - m)
            lse = m + np.log(e.sum())
            q = np.exp(zz - lse)
            if tail:
                logp = tv
                p = np.exp(tv)
                rest = max(0.0, 1.0 - p.sum()) if not np.isnan(p.sum()) else np.nan
                if len(S) == V:
                    rest = 0.0
            else:
                tt = tv / tau
                logp = tt - (tt.max() + np.log(np.exp(tt - tt.max()).sum()))
                p, rest = np.exp(logp), 0.0
            P = p.sum() + rest
            lr = 0.0
            for j in range(len(S)):
                if p[j] != 0:
                    lr += p[j] * (logp[j] - (zz[S[j]] - lse))
            d = q * P
            if rest != 0:
                other = np.ones(V, bool)
                other[S] = False
                qr = q[other].sum()
                lr += rest * (np.log(rest) - np.log(qr))
                if qr > 0:
                    d[other] -= rest * (q[other] / qr)
            d[S] = q[S] * P - p
            loss[r] = wr * tau * tau * lr
            dz[r] = gr * wr * tau * d
    return loss, dz


def distill_loss(z, idx, t, **kw):
    return distill(z, idx, t, **kw)[0]
