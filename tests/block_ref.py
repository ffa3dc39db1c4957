"""Plain 64-bit forms of the block operators, for the tests alone (CPU, numpy): the
dropout mask, the norms around a block and their backward pass, activations and their
derivatives. Beside each result stands a bound of what 32-bit arithmetic in any order
may be off: a magnitude (the same formula with every term's absolute value) times the
number of roundings on the longest way.
"""
import math

import numpy as np

EPS32 = 2.0 ** -24


def philox(counter, key):
    """Philox4x32-10 with Python's integers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def mask(rows, cols, p, seed, offset, row0=0):
    """The kept values' factors (rows, cols), zeros where a value is dropped."""
    lo = np.uint64(0xFFFFFFFF)
    n = -(-cols // 8)
    c = [np.broadcast_to(np.arange(n, dtype=np.uint64)[None, :], (rows, n)),
         np.broadcast_to(np.arange(row0, row0 + rows, dtype=np.uint64)[:, None], (rows, n)),
         np.full((rows, n), offset & 0xFFFFFFFF, np.uint64), np.full((rows, n), offset >> 32, np.uint64)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & lo, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & lo]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    u = np.stack([h for w in c for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], -1).reshape(rows, 8 * n)[:, :cols]
    t = round(65536 * p)
    return (u >= t) * (65536.0 / (65536 - t))


def statistics(v, layer, eps):
    """(mean, rstd, bound of the mean, relative bound of rstd), columns."""
    mean = v.mean(1, keepdims=True) if layer else np.zeros((v.shape[0], 1))
    rstd = 1.0 / np.sqrt(((v - mean) ** 2).mean(1, keepdims=True) + eps)
    # a lane sums up to 16 values, then 6 exchanges and up to 16 waves: 38 additions, and the division
    off = 40 * EPS32 * np.abs(v).mean(1, keepdims=True) if layer else np.zeros_like(mean)
    # squares of values that are off by `off`; half of the sum's relative error, the root's and the quotient's
    rel = 24 * EPS32 + rstd * off
    return mean, rstd, off, rel


def normalised(v, layer, eps, v_off=0.0):
    """hat and its bound; v itself is off by v_off."""
    mean, rstd, off, rel = statistics(v, layer, eps)
    hat = (v - mean) * rstd
    v_off = v_off + np.zeros_like(v)
    spread = rstd * (off + v_off + v_off.mean(1, keepdims=True) + 2 * EPS32 * (np.abs(v) + np.abs(mean)))
    shrink = np.abs(hat) * (rel + (np.abs(hat) * rstd * v_off).mean(1, keepdims=True) + 3 * EPS32)
    return hat, spread + shrink


def affine(v, off, w, b):
    w = 1.0 if w is None else w
    out = v * w + (0.0 if b is None else b)
    return out, np.abs(w) * off + 3 * EPS32 * (np.abs(v * w) + (0.0 if b is None else np.abs(b)))


def block_norm(x, y=None, *, layer=False, eps=1e-6, pre_w=None, pre_b=None, post=False, post_w=None, post_b=None, gate=None,
               alpha=1.0, m=1.0):
    """{"r", "n", "stats"} and their bounds; gate is a matrix by now (rows, cols)."""
    stats = np.zeros((x.shape[0], 4))
    s_off = np.zeros_like(stats)
    r, r_off = x, np.zeros_like(x)
    if y is not None:
        p, off = y, np.zeros_like(y)
        if post:
            mean, rstd, mo, ro = statistics(y, layer, eps)
            stats[:, :1], stats[:, 1:2], s_off[:, :1], s_off[:, 1:2] = mean, rstd, mo, ro * rstd
            p, off = affine(*normalised(y, layer, eps), post_w, post_b)
        g = alpha * m * (1.0 if gate is None else gate)
        r = x + g * p
        r_off = np.abs(g) * off + EPS32 * (np.abs(x) + 4 * np.abs(g * p))
    mean, rstd, mo, ro = statistics(r, layer, eps)
    hat, off = normalised(r, layer, eps, r_off)
    stats[:, 2:3], stats[:, 3:] = mean, rstd
    s_off[:, 2:3] = mo + r_off.mean(1, keepdims=True)
    s_off[:, 3:] = rstd * (ro + (np.abs(hat) * rstd * r_off).mean(1, keepdims=True))
    n, n_off = affine(hat, off, pre_w, pre_b)
    return {"r": r, "n": n, "stats": stats}, {"r": r_off, "n": n_off, "stats": s_off}


def block_norm_bwd(r, stats, dn=None, dr=None, y=None, *, layer=False, pre_w=None, post=False, post_w=None, post_b=None, gate=None,
                   alpha=1.0, m=1.0, group=None):
    """Gradients at the given r, y and stats, and their bounds. group: the gate row of every row."""
    rows, cols = r.shape
    n_add = 128 * EPS32   # of a row's sums (38 additions), products and differences, twice over
    col_add = (128 + rows) * EPS32
    t, t_off = np.zeros((rows, cols)), np.zeros((rows, cols))
    if dr is not None:
        t, t_off = dr, np.abs(dr) * n_add
    got, off = {}, {}

    def through(d, d_off, v, mean, rstd):
        hat, size = (v - mean) * rstd, (np.abs(v) + np.abs(mean)) * rstd
        avg = (lambda z: z.mean(1, keepdims=True))
        out = rstd * (d - (avg(d) if layer else 0.0) - hat * avg(d * hat))
        mag = rstd * (np.abs(d) + (avg(np.abs(d)) if layer else 0.0) + size * avg(np.abs(d) * size))
        more = rstd * (d_off + (avg(d_off) if layer else 0.0) + size * avg(d_off * size))
        return hat, size, out, mag * n_add + more

    if dn is not None:
        mean, rstd = stats[:, 2:3], stats[:, 3:]
        w = 1.0 if pre_w is None else pre_w
        hat, size, g, g_off = through(dn * w, EPS32 * np.abs(dn * w), r, mean, rstd)
        t, t_off = t + g, t_off + g_off + EPS32 * np.abs(t)
        got["dpre_w"], off["dpre_w"] = (dn * hat).sum(0), (np.abs(dn) * size).sum(0) * col_add
        got["dpre_b"], off["dpre_b"] = dn.sum(0), np.abs(dn).sum(0) * col_add
    got["dx"], off["dx"] = t, t_off
    if y is None:
        return got, off
    d, d_off = alpha * m * t, np.abs(alpha * m) * t_off + 2 * EPS32 * np.abs(alpha * m * t)
    p, p_off, size = y, np.zeros_like(y), None
    if post:
        mean, rstd = stats[:, :1], stats[:, 1:2]
        hat, size = (y - mean) * rstd, (np.abs(y) + np.abs(mean)) * rstd
        p, p_off = affine(hat, 2 * EPS32 * size, post_w, post_b)
    if gate is not None:
        n = int(group[-1]) + 1 if rows else 0
        got["dgate"], off["dgate"] = np.zeros((n, cols)), np.zeros((n, cols))
        np.add.at(got["dgate"], group, d * p)
        np.add.at(off["dgate"], group, d_off * np.abs(p) + np.abs(d) * p_off + col_add * np.abs(d * p))
        d, d_off = d * gate, d_off * np.abs(gate) + EPS32 * np.abs(d * gate)
    if post:
        got["dpost_w"], off["dpost_w"] = (d * hat).sum(0), (d_off * size + np.abs(d) * size * col_add).sum(0)
        got["dpost_b"], off["dpost_b"] = d.sum(0), (d_off + np.abs(d) * col_add).sum(0)
        w = 1.0 if post_w is None else post_w
        _, _, d, d_off = through(d * w, d_off * np.abs(w) + EPS32 * np.abs(d * w), y, mean, rstd)
    got["dy"], off["dy"] = d, d_off
    return got, off


# ------------------------------------------------------------- activations

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def sigmoid(u):
    e = np.exp(-np.abs(u))
    return np.where(u >= 0, 1.0, e) / (1.0 + e)


GELU_K = 2.0 * math.sqrt(2.0 / math.pi)


def act(z, kind):
    if kind == "relu":
        return np.maximum(z, 0.0)
    if kind == "gelu":
        return 0.5 * z * _erfc(-z / math.sqrt(2.0))
    if kind == "gelu_tanh":
        return z * sigmoid(GELU_K * (z + 0.044715 * z ** 3))
    if kind == "silu":
        return z * sigmoid(z)
    return z


def slope(z, kind):
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "gelu":
        return 0.5 * _erfc(-z / math.sqrt(2.0)) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        s = sigmoid(GELU_K * (z + 0.044715 * z ** 3))
        return s + z * s * sigmoid(-GELU_K * (z + 0.044715 * z ** 3)) * GELU_K * (1.0 + 3 * 0.044715 * z * z)
    if kind == "silu":
        return sigmoid(z) * (1.0 + z * sigmoid(-z))
    return np.ones_like(z)
