"""The text cache's operators in plain float64 on the CPU, for the tests: no code of the library is used."""
import math

import numpy as np
import torch

GRIDS = {"mxfp8": (448.0, -6, 3), "mxfp4": (6.0, 0, 1)}     # largest value, lowest exponent, fraction bits


def quantise(x, fmt):
    """(values, scale bytes) of x [..., D] float64: each 32 values on their own grid.  None for bf16's scales."""
    x = np.asarray(x, np.float64)
    if fmt == "bf16":
        return torch.from_numpy(x).to(torch.float32).to(torch.bfloat16).double().numpy(), None
    top, low, frac = GRIDS[fmt]
    g = x.reshape(*x.shape[:-1], -1, 32)
    values, scales = np.empty_like(g), np.empty(g.shape[:-1], np.uint8)
    for at in np.ndindex(g.shape[:-1]):
        row = g[at]
        amax = np.max(np.abs(row))
        if not np.isfinite(amax):
            values[at], scales[at] = np.nan, 255
            continue
        e = -127
        while amax > math.ldexp(top, e):
            e += 1
        u = row / math.ldexp(1.0, e)
        ex = np.frexp(u)[1] - 1
        step = np.ldexp(1.0, np.maximum(ex, low) - frac)
        values[at] = np.round(u / step) * step * math.ldexp(1.0, e)     # numpy rounds halves to even
        scales[at] = e + 127
    return values.reshape(x.shape), scales


def code_value(code, fmt):
    """The value of one code, from its fields."""
    _, low, frac = GRIDS[fmt]
    bits = 8 if fmt == "mxfp8" else 4
    sign = -1.0 if code >> (bits - 1) else 1.0
    ex, m = (code & ((1 << (bits - 1)) - 1)) >> frac, code & ((1 << frac) - 1)
    if fmt == "mxfp8" and ex == 15 and m == 7:
        return math.nan
    return sign * (math.ldexp(m, low - frac) if ex == 0 else math.ldexp((1 << frac) + m, ex - 1 + low - frac))


def held(cache, fmt, name):
    """A pool's values [pages, heads, page_tokens, D] in float64."""
    raw = getattr(cache, name + "_pages").cpu()
    if fmt == "bf16":
        return raw.view(torch.bfloat16).double().numpy()
    raw = raw.numpy()
    table = np.array([code_value(c, fmt) for c in range(256 if fmt == "mxfp8" else 16)])
    u = table[raw] if fmt == "mxfp8" else table[np.stack((raw & 15, raw >> 4), -1).reshape(*raw.shape[:-1], -1)]
    s = getattr(cache, name + "_scales").cpu().numpy().astype(np.int64)
    f = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return u * np.repeat(f, 32, axis=-1)


def gather(pool, table_row, page_tokens, length):
    """Positions 0 .. length - 1 of one sequence: [heads, length, D]."""
    pages = [pool[table_row[i]] for i in range(-(-length // page_tokens))]
    if not pages:
        return np.zeros((pool.shape[1], 0, pool.shape[3]))
    return np.concatenate(pages, axis=1)[:, :length]


def attend(q, K, V, seen, prior=None):
    """One sequence: q [n, q_heads, D], K, V [heads, T, D], seen [n, T] bool, prior (out, m, l) or None.
    Returns out, m, l and, for tolerances, the softmax's sum of |p V| and the largest sum of |q K| / sqrt(D)."""
    n, qh, D = q.shape
    G = qh // K.shape[0]
    out, m, l = np.zeros((n, qh, D)), np.full((n, qh), -np.inf), np.zeros((n, qh))
    mag, smax = np.zeros((n, qh, D)), np.zeros((n, qh))
    for i in range(n):
        at = np.nonzero(seen[i])[0]
        for j in range(qh):
            k, v = K[j // G, at], V[j // G, at]
            with np.errstate(invalid="ignore", over="ignore"):
                s = k @ q[i, j] / math.sqrt(D)
                po = np.zeros(D) if prior is None else prior[0][i, j]
                pm, pl = (-np.inf, 0.0) if prior is None else (prior[1][i, j], prior[2][i, j])
                top = max(np.max(s) if len(s) else -np.inf, pm)
                if len(s) and np.isnan(s).any():
                    top = np.nan
                if top == -np.inf:
                    continue
                p, w = np.exp(s - top), math.exp(pm - top) * pl if pm > -np.inf else 0.0
                m[i, j], l[i, j] = top, p.sum() + w
                out[i, j] = (p @ v + w * po) / l[i, j]
                mag[i, j] = (p @ np.abs(v) + w * np.abs(po)) / l[i, j]
                smax[i, j] = np.max(np.abs(k) @ np.abs(q[i, j])) / math.sqrt(D) if len(s) else 0.0
    return out, m, l, mag, smax


def visible(n, length, words):
    """[n, length]: every token before the n newest, and of those the ones in a row's word (None: 0 .. i)."""
    seen = np.ones((n, length), bool)
    for i in range(n):
        for j in range(n):
            seen[i, length - n + j] = bool(int(words[i]) >> j & 1) if words is not None else j <= i
    return seen
