"""Rotary positions, the 4-bit cache of keys and values, attention over it and low-rank adapters, in fp64.

Definitions (include/wringer.h, part (i)); the pages describe none of these operators, so the pins in
tests/test_oracle_attention.py are closed forms and explicit loops.
"""
import numpy as np


def rotary(x, positions, freqs, dim, axis_of=None, interleaved=False, inverse=False):
    """x: rows x heads * dim; positions: axes x rows; pair i turns by positions[axis_of[i]] * freqs[i]."""
    x = np.asarray(x, np.float64)
    positions = np.atleast_2d(positions)
    y = x.reshape(x.shape[0], -1, dim).copy()
    pairs = len(freqs)
    for i in range(pairs):
        axis = 0 if axis_of is None else int(axis_of[i])
        if not 0 <= axis < positions.shape[0]:
            continue
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, pairs + i)
        z = (y[:, :, a] + 1j * y[:, :, b]) * np.exp((-1j if inverse else 1j) * positions[axis].astype(np.float64) * freqs[i])[:, None]
        y[:, :, a], y[:, :, b] = z.real, z.imag
    return y.reshape(x.shape)


def kv_codes(x, group):
    """(codes, scales, offsets) of rows of x (fp32 values), groups of `group` along the last axis."""
    x = np.asarray(x, np.float32)
    t = x.reshape(*x.shape[:-1], -1, group)
    bad = ~np.isfinite(t).all(-1)
    t = np.clip(np.where(bad[..., None], np.float32(0), t), np.float32(-65024), np.float32(65024))
    off = t.min(-1).astype(np.float16)
    d = t - off.astype(np.float32)[..., None]
    scale = (d.max(-1) / np.float32(15)).astype(np.float16)
    s = scale.astype(np.float32)[..., None]
    codes = np.where(s > 0, np.clip(np.rint(d / np.where(s > 0, s, np.float32(1))), 0, 15), 0).astype(np.uint8)
    scale[bad] = off[bad] = np.nan
    codes[bad] = 0
    return codes.reshape(x.shape), scale, off


def kv_values(codes, scale, off, group):
    c = codes.reshape(*codes.shape[:-1], -1, group).astype(np.float64)
    return (off.astype(np.float64)[..., None] + scale.astype(np.float64)[..., None] * c).reshape(codes.shape)


def kv_page(k, v, group, page):
    """The bytes of a page from k and v: page x heads x dim."""
    _, heads, dim = k.shape
    out = []
    for h in range(heads):
        kc, ks, ko = kv_codes(k[:, h], group)
        vc, vs, vo = kv_codes(v[:, h], group)
        keys = np.zeros((page, 4, dim // 32, 4), np.uint8)
        for d in range(dim):
            s, g, n = d // 32, d % 32 // 8, d % 8
            keys[:, g, s, n // 2] |= kc[:, d] << (4 * (n % 2))
        values = np.zeros((page // 16, 4, 16, dim // 32, 4), np.uint8)
        for t in range(page):
            for d in range(dim):
                values[t // 16, t % 16 // 4, d % 16, d % (dim // 2) // 16, t % 4] |= vc[t, d] << (4 * (d // (dim // 2)))
        kmeta = np.stack([ks.T, ko.T], -1)
        vmeta = np.zeros((dim // group, page // 4, 2, 2, 2), np.float16)  # odd token, scale or offset, later pair
        for t in range(page):
            vmeta[:, t // 4, t % 2, 0, t % 4 // 2], vmeta[:, t // 4, t % 2, 1, t % 4 // 2] = vs[t], vo[t]
        out += [keys.ravel(), values.ravel(), kmeta.view(np.uint8).ravel(), vmeta.view(np.uint8).ravel()]
    return np.concatenate(out)


def attend(q, k, v, sees, scale):
    """(out, weights) of q (rows x dim) over k, v (tokens x dim); sees: rows x tokens.  A row that sees nothing: 0."""
    z = scale * (q @ np.where(sees.any(0)[:, None], k, 0).T)
    z = np.where(sees, z, -np.inf)
    top = z.max(1, keepdims=True, initial=-np.inf)
    w = np.exp(z - np.where(np.isneginf(top), 0, top))
    w = np.where(sees, w, 0)
    den = w.sum(1, keepdims=True)
    w = np.where(den == 0, 0, w / np.where(den == 0, 1, den))
    out = np.zeros((q.shape[0], v.shape[1]))
    for r in range(q.shape[0]):
        out[r] = w[r, sees[r]] @ v[sees[r]]
    return out, w


def sees(first, count, length, causal=True, window=0):
    """count x length: what the queries at positions first .. first + count - 1 see."""
    p = first + np.arange(count)[:, None]
    t = np.arange(length)[None]
    ok = (t <= p) if causal else np.ones((count, length), bool)
    if window:
        ok = ok & (t > p - window) & (t < p + window)
    return ok


def adapters(x, base, A, B, scales, starts, ids, ranks=None):
    """y for the rows of the requests; base: rows x outs."""
    y = np.array(base, np.float64)
    for i, a in enumerate(ids):
        if 0 <= a < len(A):
            r = A.shape[1] if ranks is None else min(max(int(ranks[a]), 0), A.shape[1])
            rows = slice(starts[i], starts[i + 1])
            y[rows] += scales[a] * (np.asarray(x, np.float64)[rows] @ A[a, :r].T) @ B[a, :, :r].T
    return y
