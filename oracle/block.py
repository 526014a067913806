"""A transformer block's norms and 8-bit products (oracle, test infrastructure only).

Definitions, in fp64:

* rms(v) = sqrt(mean(v^2) + eps); u = w_post b / rms(b); x' = rscale x + bscale g u; y = w_pre x' / rms(x');
  the gate g has one row per `gate_rows` consecutive tokens (0: one row for all);
* its gradient, from dy (of y) and dres (of x');
* 8-bit rows: scale max|v| / 127, codes rint(127 v / max|v|) with ties to even; a zero row has scale 0 and
  codes 0, a row with a non-finite value scale NaN and codes 0;
* the product of 8-bit rows with one scale per row on either side, a bias, and silu(gate) * up.
"""

import numpy as np


def _f64(v):
    return None if v is None else np.asarray(v, dtype=np.float64)


def gate_per_token(gate, gate_rows, rows):
    """The gate of every token, rows x n."""
    gate = _f64(gate)
    per = gate_rows if gate_rows else max(rows, 1)
    return gate[np.arange(rows) // per]


def inverse_rms(v, eps):
    return 1.0 / np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps)


def block_norm(eps, branch=None, resid=None, w_post=None, gate=None, gate_rows=0, bscale=1.0, rscale=1.0, w_pre=None):
    """(x', y, inverse rms of b and of x' as a rows x 2 array); y is None without w_pre."""
    b, x, wp, wq = _f64(branch), _f64(resid), _f64(w_post), _f64(w_pre)
    rows = (b if b is not None else x).shape[0]
    r1 = np.ones((rows, 1))
    out = 0.0 if x is None else rscale * x
    if b is not None:
        u = b
        if wp is not None:
            r1 = inverse_rms(b, eps)
            u = wp * b * r1
        if gate is not None:
            u = u * gate_per_token(gate, gate_rows, rows)
        out = out + bscale * u
    r2 = np.ones((rows, 1)) if wq is None else inverse_rms(out, eps)
    return out, None if wq is None else wq * out * r2, np.concatenate([r1, r2], axis=1)


def block_norm_backward(eps, branch=None, resid=None, w_post=None, gate=None, gate_rows=0, bscale=1.0, rscale=1.0,
                        w_pre=None, dy=None, dres=None):
    """Gradients of sum(y dy) + sum(x' dres): a dict with dbranch, dresid, dw_post, dgate, dw_pre (None where
    there is no such input)."""
    b, wp, wq, dy = _f64(branch), _f64(w_post), _f64(w_pre), _f64(dy)
    out, _, stats = block_norm(eps, branch, resid, w_post, gate, gate_rows, bscale, rscale, w_pre)
    rows, n = out.shape
    r1, r2 = stats[:, :1], stats[:, 1:]
    g = np.zeros((rows, n)) if dres is None else _f64(dres).copy()
    res = dict.fromkeys(("dbranch", "dresid", "dw_post", "dgate", "dw_pre"))
    if dy is not None:
        xn = out * r2
        d = dy * wq
        g += r2 * (d - xn * np.mean(d * xn, axis=1, keepdims=True))
        res["dw_pre"] = np.sum(dy * xn, axis=0)
    if resid is not None:
        res["dresid"] = rscale * g
    if b is not None:
        bn = b * r1
        u = bn if wp is None else wp * bn
        gu = bscale * g
        if gate is not None:
            per = gate_rows if gate_rows else max(rows, 1)
            res["dgate"] = np.zeros(_f64(gate).shape)
            np.add.at(res["dgate"], np.arange(rows) // per, gu * u)
            gu = gu * gate_per_token(gate, gate_rows, rows)
        if wp is None:
            res["dbranch"] = gu
        else:
            res["dw_post"] = np.sum(gu * bn, axis=0)
            e = gu * wp
            res["dbranch"] = r1 * (e - bn * np.mean(e * bn, axis=1, keepdims=True))
    return res


def quant_rows_i8(v):
    """(codes, scales) of each row of v."""
    v = _f64(v)
    codes, scales = np.zeros(v.shape), np.zeros(v.shape[0])
    for r, row in enumerate(v):
        if not np.all(np.isfinite(row)):
            scales[r] = np.nan
            continue
        top = np.max(np.abs(row))
        scales[r] = top / 127.0
        if top > 0:
            codes[r] = np.rint(127.0 * row / top)
    return codes.astype(np.int8), scales


def matmul_i8(x, x_scales, w, w_scales, bias=None, swiglu=False):
    """z = x_scales w_scales (x w^T) + bias; with swiglu silu(first half of z) * second half."""
    sums = _f64(x) @ _f64(w).T  # whole numbers far below 2^53: exact
    z = sums * _f64(x_scales)[:, None] * _f64(w_scales)[None]
    if bias is not None:
        z = z + _f64(bias)[None]
    if not swiglu:
        return z
    gate, up = z[:, :z.shape[1] // 2], z[:, z.shape[1] // 2:]
    with np.errstate(over="ignore"):
        return gate / (1.0 + np.exp(-gate)) * up
