"""GPU parity of the block norm, its gradient and the 8-bit products against the fp64 oracle.

Error bounds, derived from the kernels' fp32 arithmetic with eps32 = 2^-24 (half a unit in the last place,
relative) and sums of n values of at most 32 serial steps per lane, 6 across a wave and 16 across waves:

* sums of squares: relative error <= (32 + 6 + 16 + 2) eps32, so an inverse rms <= 28 + 3 -> 32 eps32;
* x': |error| <= eps32 (40 |bscale g u| + 4 |rscale x|);
* y: the error of x' in place, its share in rms(x') (at most the norm of x's error over the norm of x') and
  40 eps32 more;
* gradients: K eps32 times the same formula on magnitudes (|x'| replaced by |rscale x| + |bscale g u|).  xn is off
  by 40 + 32 + 60 (the last the share of x's error in rms(x'), with magnitudes at most 1.5 times x' in these inputs),
  mean(d xn) by 190 (a sum: 56), dx' by 325, mean(e bn) by 325 + 5 + 33 + 56 and dbranch by 490: K = 512; sums over
  tokens add one per token;
* outputs in bf16: 2^-8 more, relative.

Codes and scales of wr_quant_rows_i8 and the integer sums are exact.
"""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

E32, E16 = 2.0 ** -24, 2.0 ** -8
BF16, F32 = torch.bfloat16, torch.float32
CANARY = 77.0


@pytest.fixture(scope="module")
def wr():
    from post_bit_weight_amd import _lib
    return _lib


@pytest.fixture(scope="module")
def ctx(wr):
    return wr.Context(0)


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


class Padded:
    """A rows x n GPU matrix inside a larger buffer whose other values are checked afterwards."""

    def __init__(self, rows, n, dtype, pad=0, shift=0, value=None):
        self.full = torch.full((rows * (n + pad) + shift + 8,), CANARY, device="cuda").to(dtype)
        self.view = self.full[shift:shift + rows * (n + pad)].view(rows, n + pad)[:, :n]
        if value is not None:
            self.view.copy_(value)
        self.shift, self.rows, self.n, self.pad = shift, rows, n, pad

    def untouched(self):
        mask = torch.ones_like(self.full, dtype=torch.bool)
        mask[self.shift:self.shift + self.rows * (self.n + self.pad)].view(self.rows, self.n + self.pad)[:, :self.n] = False
        return bool((self.full[mask].float() == CANARY).all())


def round_err(dtype):
    return E16 if dtype == BF16 else E32


def norm_inputs(seed, rows, n, b_type, r_type, w_type, post, gate_rows, resid, pre, pad, shift):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    inp = dict(branch=Padded(rows, n, b_type, pad, shift, 2 * rnd(rows, n)).view)
    if resid:
        inp["resid"] = Padded(rows, n, r_type, pad, shift, 3 * rnd(rows, n)).view
    if post:
        inp["w_post"] = (1 + 0.3 * rnd(n)).to(w_type).cuda()
    if pre:
        inp["w_pre"] = (1 + 0.3 * rnd(n)).to(w_type).cuda()
    if gate_rows is not None:
        gates = -(-rows // gate_rows) if gate_rows else 1
        inp["gate"] = Padded(gates, n, b_type, pad, 0, rnd(gates, n)).view
        inp["gate_rows"] = gate_rows
    return inp


def host(inp):
    return {k: f64(v) if torch.is_tensor(v) else v for k, v in inp.items()}


def norm_bounds(h, eps, bscale, rscale):
    """(x', y, stats, error of x' before its rounding, of y before its rounding) in fp64."""
    out, y, stats = oracle.block_norm(eps, **h, bscale=bscale, rscale=rscale)
    zero = {k: v for k, v in h.items() if k != "resid"}
    branch = np.abs(oracle.block_norm(eps, **{**zero, "w_pre": None}, bscale=bscale)[0])
    x = 0.0 if h.get("resid") is None else np.abs(rscale * h["resid"])
    ex = E32 * (40 * branch + 4 * x)
    ey = None
    if y is not None:
        share = np.linalg.norm(ex, axis=1, keepdims=True) / np.maximum(np.linalg.norm(out, axis=1, keepdims=True), 1e-300)
        ey = np.abs(h["w_pre"]) * stats[:, 1:] * ex + np.abs(y) * (share + 40 * E32)
    return out, y, stats, ex, ey


NORM_CASES = [  # rows, n, branch type, residual type, weight type, post, gate_rows (None: no gate), resid, pre, pad, shift
    (1, 2560, BF16, BF16, BF16, True, 0, True, True, 0, 0),
    (37, 2560, BF16, F32, F32, True, 5, True, True, 8, 0),
    (5, 1, F32, F32, F32, True, 0, True, True, 0, 1),
    (9, 7, BF16, BF16, F32, True, 2, True, True, 1, 1),
    (70, 128, BF16, BF16, BF16, False, None, True, True, 0, 0),
    (33, 129, F32, F32, BF16, True, 1, True, True, 3, 3),
    (21, 257, BF16, BF16, BF16, True, 4, True, True, 0, 3),
    (6, 512, F32, BF16, F32, True, None, True, True, 0, 0),
    (7, 513, BF16, F32, BF16, False, 0, True, True, 5, 1),
    (3, 4097, BF16, BF16, BF16, True, 2, True, True, 1, 0),
    (4, 9727, F32, F32, F32, True, 3, True, True, 5, 1),
    (2, 16384, BF16, BF16, BF16, True, 0, True, True, 0, 0),
    (3, 16383, F32, F32, F32, True, 0, True, False, 0, 0),
    (4, 640, BF16, BF16, BF16, True, 0, False, True, 0, 0),
    (1500, 96, F32, F32, F32, True, 700, True, True, 0, 0),
]
IDS = [f"{c[0]}x{c[1]}" for c in NORM_CASES]


@pytest.mark.parametrize("case", NORM_CASES, ids=IDS)
def test_block_norm_matches_oracle(wr, ctx, case):
    rows, n, bt, rt, wt, post, gate_rows, resid, pre, pad, shift = case
    inp = norm_inputs(rows + n, *case[:11])
    eps, bs, rs = 1e-5, 0.75, 1.25
    out, y = Padded(rows, n, rt, pad, shift), Padded(rows, n, bt, pad, shift)
    stats = torch.empty(rows, 2, device="cuda")
    wr.wr_block_norm(ctx, eps, **inp, branch_scale=bs, resid_scale=rs, resid_out=out.view, y=y.view if pre else None,
                     stats=stats)
    h = host(inp)
    xo, yo, so, ex, ey = norm_bounds(h, eps, bs, rs)
    got = f64(out.view)
    assert np.all(np.abs(got - xo) <= ex + (np.abs(xo) + ex) * round_err(rt))
    if pre:
        assert np.all(np.abs(f64(y.view) - yo) <= ey + (np.abs(yo) + ey) * round_err(bt))
    share = np.linalg.norm(ex, axis=1) / np.maximum(np.linalg.norm(xo, axis=1), 1e-300)
    tol = np.stack([np.full(rows, 32 * E32), share + 32 * E32], axis=1)
    assert np.all(np.abs(f64(stats) / so - 1) <= tol)
    assert out.untouched() and y.untouched()


@pytest.mark.parametrize("case", [c for c in NORM_CASES if c[8]], ids=[i for i, c in zip(IDS, NORM_CASES) if c[8]])
def test_block_norm_8_bit_tokens(wr, ctx, case):
    """q and q_scales are the 8-bit form of the fp32 y: a code is that of some value within y's error bound."""
    rows, n = case[:2]
    pad, shift = case[9:11]
    inp = norm_inputs(rows + n + 1, *case[:11])
    eps = 1e-6
    q, qs = Padded(rows, n, torch.int8, pad, shift), torch.empty(rows, device="cuda")
    out = Padded(rows, n, case[3], pad, shift)
    wr.wr_block_norm(ctx, eps, **inp, resid_out=out.view, q=q.view, q_scales=qs)
    _, yo, _, _, ey = norm_bounds(host(inp), eps, 1.0, 1.0)
    top, etop = np.abs(yo).max(axis=1, keepdims=True), ey.max(axis=1, keepdims=True)
    assert np.all(np.abs(f64(qs)[:, None] - top / 127) <= (etop + 2 * E32 * top) / 127)
    t = 127 * yo / top
    et = 127 * (ey / top + np.abs(yo) * etop / top ** 2 * 1.01) + 4 * E32 * 127
    codes = f64(q.view)
    assert np.all(np.abs(codes - t) <= 0.5 + et)
    assert np.all(np.abs(codes).max(axis=1) == 127) and q.untouched() and out.untouched()


def test_block_norm_in_place(wr, ctx):
    """resid_out over resid and y over branch give the bits of separate outputs."""
    for case in (NORM_CASES[1], NORM_CASES[10], NORM_CASES[4]):
        rows, n, bt, rt = case[:4]
        inp = norm_inputs(3, *case[:11])
        out, y = torch.empty(rows, n, dtype=rt, device="cuda"), torch.empty(rows, n, dtype=bt, device="cuda")
        wr.wr_block_norm(ctx, 1e-6, **inp, resid_out=out, y=y)
        wr.wr_block_norm(ctx, 1e-6, **inp, resid_out=inp["resid"], y=inp["branch"])
        assert torch.equal(inp["resid"], out) and torch.equal(inp["branch"], y)


def test_norm_without_a_branch(wr, ctx):
    """A norm of the residual stream alone (the heads' norm, a model's first and last norm)."""
    x = torch.randn(300, 128, device="cuda").to(BF16)
    w = torch.randn(128, device="cuda").to(BF16)
    y = torch.empty_like(x)
    wr.wr_block_norm(ctx, 1e-6, resid=x, w_pre=w, y=y)
    yo = oracle.block_norm(1e-6, resid=f64(x), w_pre=f64(w))[1]  # x' = x exactly: 32 eps32 of the rms and two products
    assert np.all(np.abs(f64(y) - yo) <= np.abs(yo) * (44 * E32 + E16 * 1.0001))


def test_norm_special_rows(wr, ctx):
    """Rows of zeros, with an infinity, with a NaN: only those rows are touched by them."""
    rows, n = 6, 1000
    x = torch.randn(rows, n, device="cuda")
    b = torch.randn(rows, n, device="cuda")
    x[1], b[1] = 0, 0
    x[2, 999] = float("inf")
    b[3, 0] = float("nan")
    x[4] = 1e-30
    b[4] = 0
    w = torch.ones(n, device="cuda")
    out, y = torch.empty(rows, n, device="cuda"), torch.empty(rows, n, device="cuda")
    q, qs = torch.empty(rows, n, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda")
    wr.wr_block_norm(ctx, 1e-6, branch=b, resid=x, w_post=w, w_pre=w, resid_out=out, y=y, q=q, q_scales=qs)
    assert bool((y[1] == 0).all()) and float(qs[1]) == 0 and not bool(q[1].any())
    for r in (2, 3):
        assert bool(torch.isnan(qs[r])) and not bool(q[r].any()) and bool(torch.isnan(y[r]).any())
    for r in (0, 4, 5):
        assert bool(torch.isfinite(y[r]).all()) and int(q[r].abs().max()) == 127
    # with eps 0 a row of zeros is 0 / 0, as the formula says
    wr.wr_block_norm(ctx, 0.0, branch=b, resid=x, w_post=w, w_pre=w, y=y)
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isfinite(y[0]).all())


def backward_bounds(h, eps, bs, rs, dy, dres):
    """Magnitudes of the gradient's terms, to be multiplied by K eps32."""
    out, _, stats = oracle.block_norm(eps, **h, bscale=bs, rscale=rs)
    rows, n = out.shape
    r1, r2 = stats[:, :1], stats[:, 1:]
    ab = lambda k: None if h.get(k) is None else np.abs(h[k])  # noqa: E731
    g = oracle.gate_per_token(ab("gate"), h.get("gate_rows", 0), rows) if h.get("gate") is not None else np.ones((rows, n))
    wp = ab("w_post") if h.get("w_post") is not None else np.ones(n)
    bn = ab("branch") * r1 if h.get("branch") is not None else np.zeros((rows, n))
    mag = abs(bs) * g * wp * bn + (0.0 if h.get("resid") is None else abs(rs) * ab("resid"))
    xn = mag * r2
    gx = np.zeros((rows, n)) if dres is None else np.abs(dres)
    if dy is not None:
        d = np.abs(dy) * ab("w_pre")
        gx = gx + r2 * (d + xn * np.mean(d * xn, axis=1, keepdims=True))
    res = {"dresid": abs(rs) * gx, "dw_pre": None if dy is None else np.sum(np.abs(dy) * xn, axis=0)}
    gu = abs(bs) * gx
    if h.get("gate") is not None:
        per = h.get("gate_rows", 0) or rows
        res["dgate"] = np.zeros(h["gate"].shape)
        np.add.at(res["dgate"], np.arange(rows) // per, gu * wp * bn)
    e = gu * g * wp
    res["dw_post"] = np.sum(gu * g * bn, axis=0)
    res["dbranch"] = e if h.get("w_post") is None else r1 * (e + bn * np.mean(e * bn, axis=1, keepdims=True))
    return res


BWD_CASES = NORM_CASES + [
    (2100, 128, BF16, BF16, BF16, True, 0, True, True, 0, 0),   # several tokens a unit, one gate row
    (17000, 100, F32, F32, F32, True, 1, True, True, 0, 0),     # a gate row for every token
    (17000, 64, BF16, F32, F32, True, 3, True, True, 0, 0),     # gate rows of three tokens inside a unit
    (3000, 520, BF16, BF16, BF16, True, 2, True, True, 0, 0),
    (3000, 520, BF16, BF16, BF16, True, 100, True, True, 8, 0),
    (2051, 1030, F32, F32, F32, False, 1500, True, True, 0, 0),
]


def run_backward(wr, ctx, inp, stats, bs, rs, dy, dres, bt, rt, rows, n, pad=0, shift=0):
    db = Padded(rows, n, bt, pad, shift)
    dx = Padded(rows, n, rt, pad, shift) if "resid" in inp else None
    outs = dict(dbranch=db.view, dresid=dx.view if dx else None)
    outs["dw_post"] = torch.full((n,), CANARY, device="cuda") if "w_post" in inp else None
    outs["dw_pre"] = torch.full((n,), CANARY, device="cuda") if dy is not None else None
    outs["dgate"] = torch.full(tuple(inp["gate"].shape), CANARY, device="cuda") if "gate" in inp else None
    wr.wr_block_norm_backward(ctx, stats, **inp, branch_scale=bs, resid_scale=rs, dy=dy, dresid_out=dres, **outs)
    assert db.untouched() and (dx is None or dx.untouched())
    return outs


@pytest.mark.parametrize("case", BWD_CASES, ids=[f"{c[0]}x{c[1]}g{c[6]}" for c in BWD_CASES])
def test_backward_matches_oracle(wr, ctx, case):
    rows, n, bt, rt, wt, post, gate_rows, resid, pre, pad, shift = case
    inp = norm_inputs(rows + n + 2, *case[:11])
    eps, bs, rs = 1e-5, 0.75, 1.25
    g = torch.Generator().manual_seed(rows)
    dy = Padded(rows, n, bt, pad, shift, torch.randn(rows, n, generator=g)).view if pre else None
    dres = Padded(rows, n, rt, pad, shift, torch.randn(rows, n, generator=g)).view
    stats = torch.empty(rows, 2, device="cuda")
    wr.wr_block_norm(ctx, eps, **inp, branch_scale=bs, resid_scale=rs, stats=stats)
    outs = run_backward(wr, ctx, inp, stats, bs, rs, dy, dres, bt, rt, rows, n, pad, shift)
    h = host(inp)
    ref = oracle.block_norm_backward(eps, **h, bscale=bs, rscale=rs, dy=f64(dy), dres=f64(dres))
    mag = backward_bounds(h, eps, bs, rs, f64(dy), f64(dres))
    for name, got in outs.items():
        if got is None:
            continue
        per_token = name in ("dbranch", "dresid")
        bound = (512 if per_token else 512 + rows) * E32 * mag[name]
        last = {"dbranch": round_err(bt), "dresid": round_err(rt)}.get(name, E32)
        assert np.all(np.abs(f64(got) - ref[name]) <= bound + (np.abs(ref[name]) + bound) * last), name


@pytest.mark.parametrize("which", ["dy", "dresid_out"])
def test_backward_with_one_gradient(wr, ctx, which):
    rows, n = 19, 300
    inp = norm_inputs(5, rows, n, F32, F32, F32, True, 4, True, True, 0, 0)
    v = torch.randn(rows, n, device="cuda")
    stats = torch.empty(rows, 2, device="cuda")
    wr.wr_block_norm(ctx, 1e-6, **inp, stats=stats)
    outs = dict(dbranch=torch.empty(rows, n, device="cuda"), dresid=torch.empty(rows, n, device="cuda"))
    wr.wr_block_norm_backward(ctx, stats, **inp, **{which: v}, **outs)
    h = host(inp)
    kw = dict(dy=f64(v) if which == "dy" else None, dres=f64(v) if which != "dy" else None)
    ref, mag = oracle.block_norm_backward(1e-6, **h, **kw), backward_bounds(h, 1e-6, 1.0, 1.0, kw["dy"], kw["dres"])
    for name, got in outs.items():
        assert np.all(np.abs(f64(got) - ref[name]) <= 512 * E32 * mag[name] + E32 * np.abs(ref[name]))


def test_backward_against_differences(wr, ctx):
    """The GPU's gradient along random directions equals the fp64 loss's central difference."""
    rows, n, eps = 12, 200, 1e-5
    inp = norm_inputs(8, rows, n, F32, F32, F32, True, 5, True, True, 0, 0)
    g = torch.Generator().manual_seed(9)
    dy, dres = torch.randn(rows, n, generator=g).cuda(), torch.randn(rows, n, generator=g).cuda()
    stats = torch.empty(rows, 2, device="cuda")
    wr.wr_block_norm(ctx, eps, **inp, stats=stats)
    outs = run_backward(wr, ctx, inp, stats, 1.0, 1.0, dy, dres, F32, F32, rows, n)
    h = host(inp)

    def loss(v):
        out, y, _ = oracle.block_norm(eps, **v)
        return np.sum(out * f64(dres)) + np.sum(y * f64(dy))

    rng = np.random.default_rng(10)
    for name in ("branch", "resid", "w_post", "gate", "w_pre"):
        d = rng.normal(size=h[name].shape)
        step = 1e-4
        num = (loss({**h, name: h[name] + step * d}) - loss({**h, name: h[name] - step * d})) / (2 * step)
        got = f64(outs["d" + name])
        # the gradient: 512 eps32 = 3e-5 of magnitudes about three times the values; the difference: 1e-8
        assert abs(np.sum(got * d) - num) <= 1e-4 * np.sum(np.abs(got * d)), name


def test_backward_is_deterministic_and_in_place(wr, ctx):
    rows, n = 4000, 640
    inp = norm_inputs(11, rows, n, BF16, BF16, BF16, True, 0, True, True, 0, 0)
    dy, dres = torch.randn(rows, n, device="cuda").to(BF16), torch.randn(rows, n, device="cuda").to(BF16)
    stats = torch.empty(rows, 2, device="cuda")
    wr.wr_block_norm(ctx, 1e-6, **inp, stats=stats)
    a = run_backward(wr, ctx, inp, stats, 1.0, 1.0, dy, dres, BF16, BF16, rows, n)
    b = run_backward(wr, ctx, inp, stats, 1.0, 1.0, dy, dres, BF16, BF16, rows, n)
    assert all(torch.equal(a[k], b[k]) for k in a)
    wr.wr_block_norm_backward(ctx, stats, **inp, dy=dy, dresid_out=dres, dbranch=dy, dresid=dres)
    assert torch.equal(dy, a["dbranch"]) and torch.equal(dres, a["dresid"])


def test_backward_of_no_tokens(wr, ctx):
    n = 40
    e = torch.empty(0, n, device="cuda")
    w = torch.ones(n, device="cuda")
    dw, dp, dg = (torch.full((n,), CANARY, device="cuda") for _ in range(3))
    wr.wr_block_norm(ctx, 1e-6, branch=e, resid=e, w_post=w, gate=w[None], w_pre=w, y=e)
    wr.wr_block_norm_backward(ctx, torch.empty(0, 2, device="cuda"), branch=e, resid=e, w_post=w, gate=w[None], w_pre=w,
                              dy=e, dresid_out=e, dbranch=e, dresid=e, dw_post=dp, dgate=dg[None], dw_pre=dw)
    assert not bool(dw.any()) and not bool(dp.any()) and not bool(dg.any())


# ---------------------------------------------------------------- 8-bit rows and products

def quant32(x):
    """Codes and scales in numpy's fp32, whose division is correctly rounded."""
    x = x.astype(np.float32)
    m = np.abs(x).max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        q = np.where(m > 0, np.rint(x * np.float32(127) / m), 0)
    return q.astype(np.int8), (m[:, 0] / np.float32(127)).astype(np.float32)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,n,pad,shift", [(1, 1, 0, 0), (7, 5, 1, 1), (300, 128, 0, 0), (65, 250, 0, 3), (33, 512, 8, 0),
                                              (9, 2560, 0, 0), (5, 2531, 7, 1), (3, 9728, 0, 0), (2, 16384, 0, 0),
                                              (2, 16391, 1, 5), (2, 40000, 0, 0)])
def test_quant_rows_bit_exact(wr, ctx, dtype, rows, n, pad, shift):
    g = torch.Generator().manual_seed(rows * n)
    x = Padded(rows, n, dtype, pad, shift, torch.randn(rows, n, generator=g) * torch.randn(rows, 1, generator=g).exp())
    q, s = Padded(rows, n, torch.int8, pad, shift), torch.empty(rows, device="cuda")
    wr.wr_quant_rows_i8(ctx, x.view, q.view, s)
    host_x = x.view.float().cpu().numpy()
    ref_q, ref_s = quant32(host_x)
    assert np.array_equal(q.view.cpu().numpy(), ref_q) and np.array_equal(s.cpu().numpy(), ref_s)
    assert q.untouched()
    if dtype == BF16:  # 127 x is exact in fp32 and no quotient but a tie rounds to one: the definition's codes
        assert np.array_equal(ref_q, oracle.quant_rows_i8(host_x)[0])


def test_quant_rows_special_rows_and_ranges(wr, ctx):
    n = 777
    x = torch.randn(12, n, device="cuda")
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 776] = float("-inf")
    x[3] *= 1e38 / x[3].abs().max()      # 127 x overflows fp32
    x[4] *= 3e38 / x[4].abs().max()
    x[5] *= 1e-37 / x[5].abs().max()     # 127 / max overflows fp32
    x[6] = torch.randint(0, 70000, (n,), dtype=torch.int32).view(torch.float32).cuda()  # subnormal
    x[7] = 1.0                           # every value the largest
    x[8] = torch.arange(n, device="cuda") - 388  # ties: 127 x / 388
    x[9, 1:] = 0.5
    x[9, 0] = 1.0                        # 63.5: to even
    q, s = torch.empty(12, n, dtype=torch.int8, device="cuda"), torch.empty(12, device="cuda")
    wr.wr_quant_rows_i8(ctx, x, q, s)
    h = x.cpu().numpy().astype(np.float64)
    ref = oracle.quant_rows_i8(h)[0]
    got, gs = q.cpu().numpy(), s.cpu().numpy().astype(np.float64)
    assert np.isnan(gs[1]) and np.isnan(gs[2]) and not got[[0, 1, 2]].any() and gs[0] == 0
    keep = [3, 4, 5, 7, 8, 9, 10, 11]
    # the scale is the fp32 quotient itself, rounded once (a subnormal one in row 5)
    assert np.array_equal(gs[keep], (np.abs(x.cpu().numpy()[keep]).max(axis=1) / np.float32(127)).astype(np.float64))
    t = 127 * h[keep] / np.abs(h[keep]).max(axis=1, keepdims=True)
    assert np.all(np.abs(got[keep] - t) <= 0.5 + 127 * 2 * E32)
    assert np.array_equal(got[[7, 9]], ref[[7, 9]])
    assert np.all(np.abs(got[6] - 127 * h[6] / np.abs(h[6]).max()) <= 0.5 + 127 * 2 * E32)


def mm_inputs(seed, batch, rows, n, padx=0, padw=0, shift=0, bias=True):
    g = torch.Generator().manual_seed(seed)
    x = Padded(batch, n, torch.int8, padx, shift, torch.randint(-128, 128, (batch, n), generator=g))
    w = Padded(rows, n, torch.int8, padw, shift, torch.randint(-128, 128, (rows, n), generator=g))
    xs, ws = torch.rand(batch, generator=g).cuda() * 0.02, torch.rand(rows, generator=g).cuda() * 0.02
    b = torch.randn(rows, generator=g).cuda() if bias else None
    return x.view, xs, w.view, ws, b


def mm_bounds(x, xs, w, ws, b, swiglu):
    """(reference, error before the last rounding)."""
    ref = oracle.matmul_i8(f64(x), f64(xs), f64(w), f64(ws), f64(b), swiglu)
    z0 = np.abs(oracle.matmul_i8(f64(x), f64(xs), f64(w), f64(ws)))
    bb = 0.0 if b is None else np.abs(f64(b))[None]
    ez = E32 * (4 * z0 + 2 * bb)  # the int32 sum to fp32, two scales, the bias
    if not swiglu:
        return ref, ez
    z = oracle.matmul_i8(f64(x), f64(xs), f64(w), f64(ws), f64(b))
    h = z.shape[1] // 2
    g, u = z[:, :h], z[:, h:]
    sg = g / (1 + np.exp(-g))
    return ref, 1.1 * np.abs(u) * ez[:, :h] + np.abs(sg) * ez[:, h:] + 1.1 * ez[:, :h] * ez[:, h:] + 12 * E32 * np.abs(ref)


MM_CASES = [  # batch, rows, n, pad x, pad w, shift
    (1, 1, 1, 0, 0, 0), (1, 64, 128, 0, 0, 0), (1, 2560, 9728, 0, 0, 0), (2, 130, 2560, 0, 0, 0), (3, 34, 47, 1, 2, 3),
    (4, 514, 4096, 16, 0, 0), (5, 66, 2048, 0, 16, 0), (8, 1024, 2560, 0, 0, 0), (9, 96, 1000, 0, 0, 0),
    (16, 254, 512, 0, 0, 0), (17, 256, 528, 0, 0, 16), (31, 70, 333, 3, 0, 1), (32, 2048, 2560, 0, 0, 0),
    (33, 130, 64, 0, 0, 0), (48, 100, 4096, 0, 0, 0), (64, 192, 640, 0, 0, 0), (65, 258, 129, 7, 5, 2), (100, 1030, 2560, 0, 0, 0),
    (127, 126, 255, 1, 1, 1), (128, 256, 256, 0, 0, 0), (129, 1026, 1040, 0, 0, 0), (257, 514, 96, 0, 0, 0),
    (300, 2562, 2560, 0, 16, 0), (513, 1024, 512, 0, 0, 0), (777, 1022, 2531, 7, 7, 0), (1000, 600, 1600, 0, 0, 0),
    (4, 6, 131071, 1, 0, 0),
    # each tile and way of copying of the larger products, with a last slice that passes n
    (1100, 1100, 300, 4, 4, 0), (1100, 1100, 300, 3, 0, 1), (2100, 2200, 144, 0, 0, 0), (2100, 2200, 200, 0, 1, 0),
    (3000, 3000, 400, 0, 0, 16), (3001, 3002, 130, 14, 14, 0), (5000, 70, 260, 0, 12, 0), (40, 9000, 140, 4, 4, 0),
    (70, 5000, 520, 8, 8, 0), (200, 2100, 4200, 8, 8, 0),
]


@pytest.mark.parametrize("swiglu", [False, True], ids=["plain", "swiglu"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("batch,rows,n,padx,padw,shift", MM_CASES)
def test_matmul_i8_matches_oracle(wr, ctx, batch, rows, n, padx, padw, shift, dtype, swiglu):
    if swiglu and rows % 2:
        rows += 1
    x, xs, w, ws, b = mm_inputs(batch + rows + n, batch, rows, n, padx, padw, shift, bias=n % 3 != 0)
    if swiglu:  # keep silu's argument in a range where it bends
        xs, ws = xs * (40 / n ** 0.5), ws * (10 / n ** 0.5)
    y = Padded(batch, rows // 2 if swiglu else rows, dtype, padx, shift)
    wr.wr_matmul_i8(ctx, x, xs, w, ws, y.view, bias=b, swiglu=swiglu)
    ref, err = mm_bounds(x, xs, w, ws, b, swiglu)
    assert np.all(np.abs(f64(y.view) - ref) <= err + (np.abs(ref) + err) * round_err(dtype))
    assert y.untouched()


def test_matmul_i8_extreme_sums_and_scales(wr, ctx):
    """The longest sums of -128 * -128 stay exact, a zero scale gives zeros, a NaN scale NaN in its token only."""
    n = 131071
    x = torch.full((3, n), -128, dtype=torch.int8, device="cuda")
    w = torch.full((4, n), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    xs = torch.tensor([1.0, 0.0, float("nan")], device="cuda")
    ws = torch.ones(4, device="cuda")
    y = torch.empty(3, 4, device="cuda")
    wr.wr_matmul_i8(ctx, x, xs, w, ws, y)
    assert y[0].tolist() == [float(np.float32(n * 16384)), float(np.float32(-n * 128 * 127))] + [float(np.float32(n * 16384))] * 2
    assert not bool(y[1].any()) and bool(torch.isnan(y[2]).all())


# Tokens and weight rows for which each of the largest shared tiles takes the fewest rounds; odd strides and a last slice
# that passes n.  The sums are exact in fp64 too.
@pytest.mark.parametrize("swiglu", [False, True], ids=["plain", "swiglu"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("batch,rows,n,padx,padw", [(3000, 4090, 300, 4, 4), (4090, 4092, 150, 10, 10), (5100, 4090, 520, 8, 8),
                                                    (4090, 5100, 300, 4, 4), (5101, 4090, 131, 0, 3), (4090, 5102, 263, 0, 0)])
def test_matmul_i8_largest_tiles(wr, ctx, batch, rows, n, padx, padw, dtype, swiglu):
    x, xs, w, ws, b = mm_inputs(batch + rows + n, batch, rows, n, padx, padw)
    if swiglu:
        xs, ws = xs * (40 / n ** 0.5), ws * (10 / n ** 0.5)
    y = Padded(batch, rows // 2 if swiglu else rows, dtype, 1)
    wr.wr_matmul_i8(ctx, x, xs, w, ws, y.view, bias=b, swiglu=swiglu)
    z0 = (x.double() @ w.double().t().contiguous()) * xs.double()[:, None] * ws.double()
    ez = E32 * (4 * z0.abs() + 2 * b.double().abs())  # the int32 sum to fp32, two scales, the bias
    ref, err = z0 + b.double(), ez
    if swiglu:
        (g, u), (eg, eu) = ref.chunk(2, 1), ez.chunk(2, 1)
        sg = g / (1 + torch.exp(-g))
        ref = sg * u
        err = 1.1 * u.abs() * eg + sg.abs() * eu + 1.1 * eg * eu + 12 * E32 * ref.abs()
    assert bool(((y.view.double() - ref).abs() <= err + (ref.abs() + err) * round_err(dtype)).all())
    assert y.untouched()


def test_matmul_i8_rows_far_apart(wr, ctx):
    """Rows 8 MiB and more apart: offsets in a tile pass 32 bits."""
    n, far = 200, (1 << 23) + 5
    x, w = (torch.zeros(k * far, dtype=torch.int8, device="cuda").view(k, far)[:, :n] for k in (3, 40))
    x.copy_(torch.randint(-128, 128, (3, n)))
    w.copy_(torch.randint(-128, 128, (40, n)))
    one = torch.ones(40, device="cuda")
    for a, c in ((x, w), (x.contiguous(), w), (x, w.contiguous())):
        y = torch.empty(3, 40, device="cuda")
        wr.wr_matmul_i8(ctx, a, one[:3], c, one, y)
        assert torch.equal(y.double(), x.double() @ w.double().t().contiguous())


def test_matmul_i8_empty(wr, ctx):
    z8 = lambda *s: torch.zeros(*s, dtype=torch.int8, device="cuda")  # noqa: E731
    b = torch.randn(6, device="cuda")
    y = torch.full((5, 6), CANARY, device="cuda")
    wr.wr_matmul_i8(ctx, z8(5, 0), torch.ones(5, device="cuda"), z8(6, 0), torch.ones(6, device="cuda"), y, bias=b)
    assert torch.equal(y, b.expand(5, 6))
    e = torch.empty(0, 6, device="cuda")
    wr.wr_matmul_i8(ctx, z8(0, 9), torch.ones(0, device="cuda"), z8(6, 9), torch.ones(6, device="cuda"), e)
    e = torch.empty(5, 0, device="cuda")
    wr.wr_matmul_i8(ctx, z8(5, 9), torch.ones(5, device="cuda"), z8(0, 9), torch.ones(0, device="cuda"), e)


def test_tensors_on_the_contexts_stream(wr):
    """A context on a stream of its own orders the calls there."""
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c = wr.Context(0)
        x = torch.randn(64, 512, device="cuda")
        w = torch.randn(512, device="cuda")
        y = torch.empty_like(x)
        q, qs = torch.empty(64, 512, dtype=torch.int8, device="cuda"), torch.empty(64, device="cuda")
        wr.wr_block_norm(c, 1e-6, resid=x, w_pre=w, y=y, q=q, q_scales=qs)
        z = torch.empty(64, 64, device="cuda")
        wr.wr_matmul_i8(c, q, qs, q, qs, z)
    s.synchronize()
    v = f64(q) * f64(qs)[:, None]
    assert np.allclose(f64(z), v @ v.T, rtol=1e-5, atol=1e-5)


def test_replayed_graph_equals_eager(wr):
    """The calls recorded in a graph read their inputs anew at each replay, with other work between the replays."""
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        c = wr.Context(0, stream)
        g = torch.Generator(device="cuda").manual_seed(5)
        b, x, dy = (torch.randn(200, 640, generator=g, device="cuda").to(BF16) for _ in range(3))
        w, gate = (torch.randn(640, generator=g, device="cuda").to(BF16) for _ in range(2))
        codes = torch.randint(-127, 128, (1500, 640), generator=g, device="cuda", dtype=torch.int8)
        ws = torch.rand(1500, generator=g, device="cuda") * 0.01

        def outputs():
            return dict(xo=torch.zeros_like(x), q=torch.zeros(200, 640, dtype=torch.int8, device="cuda"),
                        qs=torch.zeros(200, device="cuda"), st=torch.zeros(200, 2, device="cuda"),
                        h=torch.zeros(200, 750, device="cuda"), hq=torch.zeros(200, 750, dtype=torch.int8, device="cuda"),
                        hs=torch.zeros(200, device="cuda"), db=torch.zeros_like(b), dw=torch.zeros(640, device="cuda"),
                        dg=torch.zeros(1, 640, device="cuda"))

        def calls(o):
            wr.wr_block_norm(c, 1e-6, branch=b, resid=x, w_post=w, gate=gate[None], w_pre=w, resid_out=o["xo"], q=o["q"],
                             q_scales=o["qs"], stats=o["st"])
            wr.wr_matmul_i8(c, o["q"], o["qs"], codes, ws, o["h"], swiglu=True)
            wr.wr_quant_rows_i8(c, o["h"], o["hq"], o["hs"])
            wr.wr_block_norm_backward(c, o["st"], branch=b, resid=x, w_post=w, gate=gate[None], w_pre=w, dy=dy,
                                      dbranch=o["db"], dw_pre=o["dw"], dgate=o["dg"])

        eager, replayed = outputs(), outputs()
        calls(eager)  # also registers the workspace
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            calls(replayed)
        for _ in range(4):
            b.copy_(torch.randn(200, 640, generator=g, device="cuda"))
            for t in replayed.values():
                t.zero_()
            graph.replay()
            calls(eager)
            stream.synchronize()
            for name in eager:
                assert torch.equal(eager[name], replayed[name]), name


# ---------------------------------------------------------------- refusals

def test_refusals(wr, ctx):
    d = dict(device="cuda")
    x, w = torch.zeros(4, 32, **d), torch.ones(32, **d)
    q, s = torch.zeros(4, 32, dtype=torch.int8, **d), torch.zeros(4, **d)
    y = torch.full((4, 32), CANARY, **d)
    bad = [
        lambda: wr.wr_quant_rows_i8(ctx, x.half(), q, s),
        lambda: wr.wr_quant_rows_i8(ctx, x, q[:, :31], s),
        lambda: wr.wr_quant_rows_i8(ctx, x, q, s[:3]),
        lambda: wr.wr_quant_rows_i8(ctx, x.cpu(), q, s),
        lambda: wr.wr_quant_rows_i8(ctx, x.t(), q.t().contiguous(), torch.zeros(32, **d)),
        lambda: wr.wr_matmul_i8(ctx, q, s, q[:, :16], s, y[:, :4]),
        lambda: wr.wr_matmul_i8(ctx, q, s, q, s, y),
        lambda: wr.wr_matmul_i8(ctx, q, s, q[:3], s[:3], y[:, :1], swiglu=True),
        lambda: wr.wr_matmul_i8(ctx, q, s, q, s, y[:, :4], bias=s.double()),
        lambda: wr.wr_block_norm(ctx, 1e-6, w_pre=w, y=y),
        lambda: wr.wr_block_norm(ctx, 1e-6, resid=x, y=y),
        lambda: wr.wr_block_norm(ctx, 1e-6, resid=x, w_pre=w),
        lambda: wr.wr_block_norm(ctx, -1.0, resid=x, w_pre=w, y=y),
        lambda: wr.wr_block_norm(ctx, 1e-6, resid=x, w_post=w, w_pre=w, y=y),
        lambda: wr.wr_block_norm(ctx, 1e-6, resid=x, w_pre=w, q=q),
        lambda: wr.wr_block_norm(ctx, 1e-6, branch=x, gate=x, gate_rows=2, w_pre=w, y=y),
        lambda: wr.wr_block_norm(ctx, 1e-6, branch=x, w_post=w.bfloat16(), w_pre=w, y=y),
        lambda: wr.wr_block_norm(ctx, 1e-6, branch=x, resid=x, w_pre=w, y=y.bfloat16()),
        lambda: wr.wr_block_norm(ctx, 1e-6, branch=x, w_pre=w, y=y, branch_scale=float("inf")),
        lambda: wr.wr_block_norm_backward(ctx, None, branch=x, w_pre=w, dy=x, dbranch=y),
        lambda: wr.wr_block_norm_backward(ctx, torch.ones(4, 2, **d), branch=x, dy=x, dbranch=y),
        lambda: wr.wr_block_norm_backward(ctx, torch.ones(4, 2, **d), branch=x, w_pre=w, dbranch=y),
        lambda: wr.wr_block_norm_backward(ctx, torch.ones(4, 2, **d), branch=x, w_pre=w, dy=x, dresid=y),
        lambda: wr.wr_block_norm_backward(ctx, torch.ones(4, 2, **d), branch=x, w_pre=w, dy=x, dw_post=w),
    ]
    for k, call in enumerate(bad):
        with pytest.raises((ValueError, RuntimeError)):
            call()
            pytest.fail(f"call {k} was not refused")
    assert bool((y == CANARY).all())
    wide = torch.zeros(1, 16385, **d)
    with pytest.raises(wr.WringerError) as e:
        wr.wr_block_norm(ctx, 1e-6, resid=wide, w_pre=wide[0], y=wide.clone())
    assert e.value.status == wr.WR_EUNSUPPORTED
    long = torch.zeros(1, 131072, dtype=torch.int8, **d)
    with pytest.raises(wr.WringerError) as e:
        wr.wr_matmul_i8(ctx, long, s[:1], long, s[:1], y[:1, :1])
    assert e.value.status == wr.WR_EUNSUPPORTED
