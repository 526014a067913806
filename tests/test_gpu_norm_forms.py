"""The block norm and its gradient in every kernel form: many rows a workgroup, wide rows, gate rows inside and across the ranges
of tokens that workgroups walk, against the oracle and, for sums over tokens, bit for bit.

Forms of the gradient on 256 CUs: rows of up to 512 values lie on 8 to 64 lanes of a wave; to 4096 (bf16 only: 8192) on a
workgroup with the parameters' sums in registers; fp32 to 6144 and to 8192 and bf16 to 12288 with them in LDS; wider rows are
walked twice.
"""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_block import (BF16, E32, F32, Padded, backward_bounds, f64, host, norm_bounds, norm_inputs, round_err,
                            run_backward)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wr():
    from post_bit_weight_amd import _lib
    return _lib


@pytest.fixture(scope="module")
def ctx(wr):
    return wr.Context(0)


# ---------------------------------------------------------------- sums over tokens, exactly

SUM_CASES = [  # rows, n, branch type, residual type, weight type, gate_rows, pad, shift
    (40000, 5, F32, F32, F32, 0, 0, 0), (40001, 7, BF16, BF16, BF16, 3, 1, 1),
    (17000, 100, F32, F32, F32, 0, 0, 0), (17001, 64, BF16, F32, F32, 1, 0, 0), (17001, 128, BF16, BF16, BF16, 3, 8, 0),
    (9001, 200, F32, F32, BF16, 7, 0, 1), (9001, 130, BF16, BF16, F32, 5000, 3, 0),
    (5000, 500, F32, BF16, BF16, 0, 0, 0), (5003, 512, BF16, BF16, BF16, 1000, 0, 0),
    (2500, 2531, BF16, BF16, BF16, 0, 5, 1), (2051, 1030, F32, F32, F32, 1500, 0, 0), (1300, 4096, F32, F32, F32, 2, 0, 0),
    (1301, 4095, BF16, F32, BF16, 300, 0, 3), (333, 1537, F32, BF16, BF16, 37, 3, 0), (3, 1537, BF16, BF16, BF16, 2, 0, 0),
]
WIDE = [(6000, BF16, BF16, BF16), (8191, BF16, BF16, F32), (9728, BF16, BF16, BF16), (12287, BF16, BF16, F32),
        (5120, F32, F32, F32), (6143, F32, BF16, BF16), (8000, F32, F32, BF16), (8191, BF16, F32, F32),
        (9727, F32, F32, F32), (12301, BF16, BF16, BF16), (16384, BF16, F32, BF16), (16383, F32, BF16, F32)]
# one gate row, gate rows that end inside a workgroup's tokens, gate rows cut over workgroups (some without tokens)
SUM_CASES += [(601, n, b, r, w, gate, n % 3, n % 2) for n, b, r, w in WIDE for gate in (0, 2, 250)]


def whole(rows, n, most, gen, mirror=0):
    """Whole numbers up to `most`, equal in columns 2 i and 2 i + 1 (mirror -1: of opposite sign, the odd last one 0)."""
    half = torch.randint(-most, most + 1, (rows, (n + 1) // 2), generator=gen, device="cuda").float()
    both = torch.stack([half, -half if mirror else half], dim=2).flatten(1)[:, :n]
    if mirror and n % 2:
        both[:, -1] = 0
    return both


@pytest.mark.parametrize("rows,n,bt,rt,wt,gate_rows,pad,shift", SUM_CASES,
                         ids=[f"{c[0]}x{c[1]}g{c[5]}" for c in SUM_CASES])
def test_sums_over_tokens_are_exact(wr, ctx, rows, n, bt, rt, wt, gate_rows, pad, shift):
    """Inputs for which fp32 holds every product and every sum, so one token left out or counted twice shows.

    All inputs are small whole numbers, the two inverse norms (the caller's `stats`) powers of two, and neighbouring
    columns equal but for dy, where they cancel: mean(d xn) is then 0, and dx' = dresid_out + r2 d.  Every term of a sum is
    a multiple of 1/16 below 10, so the sums of up to 40001 tokens stay below 2^24 sixteenths.
    """
    g = torch.Generator(device="cuda").manual_seed(rows + n)
    gates = -(-rows // gate_rows) if gate_rows else 1
    mat = lambda t, v, p=pad, s=shift: Padded(v.shape[0], n, t, p, s, v).view  # noqa: E731
    inp = dict(branch=mat(bt, whole(rows, n, 3, g)), resid=mat(rt, whole(rows, n, 4, g)), gate=mat(bt, whole(gates, n, 2, g)),
               w_post=(1 + whole(1, n, 1, g)[0].abs()).to(wt), w_pre=(1 + whole(1, n, 1, g)[0].abs()).to(wt), gate_rows=gate_rows)
    dy, dres = mat(bt, whole(rows, n, 3, g, mirror=-1)), mat(rt, torch.randint(-4, 5, (rows, n), generator=g, device="cuda"))
    r1, r2, bs, rs = 0.5, 0.25, 0.5, 2.0
    stats = torch.tensor([r1, r2], device="cuda").repeat(rows, 1)
    outs = run_backward(wr, ctx, inp, stats, bs, rs, dy, dres, bt, rt, rows, n, pad, shift)

    d = {k: v.double() if torch.is_tensor(v) else v for k, v in inp.items()}
    owner = torch.arange(rows, device="cuda") // (gate_rows or rows)
    gate = d["gate"][owner]
    bn = d["branch"] * r1
    xn = (rs * d["resid"] + bs * gate * d["w_post"] * bn) * r2
    dxo = dres.double() + r2 * dy.double() * d["w_pre"]
    ref = dict(dresid=rs * dxo, dw_pre=(dy.double() * xn).sum(0), dw_post=(bs * gate * dxo * bn).sum(0),
               dgate=torch.zeros(gates, n, dtype=torch.float64, device="cuda").index_add_(0, owner, bs * dxo * d["w_post"] * bn))
    for name, value in ref.items():
        assert torch.equal(outs[name].double(), value), name
    # the branch's gradient holds a mean: 512 units of its terms' magnitudes, as for the other forms
    e = bs * gate * d["w_post"] * dxo
    along = (e * bn).mean(1, keepdim=True)
    mag = r1 * (e.abs() + bn.abs() * (e * bn).abs().mean(1, keepdim=True))
    err = (outs["dbranch"].double() - r1 * (e - bn * along)).abs()
    assert bool((err <= 512 * E32 * mag * (1 + round_err(bt)) + round_err(bt) * (r1 * (e - bn * along)).abs()).all())


# ---------------------------------------------------------------- wide rows, ordinary values

GRAD_CASES = [(n, b, r, w, gate) for n, b, r, w in WIDE for gate in (0, 250)]


@pytest.mark.parametrize("n,bt,rt,wt,gate_rows", GRAD_CASES, ids=[f"{c[0]}g{c[4]}" for c in GRAD_CASES])
def test_wide_rows_match_the_oracle(wr, ctx, n, bt, rt, wt, gate_rows):
    """Sums over tokens: a workgroup's 2 tokens, then up to 256 partials over 32 threads and 5 halvings, 2 + 8 + 5 additions
    one after another; 100 is above that."""
    rows = 300
    inp = norm_inputs(n + gate_rows, rows, n, bt, rt, wt, True, gate_rows, True, True, 1, 1)
    eps, bs, rs = 1e-5, 0.75, 1.25
    g = torch.Generator().manual_seed(n)
    dy = Padded(rows, n, bt, 1, 1, torch.randn(rows, n, generator=g)).view
    dres = Padded(rows, n, rt, 1, 1, torch.randn(rows, n, generator=g)).view
    stats = torch.empty(rows, 2, device="cuda")
    wr.wr_block_norm(ctx, eps, **inp, branch_scale=bs, resid_scale=rs, stats=stats)
    outs = run_backward(wr, ctx, inp, stats, bs, rs, dy, dres, bt, rt, rows, n, 1, 1)
    h = host(inp)
    ref = oracle.block_norm_backward(eps, **h, bscale=bs, rscale=rs, dy=f64(dy), dres=f64(dres))
    mag = backward_bounds(h, eps, bs, rs, f64(dy), f64(dres))
    for name, got in outs.items():
        bound = (512 if name in ("dbranch", "dresid") else 612) * E32 * mag[name]
        last = {"dbranch": round_err(bt), "dresid": round_err(rt)}.get(name, E32)
        assert np.all(np.abs(f64(got) - ref[name]) <= bound + (np.abs(ref[name]) + bound) * last), name


@pytest.mark.parametrize("n,bt,rt,wt", WIDE, ids=[str(c[0]) for c in WIDE])
def test_wide_gradient_in_place_and_again(wr, ctx, n, bt, rt, wt):
    """dbranch over dy or branch and dresid over dresid_out or resid give the bits of separate outputs, every time."""
    rows = 300
    inp = norm_inputs(n, rows, n, bt, rt, wt, True, 7, True, True, 0, 0)
    dy, dres = torch.randn(rows, n, device="cuda").to(bt), torch.randn(rows, n, device="cuda").to(rt)
    stats = torch.empty(rows, 2, device="cuda")
    wr.wr_block_norm(ctx, 1e-6, **inp, stats=stats)
    a = run_backward(wr, ctx, inp, stats, 1.0, 1.0, dy, dres, bt, rt, rows, n)
    b = run_backward(wr, ctx, inp, stats, 1.0, 1.0, dy, dres, bt, rt, rows, n)
    assert all(torch.equal(a[k], b[k]) for k in a)
    for over_dy, over_dres in ((True, True), (False, False)):
        copy = {k: v.clone() if torch.is_tensor(v) else v for k, v in inp.items()}
        cy, cr = dy.clone(), dres.clone()
        db, dx = cy if over_dy else copy["branch"], cr if over_dres else copy["resid"]
        dp, dw, dg = torch.empty(n, device="cuda"), torch.empty(n, device="cuda"), torch.empty_like(a["dgate"])
        wr.wr_block_norm_backward(ctx, stats, **copy, dy=cy, dresid_out=cr, dbranch=db, dresid=dx, dw_post=dp, dw_pre=dw,
                                  dgate=dg)
        for name, got in dict(dbranch=db, dresid=dx, dw_post=dp, dw_pre=dw, dgate=dg).items():
            assert torch.equal(a[name], got), name


# ---------------------------------------------------------------- more rows than workgroups

WALKS = [  # rows, n, types, gate_rows, pad, shift: every workgroup walks to a second row at least
    (33001, 5, F32, F32, F32, 100, 0, 0), (17001, 100, BF16, BF16, BF16, 0, 4, 0), (9001, 200, BF16, F32, F32, 7, 0, 1),
    (4501, 401, F32, BF16, BF16, 1, 0, 0), (2600, 2560, BF16, BF16, BF16, 0, 0, 0), (2601, 1025, BF16, F32, BF16, 3, 1, 1),
    (700, 5001, BF16, BF16, BF16, 100, 0, 0), (1100, 9727, F32, F32, F32, 100, 5, 0), (600, 16383, BF16, BF16, BF16, 0, 0, 1),
]


@pytest.mark.parametrize("rows,n,bt,rt,wt,gate_rows,pad,shift", WALKS, ids=[f"{c[0]}x{c[1]}" for c in WALKS])
def test_norm_walks_to_further_rows(wr, ctx, rows, n, bt, rt, wt, gate_rows, pad, shift):
    """x', y and the 8-bit tokens of every row, also those that a workgroup reaches after its first; rows of zeros and with a
    NaN between them change no other row."""
    inp = norm_inputs(rows + n, rows, n, bt, rt, wt, True, gate_rows, True, True, pad, shift)
    eps, bs, rs = 1e-5, 0.75, 1.25
    inp["branch"][rows // 2], inp["resid"][rows // 2] = 0, 0
    inp["resid"][rows - 2, 0] = float("nan")
    keep = np.ones(rows, bool)
    keep[[rows // 2, rows - 2]] = False
    out, y = Padded(rows, n, rt, pad, shift), Padded(rows, n, bt, pad, shift)
    q, qs = Padded(rows, n, torch.int8, pad, shift), torch.empty(rows, device="cuda")
    wr.wr_block_norm(ctx, eps, **inp, branch_scale=bs, resid_scale=rs, resid_out=out.view, y=y.view, q=q.view, q_scales=qs)
    assert out.untouched() and y.untouched() and q.untouched()
    assert not bool(out.view[rows // 2].any()) and not bool(y.view[rows // 2].any()) and not bool(q.view[rows // 2].any())
    assert float(qs[rows // 2]) == 0 and bool(torch.isnan(qs[rows - 2])) and not bool(q.view[rows - 2].any())
    h = host(inp)
    h["branch"], h["resid"] = h["branch"][keep], h["resid"][keep]
    h["gate"], h["gate_rows"] = oracle.gate_per_token(h["gate"], gate_rows, rows)[keep], 1
    xo, yo, _, ex, ey = norm_bounds(h, eps, bs, rs)
    assert np.all(np.abs(f64(out.view)[keep] - xo) <= ex + (np.abs(xo) + ex) * round_err(rt))
    assert np.all(np.abs(f64(y.view)[keep] - yo) <= ey + (np.abs(yo) + ey) * round_err(bt))
    top, etop = np.abs(yo).max(axis=1, keepdims=True), ey.max(axis=1, keepdims=True)
    assert np.all(np.abs(f64(qs)[keep, None] - top / 127) <= (etop + 2 * E32 * top) / 127)
    et = 127 * (ey / top + np.abs(yo) * etop / top ** 2 * 1.01) + 4 * E32 * 127
    assert np.all(np.abs(f64(q.view)[keep] - 127 * yo / top) <= 0.5 + et)
