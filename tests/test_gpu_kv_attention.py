"""Attention over the 4-bit cache against the fp64 oracle on the values that the cache holds.

With u = 2^-11 (fp16), the cache's values and the weights are rounded to fp16 once each.  A score is off by at most
d_t = scale (u + D 2^-23) sum_i |q_i k_i| + 2^-21 |scale q k| (the roundings of k, the fp32 sums, the way to log2 and the exponential), so a
weight by a factor 1 +- 2 max d, and an output by
    (2 max d + 2 u + (T + 64) 2^-23) sum_t p_t |v_t| + 2^-8 |out|
with T positions in fp32 sums and the last term for bf16.  Weights below 2^-39 of the row's largest may vanish: T 2^-39
max |v| more.  Queries are exact but for parts below 2^-24 of the row's largest value, which 2^-23 sum covers.
"""
import numpy as np
import pytest
import torch

import oracle
from attention_inputs import BF16, F32, Paged, int32, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wr():
    from post_bit_weight_amd import _lib
    return _lib


@pytest.fixture(scope="module")
def ctx(wr):
    return wr.Context(0)


def rows_of(n, width, seed, spread=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, width, generator=g) * spread + shift * torch.randn(width, generator=g)).to(BF16)


def cached(x, heads, dim, group):
    t = x.float().cpu().numpy().reshape(x.shape[0], heads, dim)
    return oracle.kv_values(*oracle.kv_codes(t, group), group)


def check(q, out, k, v, seqs, heads, dim, scale, causal, window, absent=None, before=77.0):
    """seqs: (new, length) each; k, v: values, all positions one after another; absent: positions (of all) not there."""
    q64 = q.double().cpu().numpy().reshape(q.shape[0], -1, dim)
    got = out.double().cpu().numpy().reshape(q64.shape)
    share = q64.shape[1] // heads
    row = at = 0
    worst = 0.0
    for new, length in seqs:
        ok = oracle.sees(length - new, new, length, causal, window)
        if absent is not None:
            ok = ok & ~absent[at:at + length][None]
        for h in range(q64.shape[1]):
            kk, vv = k[at:at + length, h // share], v[at:at + length, h // share]
            want, w = oracle.attend(q64[row:row + new, h], kk, vv, ok, scale)
            seen = ok.any(0)
            with np.errstate(invalid="ignore"):
                size = np.abs(q64[row:row + new, h]) @ np.where(seen[:, None], np.abs(kk), 0).T
                d = abs(scale) * (2.0 ** -11 + dim * 2.0 ** -23 + 2.0 ** -21) * np.where(ok, size, 0).max(1, initial=0)
                vmax = np.nan_to_num(np.where(seen[:, None], np.abs(vv), 0))
                room = (2 * d + 2.0 ** -10 + (length + 64) * 2.0 ** -23)[:, None] * (w @ vmax)
                room += length * 2.0 ** -39 * vmax.max(initial=0) + 2.0 ** -8 * np.abs(want)
            g = got[row:row + new, h]
            assert (np.isnan(g) == np.isnan(want)).all()
            off = np.abs(g - want)
            assert (np.isnan(want) | (off <= room)).all(), (new, length, h, np.nanmax(off - room))
            worst = max(worst, float(np.nanmax(off / np.maximum(room, 1e-30), initial=0)))
        row, at = row + new, at + length
    assert (got[row:] == before).all()
    return worst


def attend(wr, ctx, lengths, new, heads, share, dim, page, group, causal=True, window=0, pad=0, scale=None, seed=0, spread=1.0):
    p = Paged(wr, lengths, heads, dim, page, group, seed=seed)
    total = sum(lengths)
    k, v = rows_of(total, heads * dim, seed + 1, spread, 1.0), rows_of(total, heads * dim, seed + 2, spread)
    p.fill(ctx, k.cuda(), v.cuda())
    rows = sum(new) + 3  # three rows behind the last sequence
    q = strided(rows_of(rows, heads * share * dim, seed + 3).cuda(), pad)
    out = strided(torch.full((rows, heads * share * dim), 77.0, dtype=BF16, device="cuda"), pad + 1)
    scale = dim ** -0.5 if scale is None else scale
    wr.wr_kv_attention(ctx, p.cache, p.sequences(new), q, out, scale, causal=causal, window=window)
    return check(q, out, cached(k, heads, dim, group), cached(v, heads, dim, group), list(zip(new, lengths)), heads, dim, scale,
                 causal, window)


FORMS = [(64, 32, 16), (64, 64, 64), (128, 32, 128), (128, 64, 32), (128, 128, 256), (256, 32, 64), (256, 64, 16), (256, 128, 32)]


@pytest.mark.parametrize("new", [1, 50])
@pytest.mark.parametrize("dim,group,page", FORMS)
def test_every_form(wr, ctx, dim, group, page, new):
    attend(wr, ctx, [150, 61], [new, new], 2, 3, dim, page, group, seed=dim + group)


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1023, 1025, 4097])
def test_one_new_token(wr, ctx, length):
    attend(wr, ctx, [length], [1], 2, 4, 128, 64, 64, seed=length)


@pytest.mark.parametrize("lengths,new", [([5, 0, 700, 33], [5, 0, 1, 33]), ([1, 1, 1], [1, 1, 1]), ([300, 40], [17, 40]), ([130], [129]),
                                         ([64, 64, 64, 64, 64], [0, 64, 0, 1, 2]), ([2000, 9], [130, 9]), ([700], [700])])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 40), (False, 13), (True, 5000)])
def test_lengths_masks_and_windows(wr, ctx, lengths, new, causal, window):
    attend(wr, ctx, lengths, new, 2, 2, 64, 16, 32, causal, window, seed=len(lengths) + window)


@pytest.mark.parametrize("heads,share", [(1, 1), (1, 64), (3, 5), (8, 4), (2, 7), (5, 16), (1, 33)])
@pytest.mark.parametrize("new", [1, 3, 70])
def test_heads(wr, ctx, heads, share, new):
    attend(wr, ctx, [200, 90], [new, new], heads, share, 64, 32, 64, seed=heads, pad=3)


@pytest.mark.parametrize("length,new,window", [(20000, 1, 0), (20000, 1, 700), (9000, 40, 0), (70000, 2, 0), (5000, 300, 1000), (40000, 1, 33000)])
def test_long(wr, ctx, length, new, window):
    attend(wr, ctx, [length, 100], [new, 1], 1, 4, 128, 128, 32, window=window, seed=length)


@pytest.mark.parametrize("pad", [1, 8])
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales(wr, ctx, scale, pad):
    """Large scores (a softmax that is nearly a choice), all weights alike, and the smallest first."""
    attend(wr, ctx, [500, 77], [1, 20], 2, 4, 128, 32, 64, scale=scale, pad=pad, seed=int(pad))


@pytest.mark.parametrize("spread", [1e-6, 1e-4, 300.0, 3e4])
def test_small_and_large_values(wr, ctx, spread):
    attend(wr, ctx, [300], [40], 1, 2, 64, 16, 32, scale=0.125 / spread, spread=spread, seed=5)
    attend(wr, ctx, [300], [1], 1, 2, 64, 16, 32, scale=0.125 / spread, spread=spread, seed=6)


@pytest.mark.parametrize("new", [1, 40])
def test_queries_of_any_size(wr, ctx, new):
    p = Paged(wr, [100], 1, 64, 16, 32)
    k, v = rows_of(100, 64, 1), rows_of(100, 64, 2)
    p.fill(ctx, k.cuda(), v.cuda())
    for spread in (2.0 ** -100, 1e-6, 1e6, 2.0 ** 100):
        q = (rows_of(new, 128, 3).float() * spread).to(BF16).cuda()
        out = torch.empty_like(q)
        wr.wr_kv_attention(ctx, p.cache, p.sequences([new]), q, out, 0.125 / spread)
        check(q, out, cached(k, 1, 64, 32), cached(v, 1, 64, 32), [(new, 100)], 1, 64, float(np.float32(0.125 / spread)), True, 0)
    q.zero_()
    wr.wr_kv_attention(ctx, p.cache, p.sequences([new]), q, out, 0.125)
    check(q, out, cached(k, 1, 64, 32), cached(v, 1, 64, 32), [(new, 100)], 1, 64, 0.125, True, 0)


@pytest.mark.parametrize("new", [1, 5, 60])
def test_non_finite_values_where_a_row_does_not_look(wr, ctx, new):
    """NaN in keys and values: rows that see them are NaN (values: in the dims of the group), the others are as without."""
    heads, dim, group, length = 1, 128, 32, 200
    p = Paged(wr, [length], heads, dim, 16, group)
    k, v = rows_of(length, dim, 1), rows_of(length, dim, 2)
    k[199, 5], v[198, 40], v[170, 100], k[20, 3] = float("nan"), float("nan"), float("inf"), float("inf")
    p.fill(ctx, k.cuda(), v.cuda())
    q = rows_of(new, dim, 3).cuda()
    for window in (0, 10, 28, 100, 190):
        out = torch.empty_like(q)
        wr.wr_kv_attention(ctx, p.cache, p.sequences([new]), q, out, dim ** -0.5, window=window)
        check(q, out, cached(k, heads, dim, group), cached(v, heads, dim, group), [(new, length)], heads, dim, dim ** -0.5, True, window)
    wr.wr_kv_attention(ctx, p.cache, p.sequences([new], lengths=[198], most=198), q, out, dim ** -0.5, window=28)
    check(q, out, cached(k, heads, dim, group)[:198], cached(v, heads, dim, group)[:198], [(new, 198)], heads, dim, dim ** -0.5, True, 28)


@pytest.mark.parametrize("new", [1, 40])
def test_non_finite_queries_stay_in_their_row_and_head(wr, ctx, new):
    p = Paged(wr, [90], 2, 64, 32, 64)
    k, v = rows_of(90, 128, 1), rows_of(90, 128, 2)
    p.fill(ctx, k.cuda(), v.cuda())
    q = rows_of(new, 256, 3).cuda()
    q[0, 70] = float("nan")
    out = torch.empty_like(q)
    wr.wr_kv_attention(ctx, p.cache, p.sequences([new]), q, out, 0.125)
    assert torch.isnan(out[0, 64:128]).all() and int(torch.isnan(out).sum()) == 64


@pytest.mark.parametrize("new", [1, 50])
def test_absent_pages_are_not_seen(wr, ctx, new):
    heads, dim, page, group, lengths = 2, 64, 16, 32, [100, 60, 48]
    p = Paged(wr, lengths, heads, dim, page, group)
    k, v = rows_of(208, 128, 1), rows_of(208, 128, 2)
    p.fill(ctx, k.cuda(), v.cuda())
    absent = np.zeros(208, bool)
    for s, n, bad in ((0, 1, -1), (0, 3, p.pages), (0, 6, 2 ** 31 - 1), (1, 0, -2 ** 31), (2, 0, -7), (2, 1, -7), (2, 2, -7)):
        p.table[s, n] = bad
        at = sum(lengths[:s])
        absent[at + 16 * n:min(at + 16 * n + 16, at + lengths[s])] = True
    new = [min(new, n) for n in lengths]
    for causal, window in ((True, 0), (False, 0), (True, 20)):
        q = rows_of(sum(new), 256, 3).cuda()
        out = torch.empty_like(q)
        wr.wr_kv_attention(ctx, p.cache, p.sequences(new), q, out, 0.125, causal=causal, window=window)
        check(q, out, cached(k, heads, dim, group), cached(v, heads, dim, group), list(zip(new, lengths)), heads, dim, 0.125, causal,
              window, absent)
        assert (out[sum(new[:2]):] == 0).all()  # the third sequence has no page


def test_left_out_sequences_and_rows_without_a_position(wr, ctx):
    heads, dim = 1, 64
    p = Paged(wr, [40, 40, 40, 5], heads, dim, 16, 32)
    k, v = rows_of(125, 64, 1), rows_of(125, 64, 2)
    p.fill(ctx, k.cuda(), v.cuda())
    q = rows_of(60, 64, 3).cuda()
    kc, vc = cached(k, 1, 64, 32), cached(v, 1, 64, 32)

    def run(starts, lengths, most_new, most):
        out = torch.full_like(q, 77.0)
        s = wr.Sequences(int32(starts), int32(lengths), int32(p.table), most_new, most)
        wr.wr_kv_attention(ctx, p.cache, s, q, out, 0.125)
        return out

    whole = run([0, 20, 30, 50, 55], [40, 40, 40, 5], 20, 40)
    check(q, whole, kc, vc, [(20, 40), (10, 40), (20, 40), (5, 5)], 1, 64, 0.125, True, 0)
    out = run([0, 20, 30, 50, 55], [40, 41, -1, 5], 20, 40)
    assert torch.equal(out[:20], whole[:20]) and torch.equal(out[50:], whole[50:]) and (out[20:50] == 77).all()
    out = run([0, 20, 30, 50, 61], [40, 40, 40, 5], 19, 40)
    assert torch.equal(out[20:30], whole[20:30]) and (out[:20] == 77).all() and (out[30:] == 77).all()
    out = run([0, 20, 10, 50, 55], [40, 40, 40, 5], 20, 40)
    assert torch.equal(out[:20], whole[:20]) and (out[20:50] == 77).all() and torch.equal(out[50:], whole[50:])
    out = run([0, 20, 30, 50, 60], [40, 40, 40, 5], 20, 40)  # ten rows, five positions
    assert (out[50:55] == 0).all() and torch.isfinite(out).all()
    assert (out[55:].float() - whole[50:55].float()).abs().max() != 0  # other queries at the same positions
    check(q[55:], out[55:], kc[120:], vc[120:], [(5, 5)], 1, 64, 0.125, True, 0)
    out = run([0, 20, 30, 50, 55], [40, 0, 40, 0], 20, 40)
    assert (out[20:30] == 0).all() and (out[50:55] == 0).all() and torch.equal(out[:20], whole[:20])


def test_recorded_and_replayed_on_new_lengths(wr):
    """A step recorded once (write, attend) and replayed as the sequences grow, with eager work between the replays."""
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        c = wr.Context(0, stream)
        heads, share, dim, lengths = 2, 4, 128, [300, 47, 1000]
        p = Paged(wr, lengths, heads, dim, 32, 64)
        k, v = rows_of(sum(lengths), heads * dim, 1).cuda(), rows_of(sum(lengths), heads * dim, 2).cuda()
        at = [290, 37, 990]
        seqs = p.sequences([1, 1, 1], lengths=at, most=1000)
        p.fill(c, k, v)
        first = np.concatenate([[0], np.cumsum(lengths)[:-1]])
        q, kn, vn = torch.zeros(3, 1024, dtype=BF16, device="cuda"), torch.zeros(3, 256, dtype=BF16, device="cuda"), torch.zeros(3, 256, dtype=BF16, device="cuda")
        out, eager = torch.empty_like(q), torch.empty_like(q)

        def step():
            wr.wr_kv_write(c, p.cache, seqs, kn, vn)
            wr.wr_kv_attention(c, p.cache, seqs, q, out, dim ** -0.5)

        step()
        stream.synchronize()
        k_held, v_held = k.clone(), v.clone()
        for f, a in zip(first, at):  # this eager step wrote rows of zeros
            k_held[int(f + a - 1)] = v_held[int(f + a - 1)] = 0
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
        for i in range(6):
            at = [n + 1 for n in at]
            seqs.lengths.copy_(int32(at))
            rows = [int(f + a - 1) for f, a in zip(first, at)]
            kn.copy_(k[rows]), vn.copy_(v[rows]), q.copy_(rows_of(3, 1024, 10 + i))
            graph.replay()
            stream.synchronize()
            other = p.sequences([1, 1, 1], lengths=at, most=1000)
            wr.wr_kv_attention(c, p.cache, other, q, eager, dim ** -0.5)
            stream.synchronize()
            assert torch.equal(out, eager)
            kk, vv = (np.concatenate([cached(t, heads, dim, 64)[f:f + a] for f, a in zip(first, at)]) for t in (k_held, v_held))
            check(q, out, kk, vv, list(zip([1] * 3, at)), heads, dim, dim ** -0.5, True, 0)


def test_the_same_call_gives_the_same_bits(wr, ctx):
    p = Paged(wr, [6000, 300], 2, 128, 64, 64)
    k, v = rows_of(6300, 256, 1).cuda(), rows_of(6300, 256, 2).cuda()
    p.fill(ctx, k, v)
    for new in ([1, 1], [90, 200]):
        q = rows_of(sum(new), 1024, 3).cuda()
        outs = [torch.empty_like(q) for _ in range(3)]
        for o in outs:
            wr.wr_kv_attention(ctx, p.cache, p.sequences(new), q, o, 0.1)
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_refusals(wr, ctx):
    p = Paged(wr, [32], 2, 64, 16, 32)
    s = p.sequences([2])
    q = torch.zeros(2, 256, dtype=BF16, device="cuda")
    out = torch.full_like(q, 7.0)
    ok = dict(ctx=ctx, cache=p.cache, seqs=s, q=q, out=out, scale=0.125)
    for change in (dict(q=q.float()), dict(out=out.float()), dict(out=out[:1]), dict(q=q[:, :255]), dict(q=q[:, :192], out=out[:, :192]),
                   dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1), dict(q=q.cpu()),
                   dict(q=torch.zeros(2, 2 * 65 * 64, dtype=BF16, device="cuda"), out=torch.zeros(2, 2 * 65 * 64, dtype=BF16, device="cuda"))):
        with pytest.raises((ValueError, wr.WringerError)):
            wr.wr_kv_attention(**dict(ok, **change))
    assert (out == 7).all()
    wr.wr_kv_attention(**dict(ok, q=q[:0], out=out[:0]))
    for args in ((2, 96, 16, 32), (2, 64, 24, 32), (2, 64, 8, 32), (2, 64, 512, 32), (2, 64, 16, 16), (2, 64, 16, 128), (0, 64, 16, 32)):
        with pytest.raises(wr.WringerError):
            wr.KvCache(4, *args)
    for args in ((int32([0, 1]), int32([1, 1]), int32([[0], [1]])), (int32([0, 1]), int32([1]), int32([0])),
                 (int32([0, 1]).long(), int32([1]), int32([[0]])), (int32([0, 1]).cpu(), int32([1]), int32([[0]]))):
        with pytest.raises(ValueError):
            wr.Sequences(*args, 1, 1)
    with pytest.raises(ValueError):
        wr.Sequences(int32([0, 1]), int32([1]), int32([[0]]), -1, 1)
    with pytest.raises(ValueError):
        wr.KvCache(4, 2, 64, 16, 32, buf=torch.zeros(5, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("n", [64, 65, 300, 1500])
def test_many_sequences(wr, ctx, n):
    """One or two new tokens of many sequences, none in some."""
    rng = np.random.default_rng(n)
    lengths = [int(x) for x in rng.integers(1, 60, n)]
    lengths[n // 2] = 2000
    new = [int(x) for x in np.minimum(rng.integers(0, 3, n), lengths)]
    attend(wr, ctx, lengths, new, 2, 4, 64, 16, 32, seed=n, pad=8)


def test_many_sequences_with_prompts(wr, ctx):
    lengths = [int(x) for x in np.random.default_rng(3).integers(1, 200, 80)]
    attend(wr, ctx, lengths, [min(n, 1 + 7 * i % 90) for i, n in enumerate(lengths)], 1, 2, 64, 32, 32, seed=3)


@pytest.mark.parametrize("new,behind", [(30, 5000), (1, 3000)])
def test_a_batch_with_many_rows_behind_the_last_sequence(wr, new, behind):
    """Positions are split, whatever the rows of no sequence are; a new context's workspace is sized for it."""
    p = Paged(wr, [6000], 1, 64, 64, 64)
    k, v = rows_of(6000, 64, 1), rows_of(6000, 64, 2)
    c = wr.Context(0)
    p.fill(c, k.cuda(), v.cuda())
    q = rows_of(new + behind, 256, 3).cuda()
    for most_new in (new, 2 * (new + behind)):
        out = torch.full_like(q, 77.0)
        wr.wr_kv_attention(c, p.cache, p.sequences([new], most_new=most_new), q, out, 0.125)
        check(q, out, cached(k, 1, 64, 64), cached(v, 1, 64, 64), [(new, 6000)], 1, 64, 0.125, True, 0)


@pytest.mark.parametrize("garbage", [0x00, 0x7b, 0x7c, 0xfb, -1])
@pytest.mark.parametrize("new", [1, 40])
def test_whatever_a_page_holds_behind_a_sequence(wr, ctx, new, garbage):
    """The last page's rest and unused pages hold zeros, the largest numbers, infinities or any bytes."""
    for lengths in ([41, 90], [63, 100]):
        p = Paged(wr, lengths, 2, 128, 32, 64)
        if garbage < 0:
            p.cache.buf.copy_(torch.randint(0, 256, p.cache.buf.shape, generator=torch.Generator().manual_seed(4), dtype=torch.uint8))
        else:
            p.cache.buf.fill_(garbage)
        k, v = rows_of(sum(lengths), 256, 1), rows_of(sum(lengths), 256, 2)
        p.fill(ctx, k.cuda(), v.cuda())
        for window in (0, 20):
            q = rows_of(2 * new, 512, 3).cuda()
            out = torch.empty_like(q)
            wr.wr_kv_attention(ctx, p.cache, p.sequences([new, new]), q, out, 0.1, window=window)
            check(q, out, cached(k, 2, 128, 64), cached(v, 2, 128, 64), [(new, n) for n in lengths], 2, 128, float(np.float32(0.1)), True, window)


@pytest.mark.parametrize("new", [1, 50])
def test_pages_past_4_gib(wr, ctx, new):
    heads, dim, page, group, length = 16, 256, 256, 32, 300
    count = (5 << 30) // int(wr.load().wr_kv_page_bytes(heads, dim, page, group)) + 1
    cache = wr.KvCache(count, heads, dim, page_tokens=page, group=group)
    k, v = rows_of(length, heads * dim, 1), rows_of(length, heads * dim, 2)
    table = int32([[count - 1, count - 3]])
    wr.wr_kv_write(ctx, cache, wr.Sequences(int32([0, length]), int32([length]), table, length, length), k.cuda(), v.cuda())
    q = rows_of(new, heads * dim, 3).cuda()
    out = torch.empty_like(q)
    wr.wr_kv_attention(ctx, cache, wr.Sequences(int32([0, new]), int32([length]), table, new, length), q, out, 0.0625)
    check(q, out, cached(k, heads, dim, group), cached(v, heads, dim, group), [(new, length)], heads, dim, 0.0625, True, 0)


def test_a_recorded_call_keeps_its_workspace(wr):
    """The context's workspace is replaced by a larger one after a call was recorded; the replay still has its own."""
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        c = wr.Context(0, stream)
        p = Paged(wr, [3000], 1, 64, 64, 64)
        k, v = rows_of(3000, 64, 1).cuda(), rows_of(3000, 64, 2).cuda()
        p.fill(c, k, v)
        q = rows_of(1, 128, 3).cuda()
        out, eager = torch.empty_like(q), torch.empty_like(q)
        seqs = p.sequences([1])
        wr.wr_kv_attention(c, p.cache, seqs, q, out, 0.125)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            wr.wr_kv_attention(c, p.cache, seqs, q, out, 0.125)
        c.ensure_workspace(3 * c.workspace.numel())
        c.workspace.fill_(255)
        for i in range(3):
            q.copy_(rows_of(1, 128, 4 + i))
            graph.replay()
            wr.wr_kv_attention(c, p.cache, seqs, q, eager, 0.125)
            stream.synchronize()
            assert torch.equal(out, eager)


def test_two_contexts_on_two_streams(wr):
    """Each has its own workspace, so calls at the same time give what they give alone."""
    streams = [torch.cuda.Stream() for _ in range(2)]
    p = Paged(wr, [5000, 200], 2, 128, 64, 64)
    k, v = rows_of(5200, 256, 1).cuda(), rows_of(5200, 256, 2).cuda()
    contexts = [wr.Context(0, s) for s in streams]
    first = wr.Context(0)
    p.fill(first, k, v)
    qs = [rows_of(n, 1024, 3 + n).cuda() for n in (2, 100)]
    seqs = [p.sequences([1, 1]), p.sequences([60, 40])]
    alone = [torch.empty_like(q) for q in qs]
    for s, q, o in zip(seqs, qs, alone):
        wr.wr_kv_attention(first, p.cache, s, q, o, 0.1)
    outs = [[torch.zeros_like(q) for _ in range(10)] for q in qs]
    torch.cuda.synchronize()
    for i in range(10):
        for c, s, q, o in zip(contexts, seqs, qs, outs):
            wr.wr_kv_attention(c, p.cache, s, q, o[i], 0.1)
    torch.cuda.synchronize()
    assert all(torch.equal(o, a) for a, each in zip(alone, outs) for o in each)


@pytest.mark.parametrize("dim,group,window", [(64, 32, 0), (128, 64, 0), (128, 128, 9), (256, 64, 0)])
@pytest.mark.parametrize("n", [60, 300])
def test_many_short_sequences(wr, ctx, n, dim, group, window):
    """So many that each wave has its own: lengths from 1, sequences without rows, absent pages and rows behind the last."""
    heads, share, page, rng = 20, 2, 16, np.random.default_rng(n + dim)
    lengths = [int(x) for x in rng.integers(1, 70, n)]
    new = [int(x) for x in np.minimum(rng.integers(0, 3, n), lengths)]
    p = Paged(wr, lengths, heads, dim, page, group, seed=n)
    k, v = rows_of(sum(lengths), heads * dim, 1), rows_of(sum(lengths), heads * dim, 2)
    p.fill(ctx, k.cuda(), v.cuda())
    absent = np.zeros(sum(lengths), bool)
    for s in range(0, n, 7):
        p.table[s, 0] = -1
        at = sum(lengths[:s])
        absent[at:at + min(page, lengths[s])] = True
    q = rows_of(sum(new) + 3, heads * share * dim, 3).cuda()
    out = torch.full_like(q, 77.0)
    scale = float(np.float32(dim ** -0.5))
    wr.wr_kv_attention(ctx, p.cache, p.sequences(new), q, out, scale, window=window)
    check(q, out, cached(k, heads, dim, group), cached(v, heads, dim, group), list(zip(new, lengths)), heads, dim, scale, True, window, absent)


@pytest.mark.parametrize("new", [1, 2, 40])
def test_sequences_that_share_pages(wr, ctx, new):
    """Three sequences begin with the same 64 positions; each then has its own."""
    lengths, heads, dim, page, group = [64 + 45, 64 + 80, 64 + 41], 2, 128, 32, 64
    p = Paged(wr, lengths, heads, dim, page, group)
    k, v = rows_of(sum(lengths), heads * dim, 1), rows_of(sum(lengths), heads * dim, 2)
    for t in (k, v):
        t[lengths[0]:lengths[0] + 64] = t[lengths[0] + lengths[1]:lengths[0] + lengths[1] + 64] = t[:64]
    p.fill(ctx, k.cuda(), v.cuda())
    p.cache.buf.view(p.pages, -1)[torch.from_numpy(p.table[1:, :2].reshape(-1).astype(np.int64)).cuda()] = 255  # their own copies are gone
    p.table[1:, :2] = p.table[0, :2]
    q = rows_of(3 * new, heads * 3 * dim, 3).cuda()
    out = torch.empty_like(q)
    wr.wr_kv_attention(ctx, p.cache, p.sequences([new] * 3), q, out, 0.1)
    check(q, out, cached(k, heads, dim, group), cached(v, heads, dim, group), [(new, n) for n in lengths], heads, dim, float(np.float32(0.1)), True, 0)


def test_the_queries_are_not_the_output(wr, ctx):
    p = Paged(wr, [32], 2, 64, 16, 32)
    q = torch.zeros(2, 256, dtype=BF16, device="cuda")
    with pytest.raises(wr.WringerError):
        wr.wr_kv_attention(ctx, p.cache, p.sequences([2]), q, q, 0.125)


@pytest.mark.parametrize("n,new", [(500, 1), (40, 50)])
def test_more_sequences_than_rows(wr, n, new):
    """All but two of many sequences are without new rows; a new context's workspace is sized for it."""
    lengths = [30] * n
    lengths[3], lengths[n - 2] = 3000, 1500
    p = Paged(wr, lengths, 1, 64, 64, 64)
    k, v = rows_of(sum(lengths), 64, 1), rows_of(sum(lengths), 64, 2)
    c = wr.Context(0)
    p.fill(c, k.cuda(), v.cuda())
    fresh = [0] * n
    fresh[3] = fresh[n - 2] = new
    q = rows_of(2 * new, 256, 3).cuda()
    out = torch.empty_like(q)
    wr.wr_kv_attention(c, p.cache, p.sequences(fresh), q, out, 0.125)
    check(q, out, cached(k, 1, 64, 64), cached(v, 1, 64, 64), list(zip(fresh, lengths)), 1, 64, 0.125, True, 0)
