"""The 4-bit cache: what is written is the oracle's bytes, what is read back the values they stand for - both exactly."""
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


def rows_of(n, width, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, width, generator=g) * spread + torch.randn(width, generator=g)).to(dtype)


def values(x, heads, dim, group):
    """What the cache holds of rows x, fp32."""
    t = x.float().numpy().reshape(x.shape[0], heads, dim)
    return oracle.kv_values(*oracle.kv_codes(t, group), group).astype(np.float32).reshape(x.shape)


def same(got, want):
    return np.array_equal(got, want, equal_nan=True)


FORMS = [(64, 32, 16), (64, 64, 64), (128, 32, 128), (128, 64, 32), (128, 128, 256), (256, 32, 64), (256, 64, 16), (256, 128, 32)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dim,group,page", FORMS)
def test_written_bytes_and_values_read_back(wr, ctx, dim, group, page, dtype):
    heads, lengths = 3, [page, 1, 2 * page + 5, 17]
    p = Paged(wr, lengths, heads, dim, page, group)
    k, v = (rows_of(sum(lengths), heads * dim, dtype, s) for s in (1, 2))
    p.fill(ctx, strided(k.cuda(), 8), strided(v.cuda(), 3))
    full = p.cache.buf.view(p.pages, -1)[int(p.table[0, 0])].cpu().numpy()
    want = oracle.kv_page(*(t[:page].float().numpy().reshape(page, heads, dim) for t in (k, v)), group, page)
    assert np.array_equal(full, want)
    for out in (BF16, F32):
        kb, vb = (strided(torch.zeros(k.shape, dtype=out).cuda(), pad) for pad in (5, 0))
        wr.wr_kv_read(ctx, p.cache, p.sequences(lengths), kb, vb)
        for got, x in ((kb, k), (vb, v)):
            assert same(got.float().cpu().numpy(), torch.from_numpy(values(x, heads, dim, group)).to(out).float().numpy())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_in_steps_of_any_size_as_at_once(wr, ctx, dtype):
    heads, dim, page, group, lengths = 2, 128, 32, 64, [75, 40, 3]
    k, v = (rows_of(sum(lengths), heads * dim, dtype, s).cuda() for s in (3, 4))
    once, steps = (Paged(wr, lengths, heads, dim, page, group) for _ in range(2))
    once.fill(ctx, k, v)
    first = np.concatenate([[0], np.cumsum(lengths)])
    at, rng = [0] * 3, np.random.default_rng(5)
    while any(a < n for a, n in zip(at, lengths)):
        new = [int(min(n - a, rng.integers(0, 20))) for a, n in zip(at, lengths)]
        at = [a + b for a, b in zip(at, new)]
        rows = np.concatenate([np.arange(f + a - b, f + a) for f, a, b in zip(first, at, new)])
        steps.wr.wr_kv_write(ctx, steps.cache, steps.sequences(new, lengths=at, most_new=20, most=75), k[rows], v[rows])
    assert torch.equal(once.cache.buf, steps.cache.buf)


def test_extreme_groups(wr, ctx):
    """Groups of one value, zeros, tiny values, values beyond fp16, infinities and NaN, each in a group of its own."""
    heads, dim, group = 1, 128, 32
    x = rows_of(6, dim, F32, 6)
    x[0, :32], x[0, 32:64] = 5.0, 0.0
    x[1, :32] *= 1e-6
    x[1, 32:64] *= 1e-30
    x[2, :32] *= 1e5
    x[2, 32:64] *= 3e37
    x[3, 5], x[3, 40], x[3, 70] = float("nan"), float("inf"), -float("inf")
    x[4, :64] = 65504.0
    x[4, 3] = -65504.0
    p = Paged(wr, [6], heads, dim, 16, group)
    p.fill(ctx, x.cuda(), x.cuda())
    kb, vb = torch.empty(6, dim, device="cuda"), torch.empty(6, dim, device="cuda")
    wr.wr_kv_read(ctx, p.cache, p.sequences([6]), kb, vb)
    want = values(x, heads, dim, group)
    assert same(kb.cpu().numpy(), want) and same(vb.cpu().numpy(), want)
    assert np.isnan(want[3]).sum() == 96 and np.isfinite(want[[0, 1, 2, 4, 5]]).all() and np.abs(want[2]).max() < 65504


def test_ties_go_to_even(wr, ctx):
    x = torch.zeros(1, 64)
    x[0, :16] = torch.arange(16) + 0.5  # with offset 0 and scale 1: every value half-way
    x[0, 16], x[0, 17] = 15.0, 0.0
    x = x.clamp(max=15.0)
    p = Paged(wr, [1], 1, 64, 16, 32)
    p.fill(ctx, x.cuda(), x.cuda())
    kb = torch.empty(1, 64, device="cuda")
    wr.wr_kv_read(ctx, p.cache, p.sequences([1]), kb, None)
    assert kb[0, :16].tolist() == [0, 2, 2, 4, 4, 6, 6, 8, 8, 10, 10, 12, 12, 14, 14, 15]


def test_keys_or_values_alone(wr, ctx):
    p = Paged(wr, [20], 2, 64, 16, 32)
    before = p.cache.buf.clone()
    k = rows_of(20, 128, BF16, 7).cuda()
    wr.wr_kv_write(ctx, p.cache, p.sequences([20]), None, k)
    kb, vb = torch.full((20, 128), 7.0, device="cuda"), torch.full((20, 128), 7.0, device="cuda")
    wr.wr_kv_read(ctx, p.cache, p.sequences([20]), None, vb)
    assert same(vb.cpu().numpy(), values(k.cpu(), 2, 64, 32)) and (kb == 7).all()
    wr.wr_kv_read(ctx, p.cache, p.sequences([20]), kb, None)
    assert torch.isnan(kb).all()  # the keys are still garbage
    wr.wr_kv_write(ctx, p.cache, p.sequences([20]), k, None)
    wr.wr_kv_read(ctx, p.cache, p.sequences([20]), kb, vb)
    assert torch.equal(kb, vb) and not torch.equal(before, p.cache.buf)


def test_bad_pages_and_sequences_write_nothing(wr, ctx):
    """A sequence with bad starts or lengths is left out; rows in absent pages are not written and read as 0; all other
    bytes stay."""
    heads, dim, page, group = 2, 64, 16, 64
    lengths = [40, 33, 20, 16, 16]
    p = Paged(wr, lengths, heads, dim, page, group, spare=3)
    p.table[0, 1], p.table[1, 0], p.table[1, 2] = p.pages, 2 ** 31 - 1, -2 ** 31
    k = rows_of(sum(lengths), heads * dim, BF16, 8).cuda()
    bad = [40, 33, 2 ** 31 - 1, -1, 16]  # lengths of sequences 2 and 3
    seqs = p.sequences(lengths, lengths=bad, most=48)
    before = p.cache.buf.clone().view(p.pages, -1)
    wr.wr_kv_write(ctx, p.cache, seqs, k, k)
    after = p.cache.buf.view(p.pages, -1)
    written = {int(t) for t in (p.table[0, 0], p.table[0, 2], p.table[1, 1], p.table[4, 0])}
    assert {i for i in range(p.pages) if not torch.equal(before[i], after[i])} == written
    back = torch.full((sum(lengths), heads * dim), 7.0, device="cuda")
    wr.wr_kv_read(ctx, p.cache, seqs, back, None)
    want = values(k.cpu(), heads, dim, group)
    want[16:32] = 0                 # sequence 0, page 1
    want[40:56] = want[72:73] = 0   # sequence 1, pages 0 and 2
    want[73:109] = 7                # sequences 2 and 3 are left out
    assert same(back.cpu().numpy(), want)
    for starts in ([0, 40, 30, 93, 109, 125], [0, 40, 73, 93, 109, 126], [-1, 40, 73, 93, 109, 125]):
        s = wr.Sequences(int32(starts), int32(lengths), int32(p.table), 40, 48)
        out = torch.full_like(back, 7.0)
        wr.wr_kv_read(ctx, p.cache, s, out, None)
        for i, n in enumerate(lengths):
            b, e = starts[i], starts[i + 1]
            if 0 <= b <= e <= 125 and e - b <= 40:
                assert not (out[b:e] == 7).any()
            elif e > b >= 0 and i + 1 == len(lengths):
                assert (out[b:e] == 7).all()
    few = wr.Sequences(int32([0, 40, 73, 93, 109, 125]), int32(lengths), int32(p.table), 33, 48)  # sequence 0 has too many rows
    out = torch.full_like(back, 7.0)
    wr.wr_kv_read(ctx, p.cache, few, out, None)
    assert (out[:40] == 7).all() and not (out[40:] == 7).any()


def test_more_rows_than_positions(wr, ctx):
    """The first rows of a sequence shorter than its rows have no position: not written, read as 0."""
    p = Paged(wr, [21], 1, 64, 16, 32)
    k = rows_of(30, 64, BF16, 9).cuda()
    seqs = p.sequences([30])
    wr.wr_kv_write(ctx, p.cache, seqs, k, k)
    kb, vb = (torch.full((30, 64), 7.0, device="cuda") for _ in range(2))
    wr.wr_kv_read(ctx, p.cache, seqs, kb, vb)
    want = values(k.cpu(), 1, 64, 32)
    want[:9] = 0
    assert same(kb.cpu().numpy(), want) and same(vb.cpu().numpy(), want)
    wr.wr_kv_write(ctx, p.cache, p.sequences([30], lengths=[0], most=21), k, k)  # no position at all
    vb.fill_(7.0)
    wr.wr_kv_read(ctx, p.cache, p.sequences([30], lengths=[0], most=21), None, vb)
    assert (vb == 0).all()


def test_pages_past_4_gib(wr, ctx):
    """Addresses beyond 32 bits: the last pages of a cache of 5 GiB."""
    heads, dim, page, group = 16, 256, 256, 32
    count = (5 << 30) // int(wr.load().wr_kv_page_bytes(heads, dim, page, group)) + 1
    cache = wr.KvCache(count, heads, dim, page_tokens=page, group=group)
    k, v = (rows_of(300, heads * dim, BF16, s).cuda() for s in (10, 11))
    seqs = wr.Sequences(int32([0, 300]), int32([300]), int32([[count - 1, count - 3]]), 300, 300)
    wr.wr_kv_write(ctx, cache, seqs, k, v)
    kb, vb = (torch.empty(300, heads * dim, device="cuda") for _ in range(2))
    wr.wr_kv_read(ctx, cache, seqs, kb, vb)
    assert same(kb.cpu().numpy(), values(k.cpu(), heads, dim, group)) and same(vb.cpu().numpy(), values(v.cpu(), heads, dim, group))
