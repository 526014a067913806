"""Rotary positions against the fp64 oracle.

The turn is formed in fp64 and its part of a turn rounded to fp32: |part| <= 1 half turns, off by 2^-25, which is an angle
of pi 2^-25; sincospi is good to 4 units in the last place (2^-22 of values up to 1).  Two products and a sum of fp32 add three
roundings of 2^-24.  A value is off by (2^-22 + 2^-23 + 3 * 2^-24) (|x0| + |x1|) < 2^-21 (|x0| + |x1|), and in bf16 by
2^-8 of itself more.
"""
import numpy as np
import pytest
import torch

import oracle
from attention_inputs import BF16, F32, int32, strided

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wr():
    from post_bit_weight_amd import _lib
    return _lib


@pytest.fixture(scope="module")
def ctx(wr):
    return wr.Context(0)


def inputs(rows, heads, dim, pairs, axes, far, dtype, pad, seed):
    g = torch.Generator().manual_seed(seed)
    x = strided(torch.randn(rows, heads * dim, generator=g).to(dtype).cuda(), pad)
    pos = torch.randint(-far, far, (axes, rows), generator=g, dtype=torch.int32)
    freqs = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / max(pairs, 1))
    axis_of = torch.randint(0, axes, (pairs,), generator=g, dtype=torch.int32)
    return x, pos, freqs, axis_of


def check(x, y, pos, freqs, axis_of, dim, interleaved, inverse):
    pairs = len(freqs)
    x64 = x.double().cpu().numpy()
    want = oracle.rotary(x64, pos.numpy(), freqs.numpy(), dim, axis_of.numpy(), interleaved, inverse)
    size = np.abs(x64).reshape(x64.shape[0], -1, dim)
    room = np.zeros_like(size)
    for i in range(pairs):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, pairs + i)
        room[:, :, a] = room[:, :, b] = 2.0 ** -21 * (size[:, :, a] + size[:, :, b])
    room = room.reshape(x64.shape) + (2.0 ** -8 * np.abs(want) if x.dtype == BF16 else 0)
    got = y.double().cpu().numpy()
    assert (np.abs(got - want) <= room).all()
    behind = got.reshape(size.shape)[:, :, 2 * pairs:]
    assert (behind == x64.reshape(size.shape)[:, :, 2 * pairs:]).all()


CASES = [  # rows, heads, dim, pairs, axes, far, pad
    (1, 40, 128, 64, 1, 40960, 0), (1, 1, 2, 1, 1, 3, 0), (5, 3, 80, 32, 2, 1000000, 8), (257, 8, 128, 64, 3, 40960, 1024),
    (33, 5, 96, 48, 1, 2 ** 31 - 1, 3), (7, 2, 33, 16, 1, 100, 1), (19, 1, 256, 128, 4, 70000, 0), (3, 2, 64, 7, 2, 50, 5),
    (2, 3, 16, 0, 1, 5, 0), (4, 1, 1024, 512, 8, 999, 2), (600, 2, 64, 16, 1, 8192, 0), (9, 4, 8, 4, 1, 77, 0), (6, 64, 72, 36, 1, 9, 0)]


@pytest.mark.parametrize("interleaved,inverse", [(False, False), (True, True), (True, False)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,heads,dim,pairs,axes,far,pad", CASES)
def test_rotary(wr, ctx, rows, heads, dim, pairs, axes, far, pad, dtype, interleaved, inverse):
    x, pos, freqs, axis_of = inputs(rows, heads, dim, pairs, axes, far, dtype, pad, rows + dim)
    y = strided(torch.full((rows, heads * dim), 77.0, dtype=dtype, device="cuda"), 1 + pad)
    wr.wr_rotary(ctx, x, y, pos.cuda(), freqs.cuda(), dim, axis_of=axis_of.cuda(), interleaved=interleaved, inverse=inverse)
    check(x, y, pos, freqs, axis_of, dim, interleaved, inverse)
    z = x.clone()  # in place
    wr.wr_rotary(ctx, z, z, pos.cuda(), freqs.cuda(), dim, axis_of=axis_of.cuda(), interleaved=interleaved, inverse=inverse)
    assert torch.equal(z, y)


def test_one_axis_needs_no_list_and_an_unknown_axis_is_copied(wr, ctx):
    x, pos, freqs, _ = inputs(6, 2, 64, 32, 2, 500, F32, 0, 1)
    y, z = torch.empty_like(x), torch.empty_like(x)
    wr.wr_rotary(ctx, x, y, pos[0].cuda(), freqs.cuda(), 64)
    check(x, y, pos[:1], freqs, torch.zeros(32, dtype=torch.int32), 64, False, False)
    axis_of = torch.tensor([0, 1, 2, -1, 2 ** 31 - 1, -2 ** 31] + [1] * 26, dtype=torch.int32)
    wr.wr_rotary(ctx, x, z, pos.cuda(), freqs.cuda(), 64, axis_of=axis_of.cuda())
    check(x, z, pos, freqs, axis_of, 64, False, False)
    assert torch.equal(z[:, 2:6], x[:, 2:6])


@pytest.mark.parametrize("interleaved", [False, True])
def test_the_inverse_is_the_gradient(wr, ctx, interleaved):
    """d/dx of sum(y * dy) is the inverse rotation of dy: the form is linear, so along any direction the difference of two
    calls is exact but for their roundings, 2^-21 of sums over 2 values, here 4 * 64 terms of magnitudes below 25."""
    x, pos, freqs, axis_of = inputs(4, 1, 64, 32, 2, 900, F32, 0, 3)
    dy, step = (inputs(4, 1, 64, 32, 2, 900, F32, 0, s)[0] for s in (4, 5))
    args = (pos.cuda(), freqs.cuda(), 64)
    y0, y1, dx = (torch.empty_like(x) for _ in range(3))
    kw = dict(axis_of=axis_of.cuda(), interleaved=interleaved)
    wr.wr_rotary(ctx, x, y0, *args, **kw)
    wr.wr_rotary(ctx, x + step, y1, *args, **kw)
    wr.wr_rotary(ctx, dy, dx, *args, inverse=True, **kw)
    by_difference = ((y1.double() - y0.double()) * dy.double()).sum()
    assert abs(float(by_difference - (dx.double() * step.double()).sum())) <= 4 * 64 * 25 * 2.0 ** -21


def test_non_finite_values_stay_in_their_pair(wr, ctx):
    x, pos, freqs, axis_of = inputs(3, 1, 64, 32, 1, 900, BF16, 0, 6)
    x[1, 3] = float("nan")
    x[2, 40] = float("inf")
    y = torch.empty_like(x)
    wr.wr_rotary(ctx, x, y, pos.cuda(), freqs.cuda(), 64)
    bad = ~torch.isfinite(y.float())
    assert bad.nonzero().tolist() == [[1, 3], [1, 35], [2, 8], [2, 40]]


def test_nothing_and_refusals(wr, ctx):
    x, pos, freqs, axis_of = inputs(4, 2, 64, 32, 2, 900, BF16, 0, 7)
    y = torch.empty_like(x)
    args = (pos.cuda(), freqs.cuda(), 64)
    wr.wr_rotary(ctx, x[:0], y[:0], pos.cuda()[:, :0], freqs.cuda(), 64, axis_of=axis_of.cuda())
    for bad in (lambda: wr.wr_rotary(ctx, x, y, *args),  # two axes without a list
                lambda: wr.wr_rotary(ctx, x, y.float(), *args, axis_of=axis_of.cuda()),
                lambda: wr.wr_rotary(ctx, x, y[:, :64], *args, axis_of=axis_of.cuda()),
                lambda: wr.wr_rotary(ctx, x, y, pos.cuda().long(), freqs.cuda(), 64, axis_of=axis_of.cuda()),
                lambda: wr.wr_rotary(ctx, x, y, pos.cuda(), freqs.cuda().float(), 64, axis_of=axis_of.cuda()),
                lambda: wr.wr_rotary(ctx, x, y, pos.cuda(), freqs.cuda(), 48, axis_of=axis_of.cuda()),
                lambda: wr.wr_rotary(ctx, x, y, pos.cuda()[:, :3], freqs.cuda(), 64, axis_of=axis_of.cuda()),
                lambda: wr.wr_rotary(ctx, x.half(), y, *args, axis_of=axis_of.cuda()),
                lambda: wr.wr_rotary(ctx, x, y, *args, axis_of=int32([0] * 31))):
        with pytest.raises((ValueError, wr.WringerError)):
            bad()


def test_more_heads_than_a_grid_has_rows(wr, ctx):
    heads, dim = 270000, 1024
    x = torch.randn(1, heads * dim, device="cuda").to(torch.bfloat16)
    y, few = torch.empty_like(x), torch.empty(1, 3 * dim, dtype=torch.bfloat16, device="cuda")
    pos = torch.tensor([77], dtype=torch.int32, device="cuda")
    freqs = torch.rand(dim // 2, dtype=torch.float64, generator=torch.Generator().manual_seed(2)).cuda()
    wr.wr_rotary(ctx, x, y, pos, freqs, dim)
    for h in (0, 65535, 139999, heads - 3):
        wr.wr_rotary(ctx, x[:, h * dim:(h + 3) * dim], few, pos, freqs, dim)
        assert torch.equal(y[:, h * dim:(h + 3) * dim], few)


def test_recorded_and_replayed_on_new_positions(wr):
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        c = wr.Context(0, stream)
        x = torch.randn(5, 256, device="cuda")
        pos, freqs = torch.zeros(5, dtype=torch.int32, device="cuda"), torch.rand(32, dtype=torch.float64, device="cuda")
        y, eager = torch.empty_like(x), torch.empty_like(x)
        wr.wr_rotary(c, x, y, pos, freqs, 64)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            wr.wr_rotary(c, x, y, pos, freqs, 64)
        for i in range(4):
            x.add_(1.0), pos.add_(3)
            graph.replay()
            wr.wr_rotary(c, x, eager, pos, freqs, 64)
            stream.synchronize()
            assert torch.equal(y, eager)
