"""Low-rank adapters of many requests against the fp64 oracle.

Products are exact and sums fp32: A x is off by (n + 3) 2^-24 of sum |A| |x| (n additions in any order, three parts), y by
(rank + 4) 2^-24 of scale sum |B| sum |A| |x| more, plus 2^-23 of |base| and |y|; in bf16 by 2^-8 of |y|.
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


def inputs(counts, n, outs, rank, pool, dtype, ytype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    rows = sum(counts)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=strided(r(rows, n).to(dtype).cuda(), pad), A=(r(pool, rank, n) * n ** -0.5).to(BF16).cuda(),
                B=(r(pool, outs, rank) * rank ** -0.5).to(BF16).cuda(), scales=(0.5 + r(pool).abs()).cuda(),
                base=strided(r(rows, outs).to(ytype).cuda(), pad))


def check(d, y, starts, ids, ranks=None, base=True, rows=None):
    h = {k: t.double().cpu().numpy() for k, t in d.items()}
    b = h["base"] if base else 0 * h["base"]
    want = oracle.adapters(h["x"], b, h["A"], h["B"], h["scales"], starts, ids, ranks)
    size = oracle.adapters(np.abs(h["x"]), 0 * b, np.abs(h["A"]), np.abs(h["B"]), np.abs(h["scales"]), starts, ids, ranks)
    room = (h["A"].shape[2] + h["A"].shape[1] + 7) * 2.0 ** -24 * size + 2.0 ** -23 * (np.abs(b) + np.abs(want))
    if y.dtype == BF16:
        room += 2.0 ** -8 * np.abs(want)
    got = y.double().cpu().numpy()
    rows = slice(None) if rows is None else rows
    assert (np.abs(got - want) <= room)[rows].all()


CASES = [  # counts, n, outs, rank, pool, ids, pad
    ([1], 64, 64, 16, 1, [0], 0), ([1] * 9, 256, 320, 8, 4, [0, 1, -1, 3, 2, 4, 0, 0, 7], 8),
    ([5, 0, 40, 1, 17], 128, 96, 13, 3, [2, 1, 0, -1, 1], 3), ([70, 33], 2560, 512, 64, 2, [1, 0], 0),
    ([3, 130], 333, 201, 1, 2, [0, 1], 0), ([200], 96, 1000, 128, 1, [0], 0), ([2, 2], 65, 63, 256, 2, [1, 0], 1),
    ([1, 1, 1], 9728, 2560, 32, 3, [2, 2, 1], 0), ([16, 16, 16], 512, 512, 16, 2, [0, -5, 1], 0), ([4], 1, 1, 1, 1, [0], 0),
    ([300, 5], 1031, 130, 100, 2, [0, 1], 5), ([1], 7, 4097, 255, 1, [0], 0)]


@pytest.mark.parametrize("dtype,ytype", [(BF16, BF16), (BF16, F32), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("counts,n,outs,rank,pool,ids,pad", CASES)
def test_adapters(wr, ctx, counts, n, outs, rank, pool, ids, pad, dtype, ytype):
    d = inputs(counts, n, outs, rank, pool, dtype, ytype, n + rank, pad)
    starts = np.concatenate([[0], np.cumsum(counts)])
    y = strided(torch.full((sum(counts), outs), 77.0, dtype=ytype).cuda(), pad)
    wr.wr_adapters(ctx, d["x"], d["A"], d["B"], d["scales"], int32(starts), int32(ids), max(counts), y, base=d["base"])
    check(d, y, starts, ids)
    z = d["base"].clone()  # in place
    wr.wr_adapters(ctx, d["x"], d["A"], d["B"], d["scales"], int32(starts), int32(ids), max(counts), z, base=z)
    assert torch.equal(z, y)
    wr.wr_adapters(ctx, d["x"], d["A"], d["B"], d["scales"], int32(starts), int32(ids), max(counts), y)
    check(d, y, starts, ids, base=False)


@pytest.mark.parametrize("counts", [[1, 1, 1, 1], [40, 3, 70, 20]])
def test_ranks_of_their_own(wr, ctx, counts):
    """Rows of A and columns of B behind an adapter's rank are not used, whatever they hold."""
    ids, ranks = [0, 1, 2, 3], [5, 0, 99, 16]
    d = inputs(counts, 320, 256, 32, 4, BF16, F32, 3)
    d["A"][0, 5:], d["B"][0, :, 5:], d["A"][1], d["B"][1], d["A"][3, 16:], d["B"][3, :, 16:] = (float("nan"),) * 6
    starts = np.concatenate([[0], np.cumsum(counts)])
    y = torch.full((sum(counts), 256), 77.0, device="cuda")
    wr.wr_adapters(ctx, d["x"], d["A"], d["B"], d["scales"], int32(starts), int32(ids), max(counts), y, base=d["base"], ranks=int32(ranks))
    d["A"].nan_to_num_(0.0), d["B"].nan_to_num_(0.0)
    check(d, y, starts, ids, ranks)


def test_rows_that_are_left_alone(wr, ctx):
    """Rows of no request and of requests left out keep what they had; NaN in a row of x stays in its row."""
    d = inputs([100], 128, 96, 16, 2, BF16, F32, 4)
    starts, ids = [5, 20, 20, 90], [1, 0, 0]
    d["x"][7, 3] = float("nan")
    y = torch.full((100, 96), 77.0, device="cuda")
    wr.wr_adapters(ctx, d["x"], d["A"], d["B"], d["scales"], int32(starts), int32(ids), 50, y, base=d["base"])
    assert (y[:5] == 77).all() and (y[20:] == 77).all()  # the third request has more than 50 rows
    assert torch.isnan(y[7]).all() and torch.isfinite(y[5:7]).all() and torch.isfinite(y[8:20]).all()
    y.fill_(77.0)
    wr.wr_adapters(ctx, d["x"], d["A"], d["B"], d["scales"], int32([-1, 20, 10, 101]), int32([0, 0, 0]), 101, y, base=d["base"])
    assert (y == 77).all()


def test_infinities_in_the_base_and_in_x(wr, ctx):
    d = inputs([3, 40], 64, 64, 8, 1, BF16, F32, 5)
    d["base"][0, 1], d["base"][1, 2], d["base"][5, 0] = float("inf"), float("nan"), -float("inf")
    y = torch.empty(43, 64, device="cuda")
    wr.wr_adapters(ctx, d["x"], d["A"], d["B"], d["scales"], int32([0, 3, 43]), int32([0, 0]), 40, y, base=d["base"])
    assert y[0, 1] == float("inf") and torch.isnan(y[1, 2]) and y[5, 0] == -float("inf") and int((~torch.isfinite(y)).sum()) == 3


def test_nothing_and_refusals(wr, ctx):
    d = inputs([4], 64, 64, 8, 2, BF16, BF16, 6)
    y = torch.full((4, 64), 7.0, dtype=BF16, device="cuda")
    s, i = int32([0, 4]), int32([0])
    ok = (ctx, d["x"], d["A"], d["B"], d["scales"], s, i, 4, y)
    wr.wr_adapters(ctx, d["x"][:0], *ok[2:5], int32([0, 0]), i, 4, y[:0])
    wr.wr_adapters(*ok[:5], int32([0]), int32([]), 4, y)
    wr.wr_adapters(*ok[:7], 0, y)
    assert (y == 7).all()
    wr.wr_adapters(ctx, d["x"], d["A"][:0].contiguous(), d["B"][:0].contiguous(), d["scales"][:0], s, i, 4, y, base=d["base"])
    assert torch.equal(y, d["base"])
    wr.wr_adapters(ctx, d["x"], d["A"][:, :0].contiguous(), d["B"][:, :, :0].contiguous(), d["scales"], s, i, 4, y)
    assert (y == 0).all()
    for change in ({1: d["x"][:, :63]}, {2: d["A"].float()}, {3: d["B"].transpose(1, 2)}, {4: d["scales"][:1]}, {5: s[:1]},
                   {5: s.long()}, {8: y[:3]}, {8: y.half()}, {1: d["x"].half()}, {7: -1}, {2: d["A"][:1]}):
        args = [change.get(j, a) for j, a in enumerate(ok)]
        with pytest.raises((ValueError, wr.WringerError)):
            wr.wr_adapters(*args)
    with pytest.raises(wr.WringerError):
        wr.wr_adapters(ctx, d["x"], torch.zeros(1, 257, 64, dtype=BF16).cuda(), torch.zeros(1, 64, 257, dtype=BF16).cuda(), d["scales"][:1], s, i, 4, y)
    with pytest.raises(ValueError):
        wr.wr_adapters(*ok, base=d["base"].float())


def test_recorded_and_replayed_with_other_requests(wr):
    """Recorded once and replayed with other values of x, starts and ids, beside eager work."""
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        c = wr.Context(0, stream)
        d = inputs([40], 320, 192, 24, 3, BF16, BF16, 7)
        starts, ids = int32([0, 10, 30, 40]), int32([0, 1, 2])
        args = (d["x"], d["A"], d["B"], d["scales"], starts, ids, 20)
        y, eager = torch.empty(40, 192, dtype=BF16, device="cuda"), torch.empty(40, 192, dtype=BF16, device="cuda")
        wr.wr_adapters(c, *args, y, base=d["base"])
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            wr.wr_adapters(c, *args, y, base=d["base"])
        for i in range(4):
            d["x"].copy_(torch.randn(40, 320, generator=torch.Generator().manual_seed(i)))
            starts.copy_(int32([0, 20 - i, 20 + i, 40 - i])), ids.copy_(int32([i % 3, -1, (i + 1) % 3]))
            y.fill_(77.0), eager.fill_(77.0)
            graph.replay()
            wr.wr_adapters(c, *args, eager, base=d["base"])
            stream.synchronize()
            assert torch.equal(y, eager)
            check(d, y, starts.cpu().numpy(), ids.cpu().numpy(), rows=slice(0, 40 - i))
            assert (y[40 - i:] == 77).all()


@pytest.mark.parametrize("most", [2, 17])
def test_many_requests(wr, ctx, most):
    rng = np.random.default_rng(most)
    counts = [int(n) for n in rng.integers(0, most + 1, 700)]
    ids = [int(n) for n in rng.integers(-1, 5, 700)]
    d = inputs(counts, 96, 130, 16, 5, BF16, F32, most)
    starts = np.concatenate([[0], np.cumsum(counts)])
    y = torch.empty(sum(counts), 130, device="cuda")
    wr.wr_adapters(ctx, d["x"], d["A"], d["B"], d["scales"], int32(starts), int32(ids), most, y, base=d["base"])
    check(d, y, starts, ids)
