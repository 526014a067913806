"""Forms of the 8-bit row quantizer and product that take many rows: the quantizer bit for bit, the product within its bound.

The quantizer's forms by rows and width on 256 CUs: more than 256 rows of more than 512 values lie on a wave (two or four
chunks of eight values a lane, to 1024 and 2048 values) or on a workgroup of four chunks a thread.
"""
import numpy as np
import pytest
import torch

from test_gpu_block import BF16, E16, E32, F32, Padded, f64, mm_bounds, mm_inputs, quant32, round_err

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wr():
    from post_bit_weight_amd import _lib
    return _lib


@pytest.fixture(scope="module")
def ctx(wr):
    return wr.Context(0)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,n,pad,shift", [
    (257, 1000, 0, 0), (5001, 1001, 0, 3), (300, 513, 1, 0), (4200, 1024, 8, 0),           # a wave, two chunks
    (300, 2047, 0, 0), (4999, 1025, 3, 1), (4300, 2048, 0, 0),                            # a wave, four chunks
    (777, 2531, 7, 1), (3001, 4096, 0, 0), (2500, 2049, 0, 0), (701, 9727, 5, 0), (600, 16384, 0, 0), (300, 16383, 1, 5),
    (66001, 5, 0, 0), (33001, 100, 4, 1), (17001, 200, 0, 0), (9001, 511, 0, 3),             # the narrow forms' further rows
    (300, 16400, 0, 0),                                                                   # wider than a workgroup's registers
])
def test_quant_many_rows_bit_exact(wr, ctx, dtype, rows, n, pad, shift):
    g = torch.Generator().manual_seed(rows * n)
    x = Padded(rows, n, dtype, pad, shift, torch.randn(rows, n, generator=g) * torch.randn(rows, 1, generator=g).exp())
    x.view[rows // 2] = 0
    x.view[rows // 3, n - 1] = float("nan")
    x.view[rows - 1, 0] = float("inf")
    q, s = Padded(rows, n, torch.int8, pad, shift), torch.empty(rows, device="cuda")
    wr.wr_quant_rows_i8(ctx, x.view, q.view, s)
    host = x.view.float().cpu().numpy()
    bad = ~np.isfinite(host).all(axis=1)
    host[bad] = 0
    ref_q, ref_s = quant32(host)
    ref_s[bad] = np.nan
    assert np.array_equal(q.view.cpu().numpy(), ref_q) and np.array_equal(s.cpu().numpy(), ref_s, equal_nan=True)
    assert bad.sum() == 2 and q.untouched()


# Between 257 and 512 tiles of 64 tokens x 128 weight rows: two workgroups a CU, one group of waves each.
@pytest.mark.parametrize("swiglu", [False, True], ids=["plain", "swiglu"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("batch,rows,n,padx,padw,shift", [(1500, 2000, 300, 4, 4, 0), (1501, 1998, 333, 3, 1, 1), (2050, 1410, 384, 0, 0, 0),
                                                          (4000, 900, 20, 0, 0, 0), (1100, 3500, 128, 0, 16, 0), (1537, 2046, 1030, 0, 0, 0)])
def test_matmul_i8_two_workgroups_a_cu(wr, ctx, batch, rows, n, padx, padw, shift, dtype, swiglu):
    assert 256 < -(-rows // 128) * -(-batch // 64) <= 512
    x, xs, w, ws, b = mm_inputs(batch + rows + n, batch, rows, n, padx, padw, shift, bias=n % 3 != 0)
    if swiglu:  # silu's argument in a range where it bends
        xs, ws = xs * (40 / n ** 0.5), ws * (10 / n ** 0.5)
    y = Padded(batch, rows // 2 if swiglu else rows, dtype, padx, shift)
    wr.wr_matmul_i8(ctx, x, xs, w, ws, y.view, bias=b, swiglu=swiglu)
    ref, err = mm_bounds(x, xs, w, ws, b, swiglu)
    assert np.all(np.abs(f64(y.view) - ref) <= err + (np.abs(ref) + err) * round_err(dtype))
    assert y.untouched()


@pytest.mark.parametrize("swiglu", [False, True], ids=["plain", "swiglu"])
@pytest.mark.parametrize("n", [9, 33])
def test_matmul_i8_more_tokens_than_a_launch(wr, ctx, n, swiglu):
    """Past 2^19 tokens a call takes several launches: the later ones' tokens, scales and outputs."""
    batch, rows = (1 << 19) + 77, 6
    x, xs, w, ws, b = mm_inputs(n, batch, rows, n, 3, 1)
    if swiglu:
        xs, ws = xs * (40 / n ** 0.5), ws * (10 / n ** 0.5)
    y = Padded(batch, rows // 2 if swiglu else rows, F32, 2)
    wr.wr_matmul_i8(ctx, x, xs, w, ws, y.view, bias=b, swiglu=swiglu)
    ref, err = mm_bounds(x, xs, w, ws, b, swiglu)
    assert np.all(np.abs(f64(y.view) - ref) <= err + (np.abs(ref) + err) * E32)
    assert y.untouched()


def test_matmul_i8_few_tokens_many_rows(wr, ctx):
    """Up to 16 tokens keep the narrow tile however many weight rows there are."""
    for swiglu in (False, True):
        x, xs, w, ws, b = mm_inputs(3, 3, 40002, 144, 0, 0)
        y = Padded(3, 20001 if swiglu else 40002, BF16, 1)
        wr.wr_matmul_i8(ctx, x, xs * 3, w, ws, y.view, bias=b, swiglu=swiglu)
        ref, err = mm_bounds(x, xs * 3, w, ws, b, swiglu)
        assert np.all(np.abs(f64(y.view) - ref) <= err + (np.abs(ref) + err) * E16) and y.untouched()
