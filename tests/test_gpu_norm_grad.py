"""The gradient of the block norm without dy, in every kernel form.

Which kernel a case takes follows from the row's width and types: up to 512 values on the lanes of a wave; to 4096 (bf16 only:
8192) on a workgroup with its sums in registers; fp32 to 8192 and bf16 to 12288 with its sums in LDS; wider rows walked.
"""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_block import (BF16, E32, F32, Padded, backward_bounds, f64, host, norm_inputs, round_err, run_backward)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wr():
    from post_bit_weight_amd import _lib
    return _lib


@pytest.fixture(scope="module")
def ctx(wr):
    return wr.Context(0)


WITHOUT_DY = [(5, 7, F32), (40, 100, BF16), (40, 300, F32), (40, 520, BF16), (9, 5120, F32), (9, 6000, BF16), (9, 8000, F32),
              (9, 9728, BF16), (9, 9727, F32), (9, 12301, BF16)]


@pytest.mark.parametrize("pre", [False, True], ids=["no_pre", "pre"])
@pytest.mark.parametrize("rows,n,dtype", WITHOUT_DY, ids=[f"{r}x{n}" for r, n, _ in WITHOUT_DY])
def test_without_dy_the_residual_takes_no_part(wr, ctx, rows, n, dtype, pre):
    """Only x' = rscale x + ... carries dresid_out back, so infinities, NaN and an overflow of rscale x in the residual
    stream leave every gradient as it is with an ordinary stream, bit for bit, and within the oracle's bounds."""
    bs, rs = 0.75, 1.5
    inp = norm_inputs(rows + n, rows, n, dtype, dtype, F32, True, 3, True, pre, 0, 0)
    dres = torch.randn(rows, n, generator=torch.Generator().manual_seed(n)).to(dtype).cuda()
    stats = torch.empty(rows, 2, device="cuda")
    wr.wr_block_norm(ctx, 1e-5, **inp, branch_scale=bs, resid_scale=rs, stats=stats)
    clean = run_backward(wr, ctx, inp, stats, bs, rs, None, dres, dtype, dtype, rows, n)
    h = host(inp)
    h["w_pre"] = None
    ref = oracle.block_norm_backward(1e-5, **h, bscale=bs, rscale=rs, dres=f64(dres))
    mag = backward_bounds(h, 1e-5, bs, rs, None, f64(dres))
    for name in ("dbranch", "dresid", "dw_post", "dgate"):
        per_token = name in ("dbranch", "dresid")
        bound = (512 if per_token else 512 + rows) * E32 * mag[name]
        last = round_err(dtype) if per_token else E32
        assert np.all(np.abs(f64(clean[name]) - ref[name]) <= bound + (np.abs(ref[name]) + bound) * last), name
    x = inp["resid"]
    x[0, n // 2] = float("inf")
    x[1, n - 1] = float("nan")
    x[2] = 3e38                       # finite, rscale x is not
    x[rows - 1, 0] = float("-inf")
    wr.wr_block_norm(ctx, 1e-5, **inp, branch_scale=bs, resid_scale=rs, stats=stats)  # 1 / rms(x') of those rows: 0 or NaN
    dirty = run_backward(wr, ctx, inp, stats, bs, rs, None, dres, dtype, dtype, rows, n)
    for name in ("dbranch", "dresid", "dw_post", "dgate"):
        assert torch.equal(clean[name], dirty[name]), name


@pytest.mark.parametrize("rows,n,dtype", WITHOUT_DY, ids=[f"{r}x{n}" for r, n, _ in WITHOUT_DY])
def test_without_dy_and_post_norm_the_branch_takes_no_part(wr, ctx, rows, n, dtype):
    """dbranch = bscale dresid_out and dresid = rscale dresid_out, whatever is in the branch."""
    b = torch.randn(rows, n, device="cuda").to(dtype)
    x, dres = b.clone(), torch.randn(rows, n, device="cuda").to(dtype)
    b[0, n - 1], b[1, 0], b[2, n // 2] = float("inf"), float("nan"), 3e38
    outs = run_backward(wr, ctx, dict(branch=b, resid=x), None, 2.0, 0.5, None, dres, dtype, dtype, rows, n)
    assert torch.equal(outs["dbranch"], 2 * dres) and torch.equal(outs["dresid"], 0.5 * dres)
