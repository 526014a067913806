"""The block norm over its own inputs: resid_out over resid, with and without each of the two norms, y over branch."""
import pytest
import torch

from test_gpu_block import BF16, F32, Padded, norm_inputs

pytestmark = pytest.mark.gpu

CASES = [  # rows, n, branch type, residual type, gate_rows: widths whose last columns two threads or waves hold, further rows
    (3, 5, F32, F32, 0), (300, 129, BF16, F32, 7), (1100, 400, BF16, BF16, None), (40, 513, BF16, BF16, 0),
    (1500, 1537, BF16, F32, 100), (1100, 2531, BF16, BF16, 0), (2000, 2560, BF16, BF16, 0), (600, 4097, F32, F32, 3),
    (700, 9727, BF16, BF16, None), (600, 9729, F32, F32, 0), (300, 16383, F32, F32, 0),
]


@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)],
                         ids=["both", "post", "pre", "neither"])
@pytest.mark.parametrize("rows,n,bt,rt,gate_rows", CASES, ids=[f"{c[0]}x{c[1]}" for c in CASES])
def test_over_the_residual_stream(rows, n, bt, rt, gate_rows, post, pre):
    """The bits of separate outputs, and nothing beside the rows."""
    from post_bit_weight_amd import _lib as wr
    ctx = wr.Context(0)
    inp = norm_inputs(rows + n, rows, n, bt, rt, F32, post, gate_rows, True, pre, 3, 1)
    out, y = Padded(rows, n, rt, 3, 1), torch.empty(rows, n, dtype=bt, device="cuda") if pre else None
    stats = torch.empty(rows, 2, device="cuda")
    args = dict(branch_scale=0.75, resid_scale=1.25)
    wr.wr_block_norm(ctx, 1e-6, **inp, **args, resid_out=out.view, y=y, stats=stats)
    own = Padded(rows, n, rt, 3, 1, inp["resid"])
    inp["resid"] = own.view
    again = torch.empty_like(stats)
    wr.wr_block_norm(ctx, 1e-6, **inp, **args, resid_out=own.view, y=inp["branch"] if pre else None, stats=again)
    assert torch.equal(own.view, out.view) and own.untouched() and torch.equal(stats, again)
    if pre:
        assert torch.equal(inp["branch"], y)
