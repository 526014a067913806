"""The 8-bit gated MLP on packed modules, against the fp64 block on the materialized weights.

Each of the two products multiplies 8-bit tokens with 8-bit weights: rounding to steps of max / 127 is an error of
(max / rms) / (127 sqrt(12)) relative to the rms, 0.6 % to 1 % for Gaussian rows of these widths; four such roundings
and the product's two factors give about 2 % in the output, held to 5 %.
"""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,n,inner,gated", [(1, 128, 192, False), (5, 320, 448, True), (70, 192, 640, True)])
def test_mlp_on_packed_modules(tokens, n, inner, gated):
    from post_bit_weight_amd import _lib as wr
    from post_bit_weight_amd import int8
    ctx = wr.Context(0)
    mods = [int8.synthetic_module(ctx, r, k, b, 64, s) for r, k, b, s in ((inner, n, 2, 1), (inner, n, 3, 2), (n, inner, 4, 3))]
    signs = (torch.randint(0, 2, (n,), generator=torch.Generator().manual_seed(5)) * 2 - 1).to(torch.int8).cuda()
    mods[1].update(had_block=64, signs=signs)  # a module stored in a rotated basis
    g = torch.Generator().manual_seed(6)
    w_pre, w_post = ((1 + 0.2 * torch.randn(n, generator=g)).cuda() for _ in range(2))
    gate = (1 + 0.2 * torch.randn(1, n, generator=g)).to(torch.bfloat16).cuda() if gated else None
    mlp = int8.Int8Mlp(ctx, int8.Int8Linear.from_packed(ctx, mods[:2]), int8.Int8Linear.from_packed(ctx, mods[2:]), w_pre,
                       w_post, gate, most_tokens=tokens)
    resid = torch.randn(tokens, n, generator=g).cuda()
    branch = torch.randn(tokens, n, generator=g).to(torch.bfloat16).cuda()
    resid_out, out = mlp(resid, branch)

    weights = []
    for m in mods:
        sg = signs.cpu().numpy().astype(np.float64) if m.get("had_block") else None
        weights.append(oracle.materialize_exact(m["buf"].cpu().numpy(), m["rows"], m["n_store"], m["bits"], m["group"],
                                                m.get("had_block", 0), sg, m["n_out"]))
    h64 = lambda t: None if t is None else t.double().cpu().numpy()  # noqa: E731
    x, y, _ = oracle.block_norm(mlp.eps, branch=h64(branch), resid=h64(resid), w_post=h64(w_post), gate=h64(gate), w_pre=h64(w_pre))
    a, b = y @ weights[0].T, y @ weights[1].T
    ref = (a / (1 + np.exp(-a)) * b) @ weights[2].T
    assert np.abs(h64(resid_out) - x).max() <= 1e-5 * np.abs(x).max()
    assert np.linalg.norm(h64(out) - ref) <= 0.05 * np.linalg.norm(ref)
    with pytest.raises(ValueError):
        mlp(torch.zeros(tokens + 1, n, device="cuda"), torch.zeros(tokens + 1, n, dtype=torch.bfloat16, device="cuda"))


def test_command_prints_a_line(capsys):
    from post_bit_weight_amd import int8
    assert int8.main(["--tokens", "3", "--hidden", "256", "--inner", "512", "--passes", "2"]) == 0
    assert "us_per_pass" in capsys.readouterr().out
