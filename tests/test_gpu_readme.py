"""README's autograd function around the block norm and its gradient, against fp64 autograd of the same formula.

Inputs are fp32, so an output is within 40 fp32 rounding units of its terms and a gradient within 512 + 40 tokens' units; the
terms of Gaussian inputs are at most ten times the outputs' rms and sixty times the gradients': 2.5e-5 and 2e-3 of the rms.
"""
import os
import re

import pytest
import torch

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not os.path.exists(README), reason="this copy is without its documents")]


def test_block_norm_as_an_autograd_function():
    with open(README) as f:
        code = re.search(r"```python\n(.*?)```", f.read(), re.S).group(1)
    g = torch.Generator(device="cuda").manual_seed(1)
    leaf = lambda *s: torch.randn(*s, generator=g, device="cuda").requires_grad_()  # noqa: E731
    given = dict(branch=leaf(40, 320), resid=leaf(40, 320), w_post=leaf(320), w_pre=leaf(320))
    space = dict(given)
    exec(code, space)
    up = [torch.randn(40, 320, generator=g, device="cuda") for _ in range(2)]
    ((space["resid_out"] * up[0]).sum() + (space["y"] * up[1]).sum()).backward()

    wide = {k: v.detach().double().requires_grad_() for k, v in given.items()}
    rms = lambda v: v / torch.sqrt(v.square().mean(1, keepdim=True) + 1e-6)  # noqa: E731
    out = wide["resid"] + wide["w_post"] * rms(wide["branch"])
    y = wide["w_pre"] * rms(out)
    ((out * up[0]).sum() + (y * up[1]).sum()).backward()
    pairs = [(space["resid_out"], out, 2.5e-5), (space["y"], y, 2.5e-5)] + [(given[k].grad, wide[k].grad, 2e-3) for k in given]
    for got, ref, share in pairs:
        got, ref = got.detach().double(), ref.detach()
        assert float((got - ref).abs().max()) <= share * float(ref.square().mean().sqrt())
