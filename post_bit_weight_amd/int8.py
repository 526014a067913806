"""Run a block's gated MLP in 8-bit integers on the weights of the container.

A quantized module leaves the container as bf16 weights (``wr_materialize``); here they become 8-bit codes with
one scale per output channel, once, and every pass multiplies them with tokens that are quantized as they come:

    x' = resid + gate * post_norm(branch)              wr_block_norm: one pass, which also writes
    q  = 8-bit tokens of pre_norm(x')                  the 8-bit tokens
    h  = silu(q G^T) * (q U^T)                         wr_matmul_i8 with the gate and up rows together
    qh = 8-bit tokens of h                             wr_quant_rows_i8
    out = qh D^T                                       wr_matmul_i8

``out`` is the next block's ``branch``: its residual add, gate and post norm happen in that block's norm.  Every step
runs in libwringer.so; torch only allocates.  The context may be on another stream than the caller: each call here is queued
behind the caller's work so far, and the caller's later work waits for it.  Run on synthetic modules of the container's format:
python -m post_bit_weight_amd.int8 [--tokens 64] [--hidden 2560] [--inner 9728]
"""

import argparse
import json
import time

import torch

from . import _lib as wr
from . import pipeline


class Int8Linear:
    """A linear layer's weights (rows x n, bf16 or fp32, on the GPU) as 8-bit codes and a scale per row.  Rows are
    padded to a multiple of 16 bytes, which the product reads fastest."""

    def __init__(self, ctx, weights):
        rows, n = weights.shape
        with ctx.behind_caller(weights) as made:
            self.codes = torch.empty(rows, n + -n % 16, dtype=torch.int8, device=weights.device)[:, :n]
            self.scales = torch.empty(rows, dtype=torch.float32, device=weights.device)
            made += [self.codes, self.scales]
            wr.wr_quant_rows_i8(ctx, weights, self.codes, self.scales)

    @classmethod
    def from_packed(cls, ctx, modules):
        """The rows of several packed modules one after the other.  modules: dicts with buf, rows, n_store, bits,
        group, n_out and optionally had_block and signs (as wr_materialize takes them), of one n_out."""
        n = modules[0]["n_out"]
        if any(m["n_out"] != n for m in modules):
            raise ValueError("the modules must have one n_out")
        with ctx.behind_caller(*[m.get(k) for m in modules for k in ("buf", "signs")]) as made:
            weights = torch.empty(sum(m["rows"] for m in modules), n, dtype=torch.bfloat16, device=ctx.device)
            row = 0
            for m in modules:
                wr.wr_materialize(ctx, m["buf"], m["rows"], m["n_store"], m["bits"], m["group"], weights[row:row + m["rows"]],
                                  m.get("had_block", 0), m.get("signs"))
                row += m["rows"]
            layer = cls(ctx, weights)
            made += [layer.codes, layer.scales]
        return layer


class Tokens:
    """Space for the 8-bit form of up to `most` tokens of n values."""

    def __init__(self, most, n, device):
        self.q = torch.empty(most, n + -n % 16, dtype=torch.int8, device=device)[:, :n]
        self.scales = torch.empty(most, dtype=torch.float32, device=device)

    def of(self, rows):
        return self.q[:rows], self.scales[:rows]


class Int8Mlp:
    """gate_up: Int8Linear of 2 h x n (the gate rows, then the up rows); down: Int8Linear of n x h; w_pre, w_post: the
    norms' weights (w_post may be None), gate: None or 1 x n in the activations' type."""

    def __init__(self, ctx, gate_up, down, w_pre, w_post=None, gate=None, eps=1e-6, most_tokens=4096):
        self.ctx, self.gate_up, self.down = ctx, gate_up, down
        self.w_pre, self.w_post, self.gate, self.eps = w_pre, w_post, gate, eps
        n, inner = self.gate_up.codes.shape[1], self.down.codes.shape[1]
        if self.gate_up.codes.shape[0] != 2 * inner or self.down.codes.shape[0] != n:
            raise ValueError("gate_up must be 2 h x n and down n x h")
        self.most = most_tokens
        with ctx.behind_caller(w_pre, w_post, gate, gate_up.codes, gate_up.scales, down.codes, down.scales):
            self.tokens, self.inner = Tokens(most_tokens, n, ctx.device), Tokens(most_tokens, inner, ctx.device)
            self.hidden = torch.empty(most_tokens, inner, dtype=torch.bfloat16, device=ctx.device)

    def __call__(self, resid, branch):
        """(x', the block's output) for tokens x n of the residual stream and the branch that is added to it."""
        rows = branch.shape[0]
        if rows > self.most:
            raise ValueError(f"{rows} tokens, but space for {self.most}")
        with self.ctx.behind_caller(resid, branch) as made:
            out = torch.empty_like(branch, memory_format=torch.contiguous_format)
            resid_out = torch.empty_like(resid, memory_format=torch.contiguous_format)
            q, scales = self.tokens.of(rows)
            wr.wr_block_norm(self.ctx, self.eps, branch=branch, resid=resid, w_post=self.w_post, gate=self.gate,
                             w_pre=self.w_pre, resid_out=resid_out, q=q, q_scales=scales)
            hidden = self.hidden[:rows]
            wr.wr_matmul_i8(self.ctx, q, scales, self.gate_up.codes, self.gate_up.scales, hidden, swiglu=True)
            qh, hscales = self.inner.of(rows)
            wr.wr_quant_rows_i8(self.ctx, hidden, qh, hscales)
            wr.wr_matmul_i8(self.ctx, qh, hscales, self.down.codes, self.down.scales, out)
            made += [resid_out, out]
        return resid_out, out


def synthetic_module(ctx, rows, n, bits, group, seed):
    """A packed module of random codes whose weights have a standard deviation near 0.02."""
    with ctx.behind_caller() as made:
        g = torch.Generator(device=ctx.device).manual_seed(seed)
        codes = torch.randint(0, 1 << bits, (rows, n), dtype=torch.uint8, device=ctx.device, generator=g)
        spread = 0.02 / (((1 << (2 * bits)) - 1) / 3.0) ** 0.5
        scales = ((0.75 + 0.5 * torch.rand(rows, n // group, device=ctx.device, generator=g)) * spread).to(torch.float16)
        buf = pipeline.pack(ctx, codes, scales, bits, group)
        made.append(buf)
    return dict(buf=buf, rows=rows, n_store=n, bits=bits, group=group, n_out=n)


def main(argv=None):
    ap = argparse.ArgumentParser(description="An 8-bit gated MLP on synthetic packed modules: time, and error against fp32.")
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--hidden", type=int, default=2560)
    ap.add_argument("--inner", type=int, default=9728)
    ap.add_argument("--passes", type=int, default=50)
    a = ap.parse_args(argv)
    ctx = wr.Context(0)
    gate, up, down = (synthetic_module(ctx, r, n, b, 64, s) for r, n, b, s in
                      ((a.inner, a.hidden, 2, 1), (a.inner, a.hidden, 2, 2), (a.hidden, a.inner, 3, 3)))
    g = torch.Generator(device=ctx.device).manual_seed(4)
    norm = (1 + 0.1 * torch.randn(2, a.hidden, device=ctx.device, generator=g)).to(torch.bfloat16)
    mlp = Int8Mlp(ctx, Int8Linear.from_packed(ctx, [gate, up]), Int8Linear.from_packed(ctx, [down]), norm[0], norm[1],
                  most_tokens=a.tokens)
    resid, branch = (torch.randn(a.tokens, a.hidden, device=ctx.device, generator=g).to(torch.bfloat16) for _ in range(2))
    resid_out, out = mlp(resid, branch)
    # the same block in fp32 on the materialized weights
    wide = []
    for m in (gate, up, down):
        w = torch.empty(m["rows"], m["n_out"], dtype=torch.bfloat16, device=ctx.device)
        wr.wr_materialize(ctx, m["buf"], m["rows"], m["n_store"], m["bits"], m["group"], w)
        wide.append(w.float())
    rms = lambda v: v * torch.rsqrt(v.square().mean(1, keepdim=True) + mlp.eps)  # noqa: E731
    x = resid.float() + rms(branch.float()) * norm[1].float()
    y = rms(x) * norm[0].float()
    ref = (torch.nn.functional.silu(y @ wide[0].t()) * (y @ wide[1].t())) @ wide[2].t()
    error = float((out.float() - ref).norm() / ref.norm())
    torch.cuda.synchronize()
    began = time.perf_counter()
    for _ in range(a.passes):
        mlp(resid, branch)
    torch.cuda.synchronize()
    print(json.dumps(dict(tokens=a.tokens, hidden=a.hidden, inner=a.inner, us_per_pass=round((time.perf_counter() - began) / a.passes * 1e6, 1),
                          relative_error=round(error, 5), residual_error=float((resid_out.float() - x).norm() / x.norm()))))
    return 0 if error < 0.05 else 1


if __name__ == "__main__":
    raise SystemExit(main())
