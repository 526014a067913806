"""The attention half of a block on packed modules, a prompt in two chunks and then single tokens, against the fp64 block.

The oracle takes keys and values as the cache holds them (read back), everything else from the materialized weights in
fp64.  Rounding to 8 bits costs each of the two products' two factors 0.6 % to 1 % of the rms, as in the MLP's test; the
queries' error changes a score by a part of itself, which the softmax passes on at most twice: 4 % in all, held to 6 %.
"""
import os
import re

import numpy as np
import pytest
import torch

import oracle
from attention_inputs import BF16, F32, int32

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def build(heads, cache_heads, dim, n, page, group, most, seqs, adapted, window=0, stream=None, seed=1, interleaved=False):
    from post_bit_weight_amd import _lib as wr
    from post_bit_weight_amd import attention, int8
    ctx = wr.Context(0, stream)
    wide, kv = heads * dim, cache_heads * dim
    mods = [int8.synthetic_module(ctx, r, c, b, 64, seed + i) for i, (r, c, b) in enumerate(((wide, n, 2), (kv, n, 3), (kv, n, 2), (n, wide, 4)))]
    g = torch.Generator().manual_seed(seed + 9)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = dict(w_pre=1 + 0.2 * r(n), w_post=1 + 0.2 * r(n), q_norm=(1 + 0.2 * r(dim)), k_norm=(1 + 0.2 * r(dim)),
             freqs=10000.0 ** (-torch.arange(dim // 2, dtype=torch.float64) * 2 / dim), axis_of=torch.arange(dim // 2, dtype=torch.int32) % 2)
    p = {k: t.cuda() for k, t in p.items()}
    pool = {}
    if adapted:
        for name, i, o in (("q", n, wide), ("k", n, kv), ("v", n, kv), ("out", wide, n)):
            pool[name] = attention.Adapters((r(2, 8, i) * i ** -0.5).to(BF16).cuda(), (r(2, o, 8) * 0.2).to(BF16).cuda(), torch.tensor([0.5, 1.5]).cuda())
    width = -(-most // page)
    cache = wr.KvCache(seqs * width + 1, cache_heads, dim, page_tokens=page, group=group)
    table = int32(np.random.default_rng(seed).permutation(seqs * width).reshape(seqs, width))
    torch.cuda.synchronize()
    block = attention.Int8Attention(ctx, int8.Int8Linear.from_packed(ctx, mods[:3]), int8.Int8Linear.from_packed(ctx, mods[3:]), cache,
                                    window=window, interleaved=interleaved, most_tokens=300, adapters=pool, **p)
    weights = [oracle.materialize_exact(m["buf"].cpu().numpy(), m["rows"], m["n_store"], m["bits"], m["group"], 0, None, m["n_out"]) for m in mods]
    return wr, ctx, block, cache, table, p, pool, weights


def h64(t):
    return None if t is None else t.double().cpu().numpy()


def reference(wr, ctx, block, cache, table, p, pool, weights, resid, branch, new, lengths, positions, ids):
    x, y, _ = oracle.block_norm(block.eps, branch=h64(branch), resid=h64(resid), w_post=h64(p["w_post"]), gate=None, w_pre=h64(p["w_pre"]))
    starts = np.concatenate([[0], np.cumsum(new)])

    def adapted(name, x, z):
        a = pool.get(name)
        return z if a is None else oracle.adapters(x, z, h64(a.A), h64(a.B), h64(a.scales), starts, ids)

    dim, heads, kv = cache.dim, block.wide // cache.dim, cache.heads
    q = adapted("q", y, y @ weights[0].T).reshape(-1, dim)
    q = (q / np.sqrt((q * q).mean(1, keepdims=True) + block.eps) * h64(p["q_norm"])).reshape(len(y), -1)
    q = oracle.rotary(q, positions, h64(p["freqs"]), dim, p["axis_of"].cpu().numpy(), block.interleaved).reshape(-1, heads, dim)
    att = np.zeros((len(y), heads, dim))
    for s, (n, length) in enumerate(zip(new, lengths)):
        every = wr.Sequences(int32([0, length]), int32([length]), table[s:s + 1], length, length)
        k, v = (torch.empty(length, kv * dim, dtype=F32, device="cuda") for _ in range(2))
        wr.wr_kv_read(ctx, cache, every, k, v)
        torch.cuda.synchronize()
        k, v = (h64(t).reshape(length, kv, dim) for t in (k, v))
        ok = oracle.sees(length - n, n, length, window=block.window)
        for h in range(heads):
            att[starts[s]:starts[s + 1], h] = oracle.attend(q[starts[s]:starts[s + 1], h], k[:, h * kv // heads], v[:, h * kv // heads], ok, block.scale)[0]
    att = att.reshape(len(y), -1)
    return x, adapted("out", att, att @ weights[3].T)


@pytest.mark.parametrize("heads,cache_heads,dim,n,page,group,adapted,window,other,interleaved",
                         [(8, 2, 64, 256, 16, 32, False, 0, False, False), (4, 4, 128, 320, 32, 64, True, 0, True, False),
                          (6, 3, 64, 192, 64, 64, True, 50, False, True)])
def test_prompt_in_chunks_then_tokens(heads, cache_heads, dim, n, page, group, adapted, window, other, interleaved):
    stream = torch.cuda.Stream() if other else None
    wr, ctx, block, cache, table, p, pool, weights = build(heads, cache_heads, dim, n, page, group, 130, 3, adapted, window, stream, interleaved=interleaved)
    g = torch.Generator().manual_seed(6)
    lengths, ids = [0, 0, 0], [1, -1, 0]
    for new in ([100, 37, 5], [20, 0, 61], [1, 1, 1], [1, 0, 1]):
        lengths = [a + b for a, b in zip(lengths, new)]
        rows = sum(new)
        pos = np.concatenate([np.arange(length - b, length) for b, length in zip(new, lengths)])
        positions = np.stack([pos, pos // 3])
        resid, branch = torch.randn(rows, n, generator=g).cuda(), torch.randn(rows, n, generator=g).to(BF16).cuda()
        seqs = wr.Sequences(int32(np.concatenate([[0], np.cumsum(new)])), int32(lengths), table, 100, 130)
        resid_out, out = block(resid, branch, seqs, int32(positions), int32(ids) if adapted else None)
        torch.cuda.synchronize()
        x, ref = reference(wr, ctx, block, cache, table, p, pool, weights, resid, branch, new, lengths, positions, ids)
        assert np.abs(h64(resid_out) - x).max() <= 1e-5 * np.abs(x).max()
        assert np.linalg.norm(h64(out) - ref) <= 0.06 * np.linalg.norm(ref), (new, np.linalg.norm(h64(out) - ref) / np.linalg.norm(ref))


def test_a_recorded_step_is_replayed():
    """One step of single tokens recorded in a graph and replayed with new inputs: bit for bit what the eager calls give."""
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        wr, ctx, block, cache, table, p, pool, weights = build(8, 2, 64, 256, 16, 32, 400, 3, True, stream=stream)
        n, lengths, g = 256, [300, 20, 111], torch.Generator().manual_seed(7)
        resid, branch = torch.zeros(3, n, device="cuda"), torch.zeros(3, n, dtype=BF16, device="cuda")
        positions, ids = int32(np.zeros((2, 3))), int32([0, 1, -1])
        seqs = wr.Sequences(int32([0, 1, 2, 3]), int32(lengths), table, 1, 400)
        cache.buf.zero_()
        block(resid, branch, seqs, positions, ids)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            resid_out, out = block(resid, branch, seqs, positions, ids)
        for i in range(5):
            resid.copy_(torch.randn(3, n, generator=g)), branch.copy_(torch.randn(3, n, generator=g))
            seqs.lengths.add_(1), positions.add_(1)
            graph.replay()
            stream.synchronize()
            got = resid_out.clone(), out.clone()
            want = block(resid, branch, seqs, positions, ids)
            stream.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals():
    wr, ctx, block, cache, table, p, pool, weights = build(8, 2, 64, 256, 16, 32, 64, 1, False)
    from post_bit_weight_amd import attention, int8
    x, b = torch.zeros(1, 256, device="cuda"), torch.zeros(1, 256, dtype=BF16, device="cuda")
    seqs = wr.Sequences(int32([0, 1]), int32([1]), table, 1, 64)
    for args in ((x, b, seqs), (x, b, seqs, int32([[0], [0]]), int32([0]))):
        with pytest.raises(ValueError):
            block(*args)
    many = torch.zeros(301, 256, device="cuda")
    with pytest.raises(ValueError):
        block(many, many.to(BF16), seqs, int32(np.zeros((2, 301))))
    qkv = int8.Int8Linear(ctx, torch.zeros(768, 256, device="cuda"))
    out = int8.Int8Linear(ctx, torch.zeros(256, 512, device="cuda"))
    attention.Int8Attention(ctx, qkv, out, cache, p["w_pre"])
    for bad in (dict(qkv=out), dict(out=qkv), dict(adapters={"gate": None})):
        with pytest.raises(ValueError):
            attention.Int8Attention(**dict(dict(ctx=ctx, qkv=qkv, out=out, cache=cache, w_pre=p["w_pre"]), **bad))


def test_command_prints_a_line(capsys):
    from post_bit_weight_amd import attention
    args = "--sequences 3 --prompt 70 --steps 4 --hidden 256 --heads 4 --cache-heads 2 --dim 64 --page 16 --group 32 --adapters 2 --rank 4"
    assert attention.main(args.split()) == 0
    assert "us_per_step" in capsys.readouterr().out


@pytest.mark.skipif(not os.path.exists(README), reason="this copy is without its documents")
def test_the_calls_in_the_readme():
    """Its step of four sequences runs, and the attention is the oracle's: one token each, which a softmax gives back."""
    from post_bit_weight_amd import _lib as wr
    with open(README) as f:
        code = re.findall(r"```python\n(.*?)```", f.read(), re.S)[1]
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
    space = dict(wr=wr, context=wr.Context(0), starts=int32(range(5)), lengths=int32([1] * 4), table=int32([[3], [0], [7], [5]]), q=r(4, 4096),
                 k=r(4, 1024), v=r(4, 1024), out=torch.empty(4, 4096, dtype=BF16, device="cuda"), positions=int32([0] * 4),
                 freqs=torch.ones(64, dtype=torch.float64, device="cuda"), A=r(2, 8, 4096), B=r(2, 64, 8), scales=torch.ones(2, device="cuda"),
                 ids=int32([-1] * 4), y=r(4, 64))
    before = space["y"].clone()
    exec(code, space)
    torch.cuda.synchronize()
    x = space["v"].double().cpu().numpy().reshape(4, 8, 128)
    want = np.repeat(oracle.kv_values(*oracle.kv_codes(x, 64), 64), 4, axis=1).reshape(4, -1)
    # the value and the weight rounded to fp16, the output to bf16
    assert (np.abs(h64(space["out"]) - want) <= (2.0 ** -10 + 2.0 ** -8) * np.abs(want) + 2.0 ** -24).all()
    assert torch.equal(space["y"], before)  # no request has an adapter


def test_rows_behind_the_last_sequence_and_no_rows():
    """A padded batch gives the sequences' rows what they get without padding; a batch of none gives none."""
    wr, ctx, block, cache, table, p, pool, weights = build(8, 2, 64, 256, 16, 32, 60, 2, True)
    g = torch.Generator().manual_seed(8)
    resid, branch = torch.randn(50, 256, generator=g).cuda(), torch.randn(50, 256, generator=g).to(BF16).cuda()
    positions, ids = int32(np.stack([np.arange(50), np.arange(50)])), int32([1, -1])
    seqs = wr.Sequences(int32([0, 30, 37]), int32([30, 7]), table, 30, 60)
    whole = block(resid, branch, seqs, positions, ids)
    alone = block(resid[:37], branch[:37], seqs, positions[:, :37].contiguous(), ids)
    torch.cuda.synchronize()
    assert all(torch.equal(a[:37], b) for a, b in zip(whole, alone))
    none = block(resid[:0], branch[:0], seqs, positions[:, :0].contiguous(), ids)
    assert none[0].shape == (0, 256) and none[1].shape == (0, 256)
