"""A context's workspace and stream on the GPU: recorded graphs, workspaces that grow, calls from another stream."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def wr():
    from post_bit_weight_amd import _lib
    return _lib


def gradient_inputs(rows, n, gate_rows, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)  # noqa: E731
    inp = dict(branch=r(rows, n), resid=r(rows, n), w_post=r(n), w_pre=r(n), gate=r(-(-rows // gate_rows), n), gate_rows=gate_rows)
    return inp, dict(dy=r(rows, n), dresid_out=r(rows, n)), torch.rand(rows, 2, generator=g, device="cuda") + 0.5


def gradient_outputs(inp):
    rows, n = inp["branch"].shape
    new = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    return dict(dbranch=new(rows, n).to(BF16), dresid=new(rows, n).to(BF16), dw_post=new(n), dw_pre=new(n),
                dgate=new(*inp["gate"].shape))


def test_a_recorded_graph_keeps_its_workspace(wr):
    """A gradient recorded with a small workspace, replayed after a larger one has replaced it and other tensors have been
    made: the gradient is right at every replay and no other tensor changes."""
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        c = wr.Context(0, stream)
        inp, up, stats = gradient_inputs(300, 2560, 50, 1)
        eager, replayed = gradient_outputs(inp), gradient_outputs(inp)
        wr.wr_block_norm_backward(c, stats, **inp, **up, **eager)
        small = c.workspace.numel()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            wr.wr_block_norm_backward(c, stats, **inp, **up, **replayed)
        large = gradient_inputs(5000, 9728, 1000, 2)
        wr.wr_block_norm_backward(c, large[2], **large[0], **large[1], **gradient_outputs(large[0]))
        assert c.workspace.numel() > small
        others = [torch.full((small // 4 // k,), 77.0, device="cuda") for k in (1, 1, 2, 2, 4, 4)]
        for k in range(3):
            up["dy"].copy_(torch.randn(300, 2560, device="cuda"))
            for t in replayed.values():
                t.zero_()
            graph.replay()
            wr.wr_block_norm_backward(c, stats, **inp, **up, **eager)
            stream.synchronize()
            assert all(torch.equal(eager[name], replayed[name]) for name in eager)
            assert all(bool((t == 77).all()) for t in others)


def test_mlp_on_a_stream_of_its_own(wr):
    """Modules loaded, run and dropped from the caller's stream with the context on another: the bits of a context on the
    caller's, while the caller's stream keeps allocating."""
    from post_bit_weight_amd import int8

    def run(ctx):
        mods = [int8.synthetic_module(ctx, r, k, b, 64, s) for r, k, b, s in ((4096, 1024, 2, 1), (4096, 1024, 2, 2), (1024, 4096, 3, 3))]
        up, down = int8.Int8Linear.from_packed(ctx, mods[:2]), int8.Int8Linear.from_packed(ctx, mods[2:])
        del mods
        noise = [torch.full((8192, 1024), 3.0, device="cuda").to(BF16) for _ in range(4)]  # the size of dropped weights
        g = torch.Generator(device="cuda").manual_seed(6)
        w = (1 + 0.1 * torch.randn(1024, generator=g, device="cuda")).to(BF16)
        mlp = int8.Int8Mlp(ctx, up, down, w, w.clone(), most_tokens=600)
        outs = []
        for _ in range(5):
            resid, branch = (torch.randn(600, 1024, generator=g, device="cuda").to(BF16) for _ in range(2))
            outs += [t.float().sum(1) for t in mlp(resid, branch)]
            del resid, branch
            noise.append(torch.full((600, 1024), 5.0, device="cuda").to(BF16))
        torch.cuda.synchronize()
        return up.codes.clone(), up.scales.clone(), *outs

    here = run(wr.Context(0))
    apart = run(wr.Context(0, torch.cuda.Stream()))
    assert all(torch.equal(a, b) for a, b in zip(here, apart))


def test_workspace_that_grows_on_a_stream_of_its_own(wr):
    """Gradients of more and more tokens are right while the caller's stream allocates what the workspaces leave."""
    stream = torch.cuda.Stream()
    here, apart = wr.Context(0), wr.Context(0, stream)
    for rows, n in ((40, 640), (300, 2560), (2000, 5120)):
        inp, up, stats = gradient_inputs(rows, n, 7, rows)
        a, b = gradient_outputs(inp), gradient_outputs(inp)
        wr.wr_block_norm_backward(here, stats, **inp, **up, **a)
        with apart.behind_caller(stats, *up.values(), *(t for t in inp.values() if torch.is_tensor(t))) as made:
            wr.wr_block_norm_backward(apart, stats, **inp, **up, **b)
            made += b.values()
        noise = [torch.full((here.workspace.numel() // 4,), 7.0, device="cuda") for _ in range(3)]
        assert all(torch.equal(a[k], b[k]) for k in a)
        assert all(bool((t == 7).all()) for t in noise)
