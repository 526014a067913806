"""Which stream the 8-bit MLP's work and memory are on, with a stand-in for streams and library (no GPU)."""
import contextlib
import types

import pytest
import torch

from post_bit_weight_amd import _lib, int8

CALLS = ("wr_block_norm", "wr_matmul_i8", "wr_quant_rows_i8", "wr_materialize", "wr_pack")


class Stream:
    def __init__(self, name, log):
        self.name, self.log, self.cuda_stream = name, log, id(self)

    def wait_stream(self, other):
        self.log.append(("wait", self.name, other.name))


class World:
    """Keeps the current stream, on which stream each memory block was allocated and for which others it was recorded."""

    def __init__(self, monkeypatch):
        self.log, self.made, self.recorded = [], {}, {}
        self.caller, self.own = Stream("caller", self.log), Stream("own", self.log)
        self.current = [self.caller]
        library = types.SimpleNamespace(wr_create=lambda *a: 0, wr_destroy=lambda *a: 0)

        @contextlib.contextmanager
        def on(stream):
            self.current.append(stream)
            try:
                yield
            finally:
                self.current.pop()

        def allocates(make):
            def wrapped(*args, **kw):
                t = make(*args, **kw)
                self.made[self.block(t)] = self.current[-1].name
                return t
            return wrapped

        def call(name):
            def wrapped(ctx, *args, **kw):
                tensors = [a for a in (*args, *kw.values()) if torch.is_tensor(a)]
                self.log.append((name, self.current[-1].name, [self.block(t) for t in tensors]))
            return wrapped

        monkeypatch.setattr(_lib, "load", lambda: library)
        monkeypatch.setattr(_lib, "packed_nbytes", lambda rows, n, bits, group: rows * n)
        for name in CALLS:
            monkeypatch.setattr(_lib, name, call(name))
        monkeypatch.setattr(torch.cuda, "stream", on)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.current[-1])
        monkeypatch.setattr(_lib, "_raw_stream", lambda device: self.current[-1].cuda_stream)
        for name in ("empty", "empty_like", "randint", "rand"):
            monkeypatch.setattr(torch, name, allocates(getattr(torch, name)))
        monkeypatch.setattr(torch.Tensor, "record_stream",
                            lambda t, stream: self.recorded.setdefault(self.block(t), set()).add(stream.name))

    @staticmethod
    def block(t):
        return t.untyped_storage().data_ptr()


@pytest.fixture
def world(monkeypatch):
    return World(monkeypatch)


def ordered(log):
    """Every call is on the context's stream, after a wait for the caller, and the caller waits after the last one."""
    calls = [k for k, entry in enumerate(log) if entry[0] in CALLS]
    return (bool(calls) and all(log[k][1] == "own" for k in calls) and ("wait", "own", "caller") in log[:calls[0]]
            and ("wait", "caller", "own") in log[calls[-1]:])


def test_layers_and_passes_from_another_stream(world):
    ctx = _lib.Context("cpu", world.own)
    keep = [int8.synthetic_module(ctx, *shape, 2, 64, 1) for shape in ((256, 128), (128, 128))]
    assert ordered(world.log)
    assert all("caller" in world.recorded[world.block(m["buf"])] for m in keep)
    signs = torch.ones(128, dtype=torch.int8)
    world.made[world.block(signs)] = "caller"
    keep[0].update(had_block=64, signs=signs)
    for m in keep:  # as if the caller had loaded them
        world.made[world.block(m["buf"])] = "caller"
        world.recorded.clear()
    del world.log[:]
    layers = [int8.Int8Linear.from_packed(ctx, [m]) for m in keep]
    assert ordered(world.log)
    w = torch.ones(128)
    world.made[world.block(w)] = "caller"
    mlp = int8.Int8Mlp(ctx, *layers, w, most_tokens=8)
    del world.log[:]
    resid, branch = torch.zeros(4, 128), torch.zeros(4, 128)
    for t in (resid, branch):
        world.made[world.block(t)] = "caller"
    outs = mlp(resid, branch)
    assert ordered(world.log)
    # the allocator hands a block on in the order of the stream it was allocated on, and of those it was recorded for
    for entry in world.log:
        if entry[0] in CALLS:
            for block in entry[2]:
                assert world.made[block] == "own" or "own" in world.recorded[block], entry[0]
    for t in outs:
        assert world.made[world.block(t)] == "own" and "caller" in world.recorded[world.block(t)]
    for m in keep:
        assert "own" in world.recorded[world.block(m["buf"])]
    assert "own" in world.recorded[world.block(signs)]


def test_an_error_inside_leaves_the_streams_as_they_were(world):
    ctx = _lib.Context("cpu", world.own)
    with pytest.raises(KeyError):
        with ctx.behind_caller():
            raise KeyError
    assert world.current == [world.caller] and world.log == [("wait", "own", "caller"), ("wait", "caller", "own")]


def test_nothing_is_done_on_the_contexts_own_stream(world):
    ctx = _lib.Context("cpu", world.caller)
    with ctx.behind_caller(torch.zeros(1)) as made:
        made.append(torch.zeros(1))
    assert world.log == [] and world.recorded == {}
