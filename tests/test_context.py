"""The context's workspace, with a stand-in for the library (no GPU)."""
import contextlib
import types

import pytest
import torch

from post_bit_weight_amd import _lib


class Library:
    """Records the workspaces that are registered."""

    def __init__(self):
        self.registered = []

    def wr_create(self, handle, device, stream):
        return 0

    def wr_destroy(self, handle):
        return 0

    def wr_set_workspace(self, handle, address, size):
        self.registered.append((address.value, size))
        return 0


@pytest.fixture
def library(monkeypatch):
    lib = Library()
    lib.current = []  # the streams made current, the innermost last

    @contextlib.contextmanager
    def on(stream):
        lib.current.append(stream)
        yield
        lib.current.pop()

    monkeypatch.setattr(_lib, "load", lambda: lib)
    monkeypatch.setattr(torch.cuda, "stream", on)
    return lib


def context():
    return _lib.Context("cpu", types.SimpleNamespace(cuda_stream=0))


def test_a_replaced_workspace_stays(library):
    """A graph recorded with it holds its address: no later tensor may get its memory while the context lives."""
    ctx = context()
    ctx.ensure_workspace(1 << 20)
    first = library.registered[0][0]
    for size in (2 << 20, 4 << 20, 8 << 20):
        ctx.ensure_workspace(size)
    later = [torch.empty(1 << 20, dtype=torch.uint8) for _ in range(16)]
    held = [t for t in ctx.replaced if t.data_ptr() == first]
    assert held and all(abs(t.data_ptr() - first) >= 1 << 20 for t in later)
    assert ctx.workspace.numel() == 8 << 20 and library.registered[-1] == (ctx.workspace.data_ptr(), 8 << 20)


def test_workspaces_grow_by_half_at_least(library):
    """Many sizes, each a little larger, do not leave as many workspaces behind."""
    ctx = context()
    for size in range(1000, 100000, 100):
        ctx.ensure_workspace(size)
        assert ctx.workspace.numel() >= size
        assert library.registered[-1] == (ctx.workspace.data_ptr(), ctx.workspace.numel())
    assert len(library.registered) <= 13 and sum(t.numel() for t in ctx.replaced) <= 2 * ctx.workspace.numel()


def test_the_first_workspace_is_what_was_asked_for(library):
    ctx = context()
    ctx.ensure_workspace(0)
    assert ctx.workspace.numel() == 256
    ctx.ensure_workspace(100)
    ctx.ensure_workspace(5000)
    assert [size for _, size in library.registered] == [256, 5000] and ctx.workspace.numel() == 5000


def test_a_workspace_belongs_to_the_contexts_stream(library, monkeypatch):
    """The allocator orders a block's next use after its last one on the stream that was current when it was allocated."""
    ctx = context()
    made_on = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made_on.append(library.current[-1:]) or empty(*a, **k))
    ctx.ensure_workspace(1 << 20)
    ctx.ensure_workspace(4 << 20)
    assert made_on == [[ctx.stream], [ctx.stream]]
