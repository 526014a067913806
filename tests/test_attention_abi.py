"""CPU checks of the attention operators' C entry points: every refusal comes before any device call.

The checks read nothing of the context, so a zeroed buffer stands in for one, and addresses that are only looked at
stand in for device memory.
"""
import ctypes
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "post_bit_weight_amd", "libwringer.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="library not built")

CTX = ctypes.create_string_buffer(1024)
A = 1 << 20   # an aligned address
ODD = A + 1
F32, BF16 = 0, 1
OK, EINVAL, EUNSUPPORTED = 0, 1, 4


@pytest.fixture(scope="module")
def wr():
    from post_bit_weight_amd import _lib
    return _lib


@pytest.fixture(scope="module")
def lib(wr):
    return wr.load()


def call(fn, usual, **changes):
    args = dict(usual, **changes)
    return fn(*args.values())


ROTARY = dict(ctx=CTX, x=A, dtype=BF16, rows=4, heads=2, dim=64, ldx=128, pairs=32, positions=A, axes=2, ldp=4, axis_of=A, freqs=A,
              flags=0, y=A + 4096, ldy=128)


@pytest.mark.parametrize("change", [dict(ctx=None), dict(x=None), dict(y=None), dict(x=ODD), dict(y=ODD), dict(dtype=2), dict(rows=-1), dict(heads=0),
                                    dict(dim=0), dict(dim=-64), dict(ldx=127), dict(ldy=127), dict(pairs=33), dict(pairs=-1), dict(positions=None),
                                    dict(positions=A + 2), dict(axes=0), dict(ldp=3), dict(axis_of=None), dict(axis_of=A + 1), dict(freqs=None),
                                    dict(freqs=A + 4), dict(flags=4), dict(rows=1 << 31), dict(y=A, ldy=129)])
def test_rotary_refusals(lib, change):
    assert call(lib.wr_rotary, ROTARY, **change) == EINVAL


def test_rotary_limits_and_nothing(lib):
    assert call(lib.wr_rotary, ROTARY, dim=1026, ldx=4000, ldy=4000) == EUNSUPPORTED
    assert call(lib.wr_rotary, ROTARY, axes=9) == EUNSUPPORTED
    assert call(lib.wr_rotary, ROTARY, rows=0, x=None, y=None, positions=None, freqs=None, axis_of=None) == OK


def cache(wr, **changes):
    return wr._KvCache(**dict(dict(pages=A, count=4, heads=2, dim=64, page_tokens=16, group=32), **changes))


def seqs(wr, **changes):
    return wr._KvSeqs(**dict(dict(starts=A, lengths=A, table=A, ldt=4, n=2, width=4, most_new=3, most_tokens=64), **changes))


def test_page_bytes(lib):
    assert lib.wr_kv_page_bytes(2, 64, 16, 32) == 2 * 16 * (64 + 16)
    assert lib.wr_kv_page_bytes(8, 128, 64, 64) == 8 * 64 * (128 + 16)
    for bad in ((0, 64, 16, 32), (2, 96, 16, 32), (2, 64, 8, 32), (2, 64, 48, 32), (2, 64, 512, 32), (2, 64, 16, 128), (2, 64, 16, 16),
                (70000, 64, 16, 32)):
        assert lib.wr_kv_page_bytes(*bad) == 0


ROWS = dict(k=A, ldk=128, v=A, ldv=128, dtype=BF16, rows=6)
BAD_ROWS = [dict(k=None, v=None), dict(k=ODD), dict(v=ODD), dict(ldk=127), dict(ldv=127), dict(dtype=3), dict(rows=-1), dict(rows=1 << 31)]
BAD_CACHE = [dict(pages=None), dict(pages=A + 8), dict(count=0), dict(count=-1)]
BAD_SEQS = [dict(starts=None), dict(lengths=None), dict(table=None), dict(starts=ODD), dict(lengths=ODD), dict(table=A + 2), dict(n=-1), dict(ldt=3),
            dict(width=-1), dict(most_new=-1), dict(most_tokens=-1)]


@pytest.mark.parametrize("name", ["wr_kv_write", "wr_kv_read"])
def test_write_and_read_refusals(lib, wr, name):
    fn = getattr(lib, name)

    def run(c=None, s=None, ctx=CTX, **rows):
        return fn(ctx, ctypes.byref(c or cache(wr)), ctypes.byref(s or seqs(wr)), *dict(ROWS, **rows).values())

    for change in BAD_ROWS:
        assert run(**change) == EINVAL, change
    for change in BAD_CACHE:
        assert run(c=cache(wr, **change)) == EINVAL, change
    for change in BAD_SEQS:
        assert run(s=seqs(wr, **change)) == EINVAL, change
    assert run(ctx=None) == EINVAL
    assert fn(CTX, None, ctypes.byref(seqs(wr)), *ROWS.values()) == EINVAL
    assert fn(CTX, ctypes.byref(cache(wr)), None, *ROWS.values()) == EINVAL
    assert run(c=cache(wr, dim=96)) == EUNSUPPORTED
    assert run(s=seqs(wr, n=1 << 30, most_new=1 << 20)) == EUNSUPPORTED
    for nothing in (dict(rows=0, k=None, v=None), dict(s=seqs(wr, n=0, starts=None, lengths=None, table=None)), dict(s=seqs(wr, most_new=0))):
        assert run(**nothing) == OK


ATTEND = dict(q=A, ldq=256, rows=6, heads=4, scale=0.125, flags=1, window=0, out=A, ldo=256)


def test_attention_refusals(lib, wr):
    def run(c=None, s=None, ctx=CTX, **changes):
        return lib.wr_kv_attention(ctx, ctypes.byref(c or cache(wr)), ctypes.byref(s or seqs(wr)), *dict(ATTEND, **changes).values())

    for change in (dict(q=None), dict(out=None), dict(q=ODD), dict(out=ODD), dict(ldq=255), dict(ldo=255), dict(rows=-1), dict(heads=0), dict(heads=3),
                   dict(heads=-2), dict(scale=float("nan")), dict(scale=float("inf")), dict(flags=2), dict(window=-1), dict(ctx=None)):
        assert run(**change) == EINVAL, change
    for change in BAD_CACHE:
        assert run(c=cache(wr, **change)) == EINVAL, change
    for change in BAD_SEQS:
        assert run(s=seqs(wr, **change)) == EINVAL, change
    assert run(heads=130, ldq=1 << 20, ldo=1 << 20) == EUNSUPPORTED
    assert run(c=cache(wr, group=16)) == EUNSUPPORTED
    assert run(s=seqs(wr, most_new=2147483647)) == EUNSUPPORTED
    assert run(rows=0, q=None, out=None) == OK


ADAPTERS = dict(ctx=CTX, x=A, x_dtype=BF16, rows=6, n=64, ldx=64, A=A, B=A, adapters=2, rank=8, outs=32, scales=A, ranks=None, starts=A, ids=A,
                n_seqs=2, most=4, base=A, ldb=32, y=A + 8192, y_dtype=F32, ldy=32)


@pytest.mark.parametrize("change", [dict(ctx=None), dict(x=None), dict(A=None), dict(B=None), dict(scales=None), dict(starts=None), dict(ids=None),
                                    dict(y=None), dict(x=ODD), dict(A=ODD), dict(B=ODD), dict(scales=A + 2), dict(ranks=A + 2), dict(starts=A + 2),
                                    dict(ids=ODD), dict(y=A + 2), dict(base=A + 2), dict(ldx=63), dict(ldb=31), dict(ldy=31), dict(rows=-1), dict(n=0),
                                    dict(adapters=-1), dict(rank=-1), dict(outs=-1), dict(n_seqs=-1), dict(most=-1), dict(x_dtype=2), dict(y_dtype=5),
                                    dict(rows=1 << 31), dict(base=A + 8192, ldb=33)])
def test_adapters_refusals(lib, change):
    assert call(lib.wr_adapters, ADAPTERS, **change) == EINVAL


def test_adapters_limits_and_nothing(lib):
    assert call(lib.wr_adapters, ADAPTERS, rank=257) == EUNSUPPORTED
    assert call(lib.wr_adapters, ADAPTERS, rows=0, x=None, y=None) == OK
    assert call(lib.wr_adapters, ADAPTERS, n_seqs=0, starts=None, ids=None) == OK
    assert call(lib.wr_adapters, ADAPTERS, most=0) == OK
    assert call(lib.wr_adapters, ADAPTERS, outs=0, y=None) == OK


def test_lengths_that_an_int32_would_not_hold(lib, wr):
    """A table so wide that a sequence could have more than 2^30 positions, and a scale that log2(e) takes out of range."""
    for s in (seqs(wr, width=1 << 28, ldt=1 << 28, most_tokens=(1 << 30) + 1), seqs(wr, most_new=(1 << 30) + 1)):
        assert lib.wr_kv_write(CTX, ctypes.byref(cache(wr)), ctypes.byref(s), *ROWS.values()) == EUNSUPPORTED
        assert lib.wr_kv_attention(CTX, ctypes.byref(cache(wr)), ctypes.byref(s), *ATTEND.values()) == EUNSUPPORTED
    for scale in (1.7e38, -3e38):
        assert lib.wr_kv_attention(CTX, ctypes.byref(cache(wr)), ctypes.byref(seqs(wr)), *dict(ATTEND, scale=scale).values()) == EUNSUPPORTED


def test_attention_does_not_write_over_its_queries(lib, wr):
    assert lib.wr_kv_attention(CTX, ctypes.byref(cache(wr)), ctypes.byref(seqs(wr)), *dict(ATTEND, q=A, out=A).values()) == EINVAL
