"""CPU checks of the block operators' C entry points: every refusal comes before any device call.

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
def lib():
    from post_bit_weight_amd import _lib
    return _lib.load()


def call(fn, base, **changes):
    args = dict(base, **changes)
    return fn(*args.values())


QUANT = dict(ctx=CTX, x=A, x_dtype=BF16, rows=4, n=64, ldx=64, q=A, ldq=64, scales=A)


@pytest.mark.parametrize("change", [dict(ctx=None), dict(x=None), dict(q=None), dict(scales=None), dict(x_dtype=7), dict(rows=-1),
                                    dict(n=0), dict(ldx=63), dict(ldq=63), dict(x=ODD), dict(scales=A + 2), dict(rows=1 << 31)])
def test_quant_rows_refusals(lib, change):
    assert call(lib.wr_quant_rows_i8, QUANT, **change) == EINVAL


def test_quant_rows_of_nothing(lib):
    assert call(lib.wr_quant_rows_i8, QUANT, rows=0, x=None, q=None, scales=None) == OK


MATMUL = dict(ctx=CTX, x=A, ldx=64, xs=A, batch=4, w=A, ldw=64, ws=A, rows=8, n=64, bias=None, flags=0, y=A, y_dtype=F32, ldy=8)


@pytest.mark.parametrize("change", [dict(ctx=None), dict(x=None), dict(w=None), dict(xs=None), dict(ws=None), dict(y=None),
                                    dict(flags=2), dict(flags=1, rows=7), dict(ldx=63), dict(ldw=63), dict(ldy=7), dict(batch=-1),
                                    dict(rows=-2), dict(n=-1), dict(y_dtype=2), dict(y=A + 2), dict(bias=ODD), dict(xs=ODD),
                                    dict(rows=1 << 30), dict(batch=1 << 31)])
def test_matmul_refusals(lib, change):
    assert call(lib.wr_matmul_i8, MATMUL, **change) == EINVAL


def test_matmul_limits_and_nothing(lib):
    assert call(lib.wr_matmul_i8, MATMUL, n=131072, ldx=131072, ldw=131072) == EUNSUPPORTED
    assert call(lib.wr_matmul_i8, MATMUL, batch=0, x=None, xs=None, y=None) == OK
    assert call(lib.wr_matmul_i8, MATMUL, rows=0, w=None, ws=None, y=None) == OK


NORM = dict(ctx=CTX, rows=4, n=64, branch=A, b_dtype=BF16, ldb=64, w_post=A, gate=A, ldg=64, gate_rows=2, bscale=1.0, resid=A,
            r_dtype=F32, ldr=64, rscale=1.0, w_pre=A, w_dtype=BF16, eps=1e-6, resid_out=A, ldo=64, y=A, ldy=64, q=A, ldq=64,
            q_scales=A, stats=A)
SHARED = [dict(ctx=None), dict(rows=-1), dict(n=0), dict(branch=None), dict(branch=None, resid=None, w_post=None, gate=None),
          dict(branch=None, w_post=None), dict(b_dtype=3), dict(r_dtype=-1), dict(w_dtype=9), dict(gate_rows=-1),
          dict(bscale=float("nan")), dict(rscale=float("inf")), dict(ldb=63), dict(ldr=10), dict(ldg=63), dict(branch=ODD),
          dict(resid=A + 2), dict(w_post=ODD), dict(gate=ODD), dict(rows=1 << 31)]


@pytest.mark.parametrize("change", SHARED + [dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(w_pre=None),
                                             dict(q_scales=None), dict(q=None), dict(ldo=63), dict(ldy=63), dict(ldq=63),
                                             dict(y=ODD), dict(resid_out=A + 2), dict(stats=ODD),
                                             dict(resid_out=None, y=None, q=None, q_scales=None, stats=None)])
def test_norm_refusals(lib, change):
    assert call(lib.wr_block_norm, NORM, **change) == EINVAL


def test_norm_limits_and_nothing(lib):
    wide = dict(n=16385, ldb=16385, ldr=16385, ldg=16385, ldo=16385, ldy=16385, ldq=16385)
    assert call(lib.wr_block_norm, NORM, **wide) == EUNSUPPORTED
    assert call(lib.wr_block_norm, NORM, rows=0) == OK


BACK = dict(ctx=CTX, rows=4, n=64, branch=A, b_dtype=BF16, ldb=64, w_post=A, gate=A, ldg=64, gate_rows=2, bscale=1.0, resid=A,
            r_dtype=F32, ldr=64, rscale=1.0, w_pre=A, w_dtype=BF16, stats=A, dy=A, lddy=64, dres=A, lddo=64, db=A, lddb=64, dx=A,
            lddr=64, dw_post=A, dgate=A, dw_pre=A)


@pytest.mark.parametrize("change", SHARED + [dict(dy=None, dres=None, dw_pre=None), dict(w_pre=None), dict(stats=None),
                                             dict(resid=None), dict(w_post=None), dict(gate=None), dict(dy=None),
                                             dict(lddy=63), dict(lddo=63), dict(lddb=63), dict(lddr=63), dict(dy=ODD), dict(dx=ODD),
                                             dict(dw_post=ODD), dict(dgate=A + 2), dict(dw_pre=A + 1)])
def test_backward_refusals(lib, change):
    assert call(lib.wr_block_norm_backward, BACK, **change) == EINVAL


def test_backward_limit_and_workspace(lib):
    from post_bit_weight_amd import _lib
    wide = {k: 16385 for k in ("n", "ldb", "ldr", "ldg", "lddy", "lddo", "lddb", "lddr")}
    assert call(lib.wr_block_norm_backward, BACK, **wide) == EUNSUPPORTED
    size = lambda rows, n, gate: _lib.wr_workspace_bytes(_lib.WR_OP_NORM_BWD, rows, n, gate)  # noqa: E731
    assert size(8192, 2560, 0) >= 2 * 256 * 2560 * 4
    assert size(8192, 2560, 0) == size(8192, 2560, 8192) == size(8192, 2560, 1 << 30)
    assert size(8192, 20000, 0) == 0 and size(8192, 2560, -1) == 0
    for rows in (1, 2, 5, 333, 8192, 100000):   # no tokens' cut needs more than the tokens themselves
        for gate in (0, 1, 2, 37, 4096):
            assert 0 < size(rows, 64, gate) <= 64 * 4 * (3 * rows + 4096) + 4096
