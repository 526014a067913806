"""CPU pins of the block oracle: hand-computed values, invariants, and the gradient against differences."""
import numpy as np
import pytest

import oracle


def test_block_norm_by_hand():
    # rms(3, 4) = sqrt(12.5); with weight sqrt(12.5) the normalised branch is (3, 4) again
    w = np.full(2, np.sqrt(12.5))
    out, y, stats = oracle.block_norm(0.0, branch=[[3.0, 4.0]], resid=[[1.0, 0.0]], w_post=w, gate=[[2.0, 0.5]],
                                      bscale=0.5, rscale=3.0, w_pre=[1.0, 2.0])
    assert np.allclose(out, [[6.0, 1.0]])
    r = np.sqrt((36.0 + 1.0) / 2)
    assert np.allclose(y, [[6.0 / r, 2.0 / r]])
    assert np.allclose(stats, [[1 / np.sqrt(12.5), 1 / r]])


def test_gate_rows_of_a_ragged_last_group():
    g = np.arange(6.0).reshape(3, 2)
    assert np.array_equal(oracle.gate_per_token(g, 2, 5)[:, 0], [0, 0, 2, 2, 4])
    assert np.array_equal(oracle.gate_per_token(g[:1], 0, 4)[:, 1], [1, 1, 1, 1])


@pytest.mark.parametrize("post,gate,resid,pre", [(1, 1, 1, 1), (0, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0),
                                                 (0, 0, 1, 1)])
def test_gradient_against_differences(post, gate, resid, pre):
    rng = np.random.default_rng(post + 2 * gate + 4 * resid + 8 * pre)
    rows, n, eps, per = 5, 7, 1e-3, 2
    inp = dict(branch=rng.normal(size=(rows, n)))
    if resid:
        inp["resid"] = rng.normal(size=(rows, n))
    if post:
        inp["w_post"] = rng.normal(size=n)
    if gate:
        inp["gate"] = rng.normal(size=(3, n))
    if pre:
        inp["w_pre"] = rng.normal(size=n)
    dy = rng.normal(size=(rows, n)) if pre else None
    dres = rng.normal(size=(rows, n))
    fixed = dict(gate_rows=per, bscale=0.7, rscale=1.3)

    def loss(v):
        out, y, _ = oracle.block_norm(eps, **v, **fixed)
        return np.sum(out * dres) + (np.sum(y * dy) if pre else 0.0)

    grads = oracle.block_norm_backward(eps, **inp, **fixed, dy=dy, dres=dres)
    for name, value in inp.items():
        got = grads["d" + name]
        num = np.zeros_like(value)
        for at in np.ndindex(value.shape):
            h = 1e-5
            hi, lo = value.copy(), value.copy()
            hi[at] += h
            lo[at] -= h
            num[at] = (loss({**inp, name: hi}) - loss({**inp, name: lo})) / (2 * h)
        # central differences: h^2 f''' ~ 1e-10 plus cancellation 1e-16 / h ~ 1e-11, times values near 10
        assert np.allclose(got, num, rtol=1e-7, atol=1e-7), name


def test_quant_rows_by_hand_and_special_rows():
    v = np.array([[127.0, -63.5, 0.5, 1.5], [0, 0, 0, 0], [1.0, np.nan, 0, 0], [np.inf, 1, 1, 1]])
    codes, scales = oracle.quant_rows_i8(v)
    assert codes[0].tolist() == [127, -64, 0, 2]  # ties to even
    assert scales[0] == 1.0 and scales[1] == 0.0 and np.isnan(scales[2]) and np.isnan(scales[3])
    assert not codes[1:].any()


def test_quantized_rows_are_within_half_a_step():
    v = np.random.default_rng(3).normal(size=(20, 333))
    codes, scales = oracle.quant_rows_i8(v)
    assert np.all(np.abs(codes * scales[:, None] - v) <= scales[:, None] * (0.5 + 1e-12))
    assert np.all(np.abs(codes).max(axis=1) == 127)


def test_matmul_i8_is_the_product_of_what_the_codes_stand_for():
    rng = np.random.default_rng(4)
    x, w = rng.integers(-128, 128, (3, 9)), rng.integers(-128, 128, (4, 9))
    xs, ws, b = rng.random(3), rng.random(4), rng.normal(size=4)
    z = (x * xs[:, None]) @ (w * ws[:, None]).T + b
    assert np.allclose(oracle.matmul_i8(x, xs, w, ws, b), z)
    ws = ws / 100
    z = (x * xs[:, None]) @ (w * ws[:, None]).T + b
    sw = oracle.matmul_i8(x, xs, w, ws, b, swiglu=True)
    assert np.allclose(sw, z[:, :2] / (1 + np.exp(-z[:, :2])) * z[:, 2:])
    assert np.array_equal(oracle.matmul_i8(x[:, :0], xs, w[:, :0], ws), np.zeros((3, 4)))
