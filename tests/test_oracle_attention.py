"""Pins for the oracle's attention operators: closed forms and explicit loops."""
import math

import numpy as np

import oracle


def test_rotary_turns_by_the_angle_and_back():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(3, 2 * 6))
    pos = np.array([[1, 2, 3], [5, 0, 7]])
    freqs, axis_of = np.array([0.5, 2.0]), np.array([0, 1])
    y = oracle.rotary(x, pos, freqs, 6, axis_of)
    for r in range(3):
        for h in range(2):
            for i in range(2):
                a = pos[axis_of[i], r] * freqs[i]
                u, v = x[r, 6 * h + i], x[r, 6 * h + 2 + i]
                assert np.isclose(y[r, 6 * h + i], u * math.cos(a) - v * math.sin(a), atol=1e-14)
                assert np.isclose(y[r, 6 * h + 2 + i], u * math.sin(a) + v * math.cos(a), atol=1e-14)
            assert (y[r, 6 * h + 4:6 * h + 6] == x[r, 6 * h + 4:6 * h + 6]).all()
    assert np.allclose(oracle.rotary(y, pos, freqs, 6, axis_of, inverse=True), x, atol=1e-14)
    z = oracle.rotary(x, pos[0], freqs, 6, interleaved=True)
    assert np.isclose(z[0, 0], x[0, 0] * math.cos(0.5) - x[0, 1] * math.sin(0.5), atol=1e-14)


def test_cache_codes_of_chosen_values():
    x = np.zeros((1, 32), np.float32)
    x[0, :16] = np.arange(16)
    codes, scale, off = oracle.kv_codes(x, 32)
    assert scale[0, 0] == 1 and off[0, 0] == 0
    assert codes[0].tolist() == list(range(16)) + [0] * 16
    x = np.full((1, 32), -3.0, np.float32)  # all alike: the offset alone
    codes, scale, off = oracle.kv_codes(x, 32)
    assert scale[0, 0] == 0 and off[0, 0] == -3 and not codes.any()
    x[0, 7] = np.inf
    codes, scale, off = oracle.kv_codes(x, 32)
    assert np.isnan(scale[0, 0]) and np.isnan(off[0, 0]) and not codes.any()
    x[0, :2] = [-1e30, 3e38]
    x[0, 7] = 0
    codes, scale, off = oracle.kv_codes(x, 32)
    top = float(off[0, 0]) + 15 * float(scale[0, 0])
    assert codes[0, 0] == 0 and codes[0, 1] == 15 and 65000 < top < 65504


def test_cache_values_are_within_half_a_step():
    x = np.random.default_rng(2).normal(size=(50, 64)).astype(np.float32) + 3
    codes, scale, off = oracle.kv_codes(x, 32)
    err = np.abs(oracle.kv_values(codes, scale, off, 32) - x).reshape(50, 2, 32)
    # half a step, the rounding of offset (2^-11 of at most 8) and of the scale (2^-11, 15 times)
    assert (err <= 0.5 * scale.astype(float)[..., None] * (1 + 30 * 2.0 ** -11) + 8 * 2.0 ** -11).all()


def test_attention_by_loops():
    rng = np.random.default_rng(3)
    q, k, v = rng.normal(size=(4, 8)), rng.normal(size=(9, 8)), rng.normal(size=(9, 8))
    ok = oracle.sees(5, 4, 9, window=3)
    assert ok.sum(1).tolist() == [3, 3, 3, 3] and ok[0, 3:6].all()
    assert oracle.sees(0, 2, 9, causal=False, window=2).sum(1).tolist() == [2, 3]
    ok[2] = False
    out, _ = oracle.attend(q, k, v, ok, 0.3)
    for r in range(4):
        w = [math.exp(0.3 * sum(q[r, d] * k[t, d] for d in range(8))) if ok[r, t] else 0 for t in range(9)]
        for d in range(8):
            assert np.isclose(out[r, d], sum(w[t] * v[t, d] for t in range(9)) / sum(w) if sum(w) else 0, atol=1e-12)


def test_adapters_by_loops():
    rng = np.random.default_rng(4)
    x, base = rng.normal(size=(5, 3)), rng.normal(size=(5, 2))
    A, B, scales = rng.normal(size=(2, 4, 3)), rng.normal(size=(2, 2, 4)), np.array([0.5, 2.0])
    y = oracle.adapters(x, base, A, B, scales, [0, 2, 3, 5], [1, -1, 0], ranks=[3, 9])
    for r in range(5):
        a = [1, 1, -1, 0, 0][r]
        for o in range(2):
            want = base[r, o]
            if a >= 0:
                want += scales[a] * sum(B[a, o, j] * sum(A[a, j, c] * x[r, c] for c in range(3)) for j in range([3, 4][a]))
            assert np.isclose(y[r, o], want, atol=1e-12)
