"""Pins of oracle/attention_oracle.py against brute force in Python numbers."""
import math

import numpy as np
import pytest

import oracle.attention_oracle as A


def test_int8_linear_by_hand():
    x = np.array([[127, -128, 3], [0, 1, 2]], np.int8)
    w = np.array([[1, 2, 3], [-128, -128, 127]], np.int8)
    acc, y, _ = A.int8_linear(x, np.float32([0.5, 2.0]), w, np.float32([1.0, 0.25]), np.float32([10.0, -1.0]))
    assert acc.tolist() == [[127 - 256 + 9, -127 * 128 + 128 * 128 + 381], [8, -128 + 254]]
    assert y.tolist() == [[-60.0 + 10.0, 509 * 0.125 - 1.0], [16.0 + 10.0, 126 * 0.5 - 1.0]]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_is_a_rotation_of_normed_heads(interleaved):
    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((3, 2, 8)), rng.standard_normal(8)
    ang = rng.uniform(0, 6, (3, 3))
    y, _ = A.heads_norm_rope(x, w, 1e-6, np.cos(ang), np.sin(ang), interleaved)
    for t in range(3):
        for h in range(2):
            r = math.sqrt(sum(v * v for v in x[t, h]) / 8 + 1e-6)
            n = [float(x[t, h, i] / r * w[i]) for i in range(8)]
            for i in range(3):
                lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + 3)
                z = complex(n[lo], n[hi]) * complex(math.cos(ang[t, i]), math.sin(ang[t, i]))
                assert abs(z - complex(y[t, h, lo], y[t, h, hi])) < 1e-12
            assert np.allclose(y[t, h, 6:], n[6:], rtol=0, atol=1e-12)


@pytest.mark.parametrize("n,kv,window,sinks", [(1, 1, 0, 0), (3, 7, 0, 0), (5, 9, 3, 2), (4, 4, 1, 0), (6, 2, 0, 0), (2, 9, 4, 100), (3, 0, 2, 1)])
def test_mask_against_the_definition(n, kv, window, sinks):
    m = A.mask(n, kv, window, sinks)
    for i in range(n):
        for j in range(kv):
            assert m[i, j] == A.sees(kv - n + i, j, window, sinks)


def test_attend_against_loops_and_empty_rows():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 4)), rng.standard_normal((5, 4)), rng.standard_normal((5, 4))
    seen = np.array([[1, 0, 1, 0, 0], [0] * 5, [1] * 5], bool)
    out, mag, size = A.attend(q, k, v, seen, 0.7)
    for i in range(3):
        w = [math.exp(0.7 * sum(q[i, d] * k[j, d] for d in range(4))) if seen[i, j] else 0.0 for j in range(5)]
        for d in range(4):
            want = sum(w[j] * v[j, d] for j in range(5)) / sum(w) if sum(w) else 0.0
            assert abs(out[i, d] - want) < 1e-12
    assert (out[1] == 0).all() and (mag[1] == 0).all() and size[1, 0] == 0


def test_gather_follows_the_table():
    cache = np.arange(4 * 1 * 2 * 1, dtype=float).reshape(4, 1, 2, 1)
    k, good = A.gather(cache, [3, -1, 1], 7)
    assert k[0, :, 0].tolist() == [6, 7, 0, 0, 2, 3, 0] and good.tolist() == [True, True, False, False, True, True, False]
