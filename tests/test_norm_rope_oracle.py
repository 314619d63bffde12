"""Pins of the norm-and-rotation oracle (CPU): closed forms, invariances and finite differences."""

import numpy as np
import pytest

from oracle.norm_rope import norm_rope64, norm_rope64_backward, rotation

RNG = np.random.default_rng(11)


def angles(T, half):
    a = np.arange(T)[:, None] * 10000.0 ** (-np.arange(half) / max(half, 1))
    return np.cos(a), np.sin(a)


@pytest.mark.parametrize("interleaved", [False, True])
def test_position_zero_is_the_norm_alone(interleaved):
    x, w = RNG.standard_normal((1, 3, 16)), RNG.standard_normal(16)
    y = norm_rope64(x, w, *angles(1, 8), 0.0, interleaved)
    assert np.allclose(y, x * w / np.sqrt((x * x).mean(-1, keepdims=True)), atol=1e-15)


def test_a_quarter_turn_swaps_the_pair():
    x = np.array([[[3.0, 4.0, 5.0, 12.0]]])
    r = np.sqrt((x * x).mean())
    for interleaved, want in ((False, [-5.0, -12.0, 3.0, 4.0]), (True, [-4.0, 3.0, -12.0, 5.0])):
        got = norm_rope64(x, np.ones(4), np.zeros((1, 2)), np.ones((1, 2)), 0.0, interleaved)
        assert np.allclose(got * r, np.array(want), atol=1e-14)


@pytest.mark.parametrize("interleaved", [False, True])
def test_products_of_rotated_rows_depend_on_the_distance_alone(interleaved):
    q, k = RNG.standard_normal((2, 1, 1, 16))
    c, s = angles(50, 8)
    dot = lambda i, j: float(np.sum(norm_rope64(q, np.ones(16), c[i:i + 1], s[i:i + 1], 0, interleaved)  # noqa: E731
                                    * norm_rope64(k, np.ones(16), c[j:j + 1], s[j:j + 1], 0, interleaved)))
    assert np.isclose(dot(7, 3), dot(41, 37), atol=1e-13) and not np.isclose(dot(7, 3), dot(7, 4), atol=1e-6)


def test_rotation_is_orthogonal():
    c, s = angles(5, 4)
    for interleaved in (False, True):
        R = rotation(c[3], s[3], 12, interleaved)
        assert np.allclose(R @ R.T, np.eye(12), atol=1e-15) and np.allclose(R[8:, 8:], np.eye(4))


@pytest.mark.parametrize("interleaved,rotary", [(False, 16), (True, 8), (False, 0)])
def test_gradients_against_differences(interleaved, rotary):
    x, dy, w = RNG.standard_normal((3, 2, 16)), RNG.standard_normal((3, 2, 16)), RNG.standard_normal(16)
    c, s = angles(3, rotary // 2)
    f = lambda x_, w_: float(np.sum(dy * norm_rope64(x_, w_, c, s, 1e-3, interleaved)))  # noqa: E731
    dx, dw = norm_rope64_backward(dy, x, w, c, s, 1e-3, interleaved)
    h = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[i]) < 1e-8
    for i in range(16):
        e = np.zeros(16)
        e[i] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i]) < 1e-8
