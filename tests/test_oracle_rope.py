"""Pins of the rotary oracle."""
import math

import numpy as np
import pytest

from oracle import rope


def test_by_hand():
    w = rope.freqs(4, base=100.0)
    np.testing.assert_allclose(w, [1.0, 0.1])
    x = np.arange(1.0, 6.0).reshape(1, 1, 5)
    for inter, pairs in ((False, ((0, 2), (1, 3))), (True, ((0, 1), (2, 3)))):
        y = rope.rotate(x, [3], w, inter, mscale=2.0)
        for i, (a, b) in enumerate(pairs):
            z = complex(x[0, 0, a], x[0, 0, b]) * complex(math.cos(3 * w[i]), math.sin(3 * w[i])) * 2
            np.testing.assert_allclose([y[0, 0, a], y[0, 0, b]], [z.real, z.imag], rtol=1e-14)
        assert y[0, 0, 4] == 5.0
    assert (rope.rotate(x, [None], w, False) == x).all()


def test_scalings():
    plain = rope.freqs(16)
    np.testing.assert_allclose(rope.freqs(16, scaling="linear", factor=4.0), plain / 4)
    # the scaled base leaves the fastest pair and slows the slowest by exactly the factor
    b = rope.freqs(16, scaling="base", factor=4.0)
    np.testing.assert_allclose([b[0], b[-1]], [plain[0], plain[-1] / 4])
    r = rope.freqs(64, scaling="ramp", factor=8.0, trained=4096)
    p = rope.freqs(64)
    turns = 4096 * p / (2 * math.pi)
    np.testing.assert_allclose(r[turns >= 32], p[turns >= 32])
    np.testing.assert_allclose(r[turns <= 1], p[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and ((r < p) & (r > p / 8))[mid].all()


@pytest.mark.parametrize("inter", [False, True])
def test_scores_depend_on_distance_and_gradient_is_the_way_back(inter):
    rng = np.random.default_rng(1)
    w = rope.freqs(16)
    q, k = rng.standard_normal((2, 1, 1, 24))
    def at(a, b):
        return float((rope.rotate(q, [a], w, inter) * rope.rotate(k, [b], w, inter)).sum())
    assert abs(at(5, 2) - at(1003, 1000)) < 1e-10 and abs(at(5, 2) - at(5, 3)) > 1e-3
    np.testing.assert_allclose(rope.rotate(rope.rotate(q, [9], w, inter), [9], w, inter, sign=-1), q,
                               atol=1e-14)
    # differences: d (g . rotate(q)) / d q
    g, h = rng.standard_normal((1, 1, 24)), 1e-6
    grad = rope.rotate(g, [7], w, inter, mscale=1.3, sign=-1)
    for i in range(24):
        e = np.zeros((1, 1, 24))
        e[..., i] = h
        num = ((rope.rotate(q + e, [7], w, inter, 1.3) - rope.rotate(q - e, [7], w, inter, 1.3)) * g).sum()
        assert abs(num / (2 * h) - grad[0, 0, i]) < 1e-8   # what is not turned is not scaled


def test_positions():
    assert rope.positions(6, [0, 2, 2, 5], [10, 0, 7]) == [10, 11, 7, 8, 9, None]
