"""Pins of the attention oracle: hand-worked values and invariances that
do not use its own code."""

import cmath
import math

import numpy as np
import pytest

from oracle import attention as A


def test_norm_hand_case():
    y = A.norm(np.array([[3.0, 4.0]]), np.array([2.0, 0.5]), 0.0)
    r = math.sqrt(12.5)                       # mean of 9 and 16
    assert np.allclose(y, [[6.0 / r, 2.0 / r]], rtol=1e-15)
    assert np.array_equal(A.norm(np.array([[3.0, 4.0]]), None, 1.0), [[3.0, 4.0]])
    assert np.array_equal(A.norm(np.zeros((1, 4)), np.ones(4), 1e-6), np.zeros((1, 4)))


@pytest.mark.parametrize("neighbours", [False, True])
def test_rotation_is_a_complex_product(neighbours):
    rng = np.random.default_rng(3)
    D, rot, T = 16, 12, 5
    x = rng.standard_normal((T, 2, D))
    pos, freq = np.array([0, 1, -7, 30, 1000]), rng.random(rot // 2)
    y = A.rotate(x, pos, freq, neighbours)
    for t in range(T):
        for h in range(2):
            for p in range(rot // 2):
                i, j = (2 * p, 2 * p + 1) if neighbours else (p, p + rot // 2)
                z = complex(x[t, h, i], x[t, h, j]) * cmath.exp(1j * float(pos[t]) * float(freq[p]))
                assert abs(z - complex(y[t, h, i], y[t, h, j])) < 1e-12
    assert np.array_equal(y[..., rot:], x[..., rot:])
    assert np.allclose(y[0], x[0], atol=0)


def test_rotation_keeps_relative_positions():
    rng = np.random.default_rng(4)
    q, k, freq = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8)), rng.random(4)
    dots = []
    for shift in (0, 11):
        a = A.rotate(q, np.array([9 + shift]), freq, False)
        b = A.rotate(k, np.array([2 + shift]), freq, False)
        dots.append(float((a * b).sum()))
    assert abs(dots[0] - dots[1]) < 1e-12


def test_attend_hand_case():
    # scores log 1, log 3 with scale 1: weights 1/4 and 3/4
    q, k = np.array([[1.0, 0.0]]), np.array([[0.0, 5.0], [math.log(3.0), -1.0], [9.0, 9.0]])
    v = np.array([[8.0, -4.0], [0.0, 4.0], [np.nan, np.inf]])
    out, lse, wabs, sabs = A.attend(q, k, v, np.array([[True, True, False]]), 1.0)
    assert np.allclose(out, [[2.0, 2.0]], rtol=1e-15) and np.allclose(wabs, [[2.0, 4.0]], rtol=1e-15)
    assert abs(lse[0] - math.log(4.0)) < 1e-15 and abs(sabs[0] - math.log(3.0)) < 1e-15
    out, lse, _, _ = A.attend(q, k, v, np.zeros((1, 3), bool), 1.0)
    assert not out.any() and lse[0] == -np.inf


def test_attend_invariances():
    rng = np.random.default_rng(5)
    q, k, v = rng.standard_normal((4, 8)), rng.standard_normal((9, 8)), rng.standard_normal((9, 8))
    seen = rng.random((4, 9)) < 0.6
    seen[:, 0] = True
    out, lse, _, _ = A.attend(q, k, v, seen, 0.3)
    order = rng.permutation(9)
    o2, l2, _, _ = A.attend(q, k[order], v[order], seen[:, order], 0.3)
    assert np.allclose(out, o2, atol=1e-14) and np.allclose(lse, l2, atol=1e-14)
    o3, l3, _, _ = A.attend(q, k, v + 2.5, seen, 0.3)                      # weights sum to one
    assert np.allclose(o3, out + 2.5, atol=1e-14) and np.array_equal(l3, lse)
    shift = np.full(8, 0.7)                                              # the same score added to every key
    o4, l4, _, _ = A.attend(q, k + shift, v, seen, 0.3)
    assert np.allclose(o4, out, atol=1e-13) and np.allclose(l4, lse + 0.3 * (q @ shift), atol=1e-13)
