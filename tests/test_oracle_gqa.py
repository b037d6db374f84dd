"""Pins of the grouped-query attention oracle: closed forms, brute force in
plain Python, invariants."""

import math

import numpy as np
import pytest

from oracle import gqa


def test_rotation_known_angles_norms_and_relative_positions():
    x = np.zeros((2, 1, 8))
    x[:, 0, 4], x[:, 0, 0] = 1.0, 5.0
    y = gqa.rotate(x, [0, 3], 4, 100.0)           # pairs (4,5) at theta^0, (6,7) at theta^(-1/2)
    np.testing.assert_allclose(y[0], x[0])
    np.testing.assert_allclose(y[1, 0], [5, 0, 0, 0, math.cos(3), math.sin(3), 0, 0], atol=1e-15)
    x[:, 0, 6] = 1.0
    np.testing.assert_allclose(gqa.rotate(x, [0, 3], 4, 100.0)[1, 0, 6:], [math.cos(0.3), math.sin(0.3)], atol=1e-15)
    rng = np.random.default_rng(0)
    a, b = rng.standard_normal((2, 1, 1, 64))
    dots = [float((gqa.rotate(a, [p + 7], 64, 1e4) * gqa.rotate(b, [p], 64, 1e4)).sum()) for p in (0, 1000, 123456)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-9)


def test_row_scale():
    np.testing.assert_array_equal(gqa.row_scale([[0.0, 0.0], [-896.0, 1.0]]), [1.0, 2.0])


@pytest.mark.parametrize("window,sink", [(0, None), (3, None), (2, [0.5, -1.0, 2.0, 0.0])])
def test_attend_brute_force(window, sink):
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((5, 4, 8)), rng.standard_normal((6, 2, 8)), rng.standard_normal((6, 2, 8))
    t = [-1, 0, 2, 4, 5]
    live = [True, False, True, True, True, True]
    out, mag, _ = gqa.attend(q, k, v, t, 0.3, window, sink, live)
    for i in range(5):
        for h in range(4):
            keys = [j for j in range(6) if j <= t[i] and live[j] and (not window or j > t[i] - window)]
            e = {j: math.exp(0.3 * sum(q[i, h, c] * k[j, h // 2, c] for c in range(8))) for j in keys}
            den = sum(e.values()) + (math.exp(sink[h]) if sink else 0)
            want = [sum(e[j] * v[j, h // 2, c] for j in keys) / den if keys else 0.0 for c in range(8)]
            np.testing.assert_allclose(out[i, h], want, atol=1e-12)
    assert (mag >= np.abs(out) - 1e-12).all()


def test_masked_keys_take_no_part_whatever_they_hold():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((3, 2, 8)), rng.standard_normal((5, 1, 8)), rng.standard_normal((5, 1, 8))
    want, _, _ = gqa.attend(q, k[:4], v[:4], [1, 2, 3], 1.0)
    k[4], v[4] = np.nan, np.inf
    got, _, _ = gqa.attend(q, k, v, [1, 2, 3], 1.0)
    np.testing.assert_array_equal(got, want)
    v[3, 0, 5] = np.nan                            # seen by the last query alone
    got, _, _ = gqa.attend(q, k, v, [1, 2, 3], 1.0)
    np.testing.assert_array_equal(got[:2], want[:2])
    assert np.isnan(got[2, :, 5]).all() and np.isfinite(np.delete(got[2], 5, -1)).all()
