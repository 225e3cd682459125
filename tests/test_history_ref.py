"""The 64-bit event-history formulas themselves: gradients against
differences, the rotation and the attention against their properties."""
import numpy as np
import pytest

from tests import _history_ref as R

RNG = np.random.default_rng


def rope(length, rot):
    a = np.arange(length)[:, None] * 100.0 ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(a), np.sin(a)], 1)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(8, 8), (10, 4), (2, 2)])
def test_gradient_is_the_limit_of_differences(d, rot, interleaved):
    g = RNG(d + rot)
    x, w, dy = g.standard_normal((3, 2, d)), g.standard_normal(d), g.standard_normal((3, 2, d))
    table, at = rope(5, rot), np.array([4, 0, 2])
    f = lambda x, w: (R.norm_rope(x, w, 0.1, table, at, interleaved)[0] * dy).sum()
    dx, _, dw, _ = R.norm_rope_bwd(dy, x, w, 0.1, table, at, interleaved)
    h = 1e-6  # differences of second order: off by h^2 of the third derivative and 2^-53 / h of the value
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[i]) < 1e-7
    for i in range(d):
        e = np.zeros(d)
        e[i] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i]) < 1e-7


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_sees_only_distances(interleaved):
    g = RNG(1)
    q, k = g.standard_normal((1, 1, 8)), g.standard_normal((1, 1, 8))
    table = rope(64, 8)
    dots = []
    for shift in (0, 7, 40):
        a, _ = R.norm_rope(q, None, 0, table, np.array([5 + shift]), interleaved)
        b, _ = R.norm_rope(k, None, 0, table, np.array([2 + shift]), interleaved)
        np.testing.assert_allclose((a * a).sum(), (q * q).sum(), rtol=1e-13)
        dots.append((a * b).sum())
    np.testing.assert_allclose(dots, dots[0], rtol=1e-11)


def test_attention_by_hand():
    # two stored tokens of equal keys weigh the same; the window leaves one of them
    kc, vc = np.ones((2, 2, 1, 2)), np.zeros((2, 2, 1, 2))
    vc[1, 0, 0], vc[1, 1, 0] = (1, 3), (5, 7)
    table, q = np.array([[1]]), np.full((1, 2, 2), 0.5)
    out, lse, *_ = R.attention(q, [1], [2], table, kc, vc, 1.0, True, 0)
    np.testing.assert_allclose(out, [[[3, 5], [3, 5]]])
    np.testing.assert_allclose(lse, 1 + np.log(2))
    out, *_ = R.attention(q, [1], [2], table, kc, vc, 1.0, True, 1)
    np.testing.assert_allclose(out, [[[5, 7], [5, 7]]])
    out, lse, *_ = R.attention(q, [1], [0], table, kc, vc, 1.0, False, 0)
    assert not out.any() and np.isneginf(lse).all()
