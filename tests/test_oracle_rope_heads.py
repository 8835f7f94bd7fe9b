"""Pins of the rotary and norm oracle: lengths, the transpose, layouts as permutations, gradients as differences."""

import numpy as np
import pytest

from oracle import rope_heads as R

LAYOUTS = ["half", "interleaved", "interleaved_to_half"]


def tables(T, half, seed=0):
    a = np.random.default_rng(seed).uniform(-9, 9, (T, half))
    return np.cos(a), np.sin(a)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_lengths_and_transpose(layout):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((4, 3, 24))
    cos, sin = tables(4, 6)
    y, _ = R.rotate(x, cos, sin, layout, offset=8)
    np.testing.assert_array_equal(y[..., :8], x[..., :8])
    np.testing.assert_array_equal(y[..., 20:], x[..., 20:])
    xi = x[..., 8:20]
    yi = y[..., 8:20]
    pin = (xi[..., :6], xi[..., 6:]) if layout == "half" else (xi[..., 0::2], xi[..., 1::2])
    pout = (yi[..., 0::2], yi[..., 1::2]) if layout == "interleaved" else (yi[..., :6], yi[..., 6:])
    np.testing.assert_allclose(np.hypot(*pout), np.hypot(*pin), rtol=1e-14)
    # the angle between pair and image is the table's
    np.testing.assert_allclose(pin[0] * pout[0] + pin[1] * pout[1], np.hypot(*pin) ** 2 * cos[:, None], atol=1e-13)
    back, _ = R.rotate(y, cos, sin, layout, offset=8, transpose=True)
    np.testing.assert_allclose(back, x, atol=1e-14)
    # <R x, g> = <x, R^T g>, with factors on the tables too
    g = rng.standard_normal(x.shape)
    y2, _ = R.rotate(x, 1.3 * cos, 1.3 * sin, layout, offset=8)
    gt, _ = R.rotate(g, 1.3 * cos, 1.3 * sin, layout, offset=8, transpose=True)
    np.testing.assert_allclose((y2 * g).sum(), (x * gt).sum(), rtol=1e-12)


def test_interleaved_is_half_between_permutations():
    x = np.random.default_rng(2).standard_normal((3, 2, 16))
    cos, sin = tables(3, 8)
    to_half = np.concatenate((np.arange(0, 16, 2), np.arange(1, 16, 2)))
    want, _ = R.rotate(x[..., to_half], cos, sin, "half")
    got, _ = R.rotate(x, cos, sin, "interleaved")
    np.testing.assert_array_equal(got[..., to_half], want)
    np.testing.assert_array_equal(R.rotate(x, cos, sin, "interleaved_to_half")[0], want)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_gradients_are_differences(layout):
    rng = np.random.default_rng(3)
    x, w, g = rng.standard_normal((2, 2, 12)), rng.standard_normal(12), rng.standard_normal((2, 2, 12))
    cos, sin = tables(2, 4)
    loss = lambda x, w: (R.norm_rotate(x, w, cos, sin, layout, 4)[0] * g).sum()  # noqa: E731
    dx, dw, _, _ = R.norm_rotate_backward(g, x, w, cos, sin, layout, 4)
    h = 1e-6
    for at in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[at] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[at]) < 1e-7
    for i in range(12):
        e = np.zeros(12)
        e[i] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[i]) < 1e-7
