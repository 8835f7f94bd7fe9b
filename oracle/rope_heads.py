"""Rotary positions and the per-head norm of queries and keys, forward and backward, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

``rotate`` turns the pairs (a_i, b_i) of the rotary features [offset, offset + rot) of x (T, H, D):
a' = a cos - b sin, b' = b cos + a sin, with cos, sin (T, rot / 2) the token's table rows; ``transpose`` is its
transposed map.  ``norm_rotate`` is rotate(x / sqrt(mean(x^2) + eps) * w), ``norm_rotate_backward`` its gradients.
Each also returns the sum of the magnitudes of the terms of every output, which the tolerances scale with.

Pins (``tests/test_oracle_rope_heads.py``): a rotation keeps the length of every pair; the transpose undoes it; the
interleaved form is the half form between permutations; gradients equal central differences of the forward.
"""

import numpy as np


def _split(part, halves):
    h = part.shape[-1] // 2
    return (part[..., :h], part[..., h:]) if halves else (part[..., 0::2], part[..., 1::2])


def _join(a, b, halves):
    return np.concatenate((a, b), -1) if halves else np.stack((a, b), -1).reshape(a.shape[:-1] + (-1,))


def rotate(x, cos, sin, layout, offset=0, transpose=False):
    """(y, magnitudes) of x (T, H, D) float64."""
    x = np.asarray(x, np.float64)
    rot = 2 * cos.shape[-1]
    c, s = np.asarray(cos, np.float64)[:, None], np.asarray(sin, np.float64)[:, None]
    if transpose:
        s = -s
    halves_in, halves_out = layout == "half", layout != "interleaved"
    if transpose:
        halves_in, halves_out = halves_out, halves_in
    y, mag = x.copy(), np.abs(x)
    a, b = _split(x[..., offset:offset + rot], halves_in)
    y[..., offset:offset + rot] = _join(a * c - b * s, b * c + a * s, halves_out)
    mag[..., offset:offset + rot] = _join(np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s), halves_out)
    return y, mag


def norm_rotate(x, w, cos, sin, layout, offset=0, eps=1e-6):
    x = np.asarray(x, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return rotate(x * r * np.asarray(w, np.float64), cos, sin, layout, offset)


def norm_rotate_backward(g, x, w, cos, sin, layout, offset=0, eps=1e-6):
    """(dx, dw, magnitudes of dx, magnitudes of dw)."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    u, umag = rotate(g, cos, sin, layout, offset, transpose=True)
    dn = u * w
    dx = r * (dn - n * (dn * n).mean(-1, keepdims=True))
    mag = r * (umag * np.abs(w) + np.abs(n) * (umag * np.abs(w * n)).mean(-1, keepdims=True))
    return dx, (u * n).sum((0, 1)), mag, (umag * np.abs(n)).sum((0, 1))
