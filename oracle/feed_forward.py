"""What follows a product (bias, activation, gate, residual), its gradients, and rows in groups, in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Pins (``tests/test_oracle_feed_forward.py``): activations against their scalar definitions with ``math``, slopes against
differences of the values, and the grouped quantiser against the plain one on each group's rows.
"""

import math

import numpy as np

from . import block128

ACTIVATIONS = (None, "relu", "silu", "gelu", "gelu_tanh")


def sigmoid(u):
    e = np.exp(-np.abs(u))
    return np.where(u >= 0, 1 / (1 + e), e / (1 + e))


def activation(z, kind):
    """(value, slope) of float64 z."""
    z = np.asarray(z, np.float64)
    if kind is None:
        return z, np.ones_like(z)
    if kind == "relu":
        return np.maximum(z, 0), (z > 0).astype(np.float64)
    if kind == "silu":
        s = sigmoid(z)
        return z * s, s + z * s * sigmoid(-z)
    if kind == "gelu":
        from scipy.special import erfc
        p = 0.5 * erfc(-z * math.sqrt(0.5))
        return z * p, p + z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        a = 2 * math.sqrt(2 / math.pi)
        u, du = a * (z + 0.044715 * z ** 3), a * (1 + 3 * 0.044715 * z * z)
        s = sigmoid(u)
        return z * s, s + z * s * sigmoid(-u) * du
    raise ValueError(kind)


def group_blocks(rows, groups):
    """Blocks of 128 rows that so many groups of so many rows in all take at most."""
    filled = min(rows, groups)  # the worst is one row in each block but the last group's
    return 0 if groups == 0 else (rows + 127 * filled) // 128


def quantize_grouped(x, offsets, fmt=0, rows=True, pow2=False):
    """(q, s, qt, st): block128.quantize with the blocks along the rows starting at every group's first row."""
    T, K = x.shape
    q, s, _, _ = block128.quantize(x, fmt, True, False, False, pow2)
    blocks = group_blocks(T, len(offsets) - 1)
    qt, st = np.zeros((K, 128 * blocks), np.uint8), np.zeros((blocks, K), np.float32)
    at = 0
    for lo, hi in zip(offsets[:-1], offsets[1:]):
        n = -(-(hi - lo) // 128)
        if n:
            _, _, c, t = block128.quantize(x[lo:hi], fmt, False, True, False, pow2)
            qt[:, 128 * at:128 * at + c.shape[1]] = c
            st[at:at + n] = t
        at += n
    return (q, s, qt, st) if rows else (None, None, qt, st)
