"""Pins of the feed-forward oracle: activations against their scalar definitions, slopes against differences, the grouped
quantiser against the plain one, and the bound on the groups' blocks against all ways to share out rows."""

import itertools
import math

import numpy as np
import pytest

from oracle import block128 as B
from oracle import feed_forward as F


def scalar(z, kind):
    if kind is None:
        return z
    if kind == "relu":
        return max(z, 0.0)
    if kind == "silu":
        return z / (1 + math.exp(-z))
    if kind == "gelu":
        return 0.5 * z * (1 + math.erf(z / math.sqrt(2)))
    return 0.5 * z * (1 + math.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


@pytest.mark.parametrize("kind", F.ACTIVATIONS)
def test_values(kind):
    """The scalar forms cancel in the lower tail, by 2^-52 of z there."""
    z = np.linspace(-20, 20, 4001)
    got = F.activation(z, kind)[0]
    want = np.array([scalar(float(v), kind) for v in z])
    assert np.all(np.abs(got - want) <= 4 * 2.0 ** -52 * np.maximum(np.abs(z), 1))


@pytest.mark.parametrize("kind", F.ACTIVATIONS)
def test_slopes_are_differences(kind):
    z, h = np.linspace(-9.9995, 9.9995, 2000), 1e-4
    got = F.activation(z, kind)[1]
    want = (F.activation(z + h, kind)[0] - F.activation(z - h, kind)[0]) / (2 * h)
    # a third derivative below 2, and the values' rounding over the step
    assert np.all(np.abs(got - want) <= 2 * h * h / 6 + 20 * 2.0 ** -52 / h)


def test_far_values_are_finite():
    for kind in F.ACTIVATIONS:
        for v in F.activation(np.array([-1e30, -1e4, 1e4, 1e30]), kind):
            assert np.all(np.isfinite(v))
    assert F.activation(np.array([-30.0]), "gelu")[0][0] < 0  # the tail is not lost


def test_blocks_of_groups_are_the_most_there_can_be():
    for groups in range(5):
        for rows in (0, 1, 2, 3, 5, 127, 128, 129, 130, 257, 384, 400):
            cuts = itertools.combinations_with_replacement(sorted({0, 1, 2, 3, rows // 2, 127, 128, 129, 130, 256, 257, rows - 1, rows}
                                                                  & set(range(rows + 1))), max(groups - 1, 0))
            most = 0
            for c in cuts:
                if groups == 0:
                    break
                edges = (0, *c, rows)
                most = max(most, sum(-(-(b - a) // 128) for a, b in zip(edges, edges[1:])))
            assert most <= F.group_blocks(rows, groups)
            if groups and rows >= groups:  # one row in every group but the last
                assert F.group_blocks(rows, groups) == groups - 1 + -(-(rows - groups + 1) // 128)


def test_grouped_quantiser():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((300, 40)).astype(np.float32)
    offsets = [3, 3, 133, 140, 290]
    q, s, qt, st = F.quantize_grouped(x, offsets)
    want = B.quantize(x)
    assert np.array_equal(q, want[0]) and np.array_equal(s, want[1])
    at = 0
    for lo, hi in zip(offsets, offsets[1:]):
        for first in range(lo, hi, 128):
            part = x[first:min(first + 128, hi)]
            block = qt[:, 128 * at:128 * at + 128]
            scale = np.maximum(np.abs(part).max(axis=0), B.TINY) / B.FMAX[0]
            assert np.array_equal(st[at], scale.astype(np.float32))
            assert not block[:, len(part):].any()
            from oracle.codecs import decode
            back = decode(block[:, :len(part)], 0).T * st[at]
            assert np.all(np.abs(back - part) <= np.abs(part) / 16 + st[at] * 2.0 ** -10)
            at += 1
    assert not qt[:, 128 * at:].any() and not st[at:].any() and len(st) == F.group_blocks(300, 4)
