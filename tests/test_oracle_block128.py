"""Pins of the block-128 oracle: the scale rule against exact fractions, codes against a brute-force nearest search,
the product against a scalar loop over blocks."""

from fractions import Fraction

import numpy as np
import pytest

import oracle
from oracle import block128 as B
from oracle.codecs import decode


def table(fmt):
    v = decode(np.arange(256, dtype=np.uint8), fmt)
    return v[np.isfinite(v)]


@pytest.mark.parametrize("fmt,fmax", [(0, 448), (1, 57344)])
def test_power_of_two_scale_is_the_smallest_that_fits(fmt, fmax):
    rng = np.random.default_rng(fmt)
    a = np.concatenate([np.exp2(rng.uniform(-80, 80, 500)).astype(np.float32),
                        np.float32(fmax) * np.exp2(np.arange(-60, 60, 7)).astype(np.float32),
                        np.nextafter(np.float32(fmax) * np.exp2(np.arange(-60, 60, 7)).astype(np.float32), np.float32(np.inf))])
    s, inv = B.block_scales(a, fmt, True)
    for x, sc, iv in zip(a, s, inv):
        x, sc = Fraction(float(x)), Fraction(float(sc))
        assert fmax * sc >= x and fmax * sc / 2 < x and sc * Fraction(float(iv)) == 1


@pytest.mark.parametrize("fmt", [0, 1])
def test_quotient_scale_is_nearest(fmt):
    a = np.exp2(np.random.default_rng(3).uniform(-60, 60, 300)).astype(np.float32)
    s, inv = B.block_scales(a, fmt, False)
    fm = Fraction(float(B.FMAX[fmt]))
    for x, sc, iv in zip(a, s, inv):
        x = Fraction(float(x))
        for exact, got in ((x / fm, sc), (fm / x, iv)):
            err = abs(Fraction(float(got)) - exact)
            assert err <= Fraction(float(np.spacing(got))) / 2
    zero, _ = B.block_scales(np.zeros(1, np.float32), fmt, False)
    assert zero[0] == B.TINY / B.FMAX[fmt]


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("square", [False, True])
def test_codes_are_nearest_and_blocks_are_where_they_should_be(fmt, square):
    rng = np.random.default_rng(7)
    x = (rng.standard_normal((131, 150)) * np.exp2(rng.integers(-6, 6, (131, 150)))).astype(np.float32)
    q, s, qt, st = B.quantize(x, fmt, True, True, square)
    assert q.shape == (131, 160) and qt.shape == (150, 144)
    assert not q[:, 150:].any() and not qt[:, 131:].any()
    vals = table(fmt)
    for _ in range(300):
        m, k = rng.integers(131), rng.integers(150)
        mb, kb = m // 128, k // 128
        rows, cols = slice(128 * mb, 128 * mb + 128), slice(128 * kb, 128 * kb + 128)
        if square:
            a1 = a2 = np.abs(x[rows, cols]).max()
            assert s[mb, kb] == st[kb, mb] == a1 / B.FMAX[fmt]
        else:
            a1, a2 = np.abs(x[m, cols]).max(), np.abs(x[rows, k]).max()
            assert s[kb, m] == a1 / B.FMAX[fmt] and st[mb, k] == a2 / B.FMAX[fmt]
        for code, a in ((q[m, k], a1), (qt[k, m], a2)):
            v = float(np.float32(float(x[m, k]) * float(B.FMAX[fmt]) / float(a)))
            assert abs(decode(np.array([code]), fmt)[0] - v) == np.abs(vals - v).min()


@pytest.mark.parametrize("b_block", [1, 128])
def test_product_against_a_loop_over_blocks(b_block):
    rng = np.random.default_rng(11)
    a, sa, _, _ = B.quantize(rng.standard_normal((5, 272)).astype(np.float32), 1)
    b, sb, _, _ = B.quantize(rng.standard_normal((130, 272)).astype(np.float32), 0, square=b_block == 128)
    c, big = oracle.block128.gemm(a, sa, b, sb, 1, 0, b_block)
    da, db = decode(a, 1), decode(b, 0)
    for m, n in ((0, 0), (4, 129), (2, 127), (3, 128)):
        want = mag = 0.0
        for j in range(3):
            w = float(sa[j, m]) * float(sb[j, n] if b_block == 1 else sb[n // 128, j])
            at = slice(128 * j, 128 * j + 128)
            want += w * sum(x * y for x, y in zip(da[m, at], db[n, at]))
            mag += w * sum(abs(x * y) for x, y in zip(da[m, at], db[n, at]))
        assert abs(c[m, n] - want) <= 1e-12 * mag and abs(big[m, n] - mag) <= 1e-12 * mag


def near_boundaries(fmt, rows, seed, block=1):
    """(rows, 128) float32: in each row one largest magnitude a, the same in `block` rows, and 127 values that float32 has around boundary * a / FMAX,
    boundaries being the midpoints of neighbouring codes."""
    rng = np.random.default_rng(seed)
    vals = np.unique(table(fmt)[table(fmt) >= 0])
    mid = (vals[1:] + vals[:-1]) / 2
    a = np.repeat(rng.uniform(1, 2, (rows // block, 1)).astype(np.float32), block, 0)
    x = (rng.choice(mid, (rows, 128)) * a / B.FMAX[fmt]).astype(np.float32)
    x = (x.view(np.int32) + rng.integers(-1, 2, x.shape, dtype=np.int32)).view(np.float32)
    x *= rng.choice(np.float32([-1, 1]), x.shape)
    x[:, 5] = a[:, 0]
    return x


@pytest.mark.parametrize("fmt", [0, 1])
def test_codes_next_to_boundaries(fmt):
    x = near_boundaries(fmt, 6, 4)
    q = decode(B.quantize(x, fmt)[0], fmt)
    vals = [Fraction(float(v)) for v in np.unique(table(fmt))]
    for row, codes in zip(x, q):
        a = Fraction(float(np.abs(row).max()))
        for v, c in zip(row, codes):
            e = Fraction(float(v)) * Fraction(float(B.FMAX[fmt])) / a
            best = min(abs(t - e) for t in vals)
            assert abs(Fraction(float(c)) - e) == best
