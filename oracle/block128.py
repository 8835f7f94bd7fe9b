"""Quantisation with one float32 scale per block of 128, and the product of two such operands.

TEST INFRASTRUCTURE ONLY (see the package docstring).

``quantize``: for a block with largest magnitude a, at least 448 * 2^-100, scale = float32(a / FMAX) and code =
nearest(x FMAX / a), or with powers of two scale = 2^e with the smallest e that has FMAX * 2^e >= a and code =
nearest(x 2^-e), where nearest looks at the exact quotient; the GPU must give the same bits.  ``gemm`` dequantises to
float64 and contracts; it also returns S = sum |a||b|, which the tolerances scale with.

Pins (``tests/test_oracle_block128.py``): the scale rule against exact fractions, codes against a brute-force nearest
search over the decode table, and the product against a scalar loop over blocks.
"""

import numpy as np

from .codecs import decode
from .mx_quantize import encode_rne

FMAX = {0: np.float32(448.0), 1: np.float32(57344.0)}
TINY = np.float32(448.0 * 2.0 ** -100)


def block_scales(amax, fmt, pow2):
    """(scale, multiplier) float32 of float32 block maxima; those that are not finite give a scale that is not."""
    a = np.maximum(np.asarray(amax, np.float32), TINY)     # propagates NaN
    with np.errstate(invalid="ignore", over="ignore"):
        scale, inv = (a / FMAX[fmt]).astype(np.float32), (FMAX[fmt] / a).astype(np.float32)
    if pow2:
        mant, exp = np.frexp(np.where(np.isfinite(a), a, np.float32(1)))
        e = exp - (9 if fmt == 0 else 16) + (mant > np.float32(0.875))
        ok = np.isfinite(a)
        scale = np.where(ok, np.ldexp(np.float32(1), e), scale).astype(np.float32)
        inv = np.where(ok, np.ldexp(np.float32(1), -e), inv).astype(np.float32)
    return scale, inv


def _codes(x, amax, fmt, pow2):
    """uint8 codes of finite float32 x in blocks with largest magnitudes amax (broadcast against x)."""
    a = np.maximum(np.asarray(amax, np.float32), TINY).astype(np.float64)
    if pow2:
        q = x.astype(np.float64) * block_scales(amax, fmt, True)[1].astype(np.float64)
    else:
        q = x.astype(np.float64) * float(FMAX[fmt]) / a  # exact product; boundaries between codes are 2^-30 away or hit
    return encode_rne(q, fmt)


def _pad(x, axis, m):
    n = -x.shape[axis] % m
    widths = [(0, 0)] * x.ndim
    widths[axis] = (0, n)
    return np.pad(x, widths)


def quantize(x, fmt=0, rows=True, cols=False, square=False, pow2=False):
    """(q, s, qt, st) of finite float32 x (M, K), None for what is not asked for; codes uint8."""
    x = np.asarray(x, np.float32)
    M, K = x.shape
    k16, m16 = -(-K // 16) * 16, -(-M // 16) * 16
    full = _pad(_pad(x, 1, 128), 0, 128)
    mb, kb = full.shape[0] // 128, full.shape[1] // 128
    t = full.reshape(mb, 128, kb, 128)
    q = s = qt = st = None
    if square:
        amax = np.abs(t).max(axis=(1, 3))
        scale = block_scales(amax, fmt, pow2)[0]
        codes = _codes(t, amax[:, None, :, None], fmt, pow2).reshape(full.shape)
        if rows:
            q, s = codes[:M, :k16], scale
        if cols:
            qt, st = codes[:m16, :K].T, scale.T
        return q, s, qt, st
    if rows:
        amax = np.abs(t).max(axis=3)                                            # (mb, 128, kb)
        scale = block_scales(amax, fmt, pow2)[0]
        codes = _codes(t, amax[..., None], fmt, pow2).reshape(full.shape)
        q, s = codes[:M, :k16], scale.reshape(mb * 128, kb)[:M].T
    if cols:
        amax = np.abs(t).max(axis=1)                                            # (mb, kb, 128)
        scale = block_scales(amax, fmt, pow2)[0]
        codes = _codes(t, amax[:, None], fmt, pow2).reshape(full.shape)
        qt, st = codes[:m16, :K].T, scale.reshape(mb, kb * 128)[:, :K]
    return q, s, qt, st


def dequantize(codes, scales, fmt, square):
    """float64 (rows, K) of codes with scales (ceil(K/128), rows), or (ceil(rows/128), ceil(K/128)) when square."""
    n, K = codes.shape
    s = np.asarray(scales, np.float64)
    s = np.repeat(s, 128, axis=0)[:n] if square else s.T
    return decode(codes, fmt) * np.repeat(s, 128, axis=1)[:, :K]


def gemm(a, sa, b, sb, a_fmt, b_fmt, b_block):
    """(C, S) float64: the product and sum |a||b|."""
    x, w = dequantize(a, sa, a_fmt, False), dequantize(b, sb, b_fmt, b_block == 128)
    return x @ w.T, np.abs(x) @ np.abs(w).T
