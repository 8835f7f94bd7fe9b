"""What follows a product, to the last bits: with one code in each row of A a product is a single term, which the matrix cores
give exactly, so nothing hides an error of bias, activation, gate, residual or of a rounding.

Bounds: the two scales' product and its product with the term round once each, by h = 2^-24 at most: p is off by 2.01 h of it.  A bias adds h |z|.  The rest is as in test_gpu_feed_forward.py: the activation's slope
is at most 1.13 and its own arithmetic off by A of its value, gate and residual round once each, and so does the result.
"""

import pytest
import torch

import feed_forward_paths as P
from test_gpu_feed_forward import A, DT, GROUPS, SIZES, TINY, U, act64, close, lib, offsets_of, padded, rand, wide  # noqa: F401

pytestmark = pytest.mark.gpu
H = 2.0 ** -24
F8 = torch.float8_e4m3fn


def codes(shape, seed):
    """e4m3 codes of all magnitudes but NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    magnitude = torch.randint(1, 127, shape, generator=g, device="cuda")
    sign = torch.randint(0, 2, shape, generator=g, device="cuda")
    return (magnitude + 128 * sign).to(torch.uint8)


def operands(m, n, k, seed, groups=None):
    """A with one code in a row, B with all; scales of no particular value.  Their products are of the order of one."""
    a = torch.zeros(m, k, dtype=torch.uint8, device="cuda")
    at = torch.arange(m, device="cuda") * 37 % k
    a[torch.arange(m, device="cuda"), at] = codes((m,), seed)
    lead = () if groups is None else (groups,)
    b = codes((*lead, n, k), seed + 1)
    sa = (torch.rand(-(-k // 128), m, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)) + 0.5) / 64
    sb = (torch.rand(*lead, -(-n // 128), -(-k // 128), device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed + 1)) + 0.5) / 64
    return a.view(F8), sa, b.view(F8), sb


def product(a, sa, b, sb):
    return wide(a, sa, 1) @ wide(b, sb, 128).t().contiguous()


def bounds(p, dtype, bias, kind, gate, residual):
    """((y, its bound), (z, its bound))"""
    z = p if bias is None else p + bias.double()
    dz = 2.01 * H * p.abs() + (0 if bias is None else H * z.abs())
    y, _ = act64(z, kind)
    dy = dz * (1.13 if kind else 1) + (A[dtype] * y.abs() + 2.0 ** -126 * z.abs() if kind else 0)
    if gate is not None:
        y, dy = y * gate.double(), dy * gate.double().abs()
        dy = dy + H * y.abs()
    if residual is not None:
        y = y + residual.double()
        dy = dy + H * y.abs()
    return (y, dy + U[dtype] * (y.abs() + dy) + TINY[dtype]), (z, dz + U[dtype] * (z.abs() + dz) + TINY[dtype])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("m,n,k", SIZES + [c[0] for c in P.LINEAR])
def test_linear(lib, m, n, k, dtype):  # noqa: F811
    dt = DT[dtype]
    operand = operands(m, n, k, m)
    p = product(*operand)
    bias, gate, residual = (0.5 * rand(n, seed=2)).to(dt), rand(m, n, seed=3).to(dt), (2 * rand(m, n, seed=4)).to(dt)
    for b, kind, g, r, pad in ((None, None, None, None, None), (bias, None, None, residual, None), (bias, "gelu", gate, residual, None),
                               (None, "silu", gate, None, (5, 1)), (bias.float(), "gelu_tanh", None, None, (8, 8)),
                               (bias, "relu", gate, residual, (3, 0))):
        c = None
        if pad:
            g, r = (t if t is None else padded(t, *pad) for t in (g, r))
            c = padded(torch.zeros(m, n, device="cuda", dtype=dt), *pad)
        (y, by), (z, bz) = bounds(p, dt, b, kind, g, r)
        got, kept = lib.block128_linear(*operand, b, kind, g, r, preact=True, c_dtype=dt, c=c)
        close(got, y, by, f"y, {kind}")
        close(kept, z, bz, f"z, {kind}")


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", range(len(GROUPS) + len(P.GROUPED)))
def test_grouped(lib, case, dtype):  # noqa: F811
    dt = DT[dtype]
    sizes, n, k, head, tail = (GROUPS + [c[0] for c in P.GROUPED])[case]
    T, at = sum(sizes) + head + tail, offsets_of(sizes, head)
    a, sa, b, sb = operands(T, n, k, case, len(sizes))
    gate = rand(T, n, seed=3).to(dt)
    p, lo = torch.zeros(T, n, dtype=torch.float64, device="cuda"), head
    for e, rows in enumerate(sizes):
        if rows:
            p[lo:lo + rows] = product(a[lo:lo + rows], sa[:, lo:lo + rows], b[e], sb[e])
        lo += rows
    for kind, g, pad in ((None, None, None), ("gelu", gate, None), ("silu", gate, (5, 1)), ("gelu_tanh", None, (8, 8))):
        c = padded(torch.zeros(T, n, device="cuda", dtype=dt), *pad) if pad else None
        g = padded(g, *pad) if pad and g is not None else g
        (y, by), (z, bz) = bounds(p, dt, None, kind, g, None)
        got, kept = lib.block128_grouped_gemm(a, sa, b, sb, at, kind, g, preact=True, c_dtype=dt, c=c)
        close(got, y, by, f"y, {kind}")
        close(kept, z, bz, f"z, {kind}")
