"""Counts near the ends of 32-bit arithmetic: launches of 2^32 work items and more, tensors of 2^31 elements and more,
scales whose blocks lie 2^31 bytes apart.  Expected results come from small calls on the repeating part of the inputs, which
are checked elsewhere, or from the oracle."""

import numpy as np
import pytest
import torch

from oracle import block128 as B
from oracle import rope_heads as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import block_scaled_precision_e4m3_amd as lib
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return lib


@pytest.fixture(autouse=True)
def memory():
    """Leaves the card to the next test."""
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def need(gib):
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"{gib} GiB of device memory are not free")


def normal(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def repeats(got, part):
    """Whether got is part over and over along its first axis, to the last, incomplete one."""
    n, p = got.shape[0], part.shape[0]
    got, part = got.reshape(n, -1).view(torch.uint8), part.reshape(p, -1).view(torch.uint8)
    whole = n // p * p
    assert got.shape[1] == part.shape[1]
    for at in range(0, whole, p * 512):
        if not torch.all(got[at:min(whole, at + p * 512)].view(-1, *part.shape) == part).item():
            return False
    return torch.equal(got[whole:], part[:n - whole])


def over(part, n):
    """(n, ...) made of part over and over."""
    p = part.shape[0]
    out = torch.empty((n, *part.shape[1:]), dtype=part.dtype, device="cuda")
    whole = n // p * p
    out[:whole].view(-1, *part.shape).copy_(part.expand(whole // p, *part.shape))
    out[whole:] = part[:n - whole]
    return out


PERIOD = 4096


def test_rope_and_norm_of_many_tokens(lib):
    """2^26 tokens of one head are 2^26 waves of work."""
    need(24)
    T, D = (1 << 26) + 5, 16
    print(f"rope, norm {T}x1x{D}", flush=True)
    cos, sin = lib.rope_table(PERIOD, D)
    part = normal(PERIOD, 1, D).bfloat16()
    x, pos = over(part, T), over(torch.arange(PERIOD, device="cuda", dtype=torch.int32), T)
    w = normal(D, seed=1)
    want = lib.rope(part, cos, sin)
    assert repeats(lib.rope(x, cos, sin, pos), want)
    assert repeats(lib.qk_norm_rope(x, None, w, None, cos, sin, pos)[0], lib.qk_norm_rope(part, None, w, None, cos, sin)[0])
    dx, _, dw, _ = lib.qk_norm_rope_backward(x, None, x, None, w, None, cos, sin, pos)
    assert repeats(dx, lib.qk_norm_rope_backward(part, None, part, None, w, None, cos, sin)[0])
    # the weights' gradient: at most 2^14 + 1 terms to a wave's running sum, and fewer than 256 additions of those
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    ref = mag = 0.0
    for rows, times in ((PERIOD, T // PERIOD), (T % PERIOD, 1)):
        r = R.norm_rotate_backward(f64(part[:rows]), f64(part[:rows]), f64(w), f64(cos[:rows]), f64(sin[:rows]), "half", 0, 1e-6)
        ref, mag = ref + r[1] * times, mag + r[3] * times
    assert (np.abs(f64(dw) - ref) <= (2 ** 14 + 256 + D) * 2.0 ** -24 * mag).all()


def test_quantize_many_batches(lib):
    """More batches than one dimension of a launch has workgroups, and more than 2^31 elements."""
    need(70)
    L, K = (1 << 24) + 3, 144
    print(f"quantise {L}x1x{K}", flush=True)
    part = normal(PERIOD, 1, K).bfloat16()
    x = over(part, L)
    for rows, cols, square in ((True, False, False), (False, True, False)):
        got, want = lib.block128_quantize(x, 0, rows, cols, square), lib.block128_quantize(part, 0, rows, cols, square)
        for g, w in zip(got, want):
            assert (g is None) == (w is None)
            assert g is None or repeats(g, w)
        del got


def test_product_of_many_batches(lib):
    """As many small products as there are weights of a very wide mixture: one row each."""
    need(12)
    L, N, K = (1 << 23) + 1, 16, 16
    print(f"gemm {L}x1x{N}x{K}", flush=True)
    a, sa, _, _ = lib.block128_quantize(normal(PERIOD, 1, K))
    b, sb, _, _ = lib.block128_quantize(normal(PERIOD, N, K, seed=1), square=True)
    big = [over(t.view(torch.uint8), L).view(t.dtype) for t in (a, sa, b, sb)]
    for dtype in (torch.bfloat16, torch.float32):
        assert repeats(lib.block128_gemm(*big, c_dtype=dtype), lib.block128_gemm(a, sa, b, sb, c_dtype=dtype))


def test_quantize_and_product_past_32_bits(lib):
    """Operands and outputs of more than 2^31 elements, the rows past it among those looked at."""
    need(30)
    M, N, K = (1 << 20) + 130, 2056, 2064
    print(f"quantise {M}x{K}, gemm {M}x{N}x{K}", flush=True)
    part = normal(PERIOD, K).bfloat16()
    x = over(part, M)
    q, s, qt, st = lib.block128_quantize(x, 0, True, True)
    want = lib.block128_quantize(part, 0, True, True)
    assert repeats(q, want[0]) and torch.equal(s[:, -130:], want[1][:, :130])
    assert repeats(st[:-1], want[3])       # the last block of 128 rows holds two
    assert torch.equal(qt[:, (1 << 20):(1 << 20) + 128].contiguous().view(torch.uint8), want[2][:, :128].contiguous().view(torch.uint8))
    del x, qt, st
    b, sb, _, _ = lib.block128_quantize(normal(N, K, seed=1), square=True)
    for dtype in (torch.bfloat16, torch.float32):
        # K is not divided at either size, and every tile sums a row's blocks in one order
        assert repeats(lib.block128_gemm(q, s, b, sb, c_dtype=dtype), lib.block128_gemm(*want[:2], b, sb, c_dtype=dtype))
        torch.cuda.empty_cache()


def test_row_scales_of_many_rows(lib):
    """Row scales of one block of K to the next lie 4 M bytes apart: 2^31 and more here, 2^32 and more for two blocks."""
    need(160)
    M, N, K = (1 << 29) + 5, 8, 272
    print(f"gemm {M}x{N}x{K}", flush=True)
    rng = np.random.default_rng(3)
    rows = 96
    host = B.quantize((rng.standard_normal((3 * rows, K)) * np.exp2(rng.integers(-9, 9, (3 * rows, 1)))).astype(np.float32))
    hb, hsb, _, _ = B.quantize(rng.standard_normal((N, K)).astype(np.float32), square=True)
    at = (0, M // 2 - 7, M - rows)             # the rows looked at; nothing depends on what the others hold
    a = torch.empty((M, K), dtype=torch.uint8, device="cuda")
    sa = torch.empty((3, M), device="cuda")
    for i, r in enumerate(at):
        a[r:r + rows] = torch.from_numpy(host[0][i * rows:(i + 1) * rows].copy()).cuda()
        sa[:, r:r + rows] = torch.from_numpy(host[1][:, i * rows:(i + 1) * rows].copy()).cuda()
    c = lib.block128_gemm(a.view(torch.float8_e4m3fn), sa, torch.from_numpy(hb.copy()).cuda().view(torch.float8_e4m3fn),
                          torch.from_numpy(hsb.copy()).cuda())
    ref, s = B.gemm(host[0], host[1], hb, hsb, 0, 0, 128)
    for i, r in enumerate(at):
        got, want, mag = c[r:r + rows].double().cpu().numpy(), ref[i * rows:(i + 1) * rows], s[i * rows:(i + 1) * rows]
        # bfloat16, and what the 8-bit products may drop: as for the other sizes
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * mag).all(), r
