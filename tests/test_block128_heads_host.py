"""Refusals of the block-128, rotary and norm entry points, before any device work (no GPU needed), and the rotary
tables against their formulas."""

import ctypes
import math
import os

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GOOD = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    if not os.path.exists(os.path.join(ROOT, "block_scaled_precision_e4m3_amd", "libmxgemm.so")):
        __graft_entry__.build()
    import block_scaled_precision_e4m3_amd as lib
    return lib


def test_quantize_refusals(lib):
    f = lib._lib.mxgemm_block128_quantize

    def call(X=GOOD, ldx=256, Q=GOOD, S=GOOD, QT=None, ST=None, M=64, K=256, L=1, dt=1, fmt=0, flags=0):
        return f(X, ldx, Q, S, QT, ST, M, K, L, dt, fmt, flags, None)
    assert call() == lib.MXG_ERR_DEVICE                      # valid; no GPU owns these pointers here
    assert call(ldx=255) == lib.MXG_ERR_SHAPE
    for bad in ({"M": -1}, {"K": -1}, {"L": -1}, {"M": 1 << 31}, {"M": 1 << 30, "K": 1 << 30, "ldx": 1 << 30}):
        assert call(**bad) == lib.MXG_ERR_SHAPE, bad
    assert call(dt=3) == lib.MXG_ERR_FMT and call(dt=-1) == lib.MXG_ERR_FMT
    assert call(fmt=2) == lib.MXG_ERR_FMT and call(fmt=-1) == lib.MXG_ERR_FMT
    assert call(flags=4) == lib.MXG_ERR_FLAGS
    for bad in ({"X": None}, {"Q": None}, {"S": None}, {"Q": None, "S": None}, {"QT": GOOD}, {"ST": GOOD}):
        assert call(**bad) == lib.MXG_ERR_NULL, bad
    for bad in ({"X": GOOD + 1}, {"Q": GOOD + 8}, {"S": GOOD + 2}, {"QT": GOOD + 4, "ST": GOOD},
                {"QT": GOOD, "ST": GOOD + 1}):
        assert call(**bad) == lib.MXG_ERR_ALIGN, bad
    assert call(X=None, M=0) == lib.MXG_OK and call(K=0, ldx=0) == lib.MXG_OK and call(L=0) == lib.MXG_OK


def test_gemm_refusals(lib):
    f = lib._lib.mxgemm_block128

    def call(A=GOOD, SA=GOOD, B=GOOD, SB=GOOD, C=GOOD, ldc=128, M=64, N=128, K=256, L=1, fa=0, fb=0, ct=1, flags=0,
             ws=GOOD, nws=1 << 40):
        return f(A, SA, B, SB, C, ldc, M, N, K, L, fa, fb, ct, flags, ws, nws, None)
    assert call() == lib.MXG_ERR_DEVICE
    for bad in ({"M": -1}, {"N": -1, "ldc": 0}, {"K": -16}, {"L": -1}, {"ldc": 127}, {"K": 1 << 23}, {"M": 1 << 31},
                {"L": 1 << 30, "M": 1 << 20}, {"ldc": (1 << 21) + 1}):
        assert call(**bad) == lib.MXG_ERR_SHAPE, bad
    assert call(fa=2) == lib.MXG_ERR_FMT and call(fb=2) == lib.MXG_ERR_FMT and call(ct=3) == lib.MXG_ERR_FMT
    assert call(flags=4) == lib.MXG_ERR_FLAGS
    assert call(flags=lib.MXG_B128_ACCUMULATE) == lib.MXG_ERR_FLAGS           # a 16-bit C
    assert call(flags=lib.MXG_B128_ACCUMULATE, ct=0) == lib.MXG_ERR_DEVICE
    assert call(K=100) == lib.MXG_ERR_ALIGN
    for name in ("A", "SA", "B", "SB", "C"):
        assert call(**{name: None}) == lib.MXG_ERR_NULL, name
        assert call(**{name: GOOD + 1}) == lib.MXG_ERR_ALIGN, name
    assert call(C=None, M=0) == lib.MXG_OK and call(C=None, N=0) == lib.MXG_OK and call(C=None, L=0) == lib.MXG_OK
    assert call(A=None, SA=None, B=None, SB=None, K=0) == lib.MXG_ERR_DEVICE  # C = 0 reads no operand


STRIDES = (ctypes.c_int64 * 12)(*([512, 128] * 6))


def test_rope_refusals(lib):
    f = lib._lib.mxgemm_rope

    def call(X=GOOD, Y=GOOD, cos=GOOD, sin=GOOD, pos=GOOD, strides=STRIDES, T=4, H=4, D=128, rot=64, off=64, rows=4,
             layout=0, dt=1, flags=0):
        return f(X, Y, cos, sin, pos, strides, T, H, D, rot, off, rows, layout, dt, flags, None)
    assert call() == lib.MXG_ERR_DEVICE
    for bad in ({"T": -1}, {"H": -1}, {"D": 0, "rot": 0, "off": 0}, {"D": 1025}, {"rot": 63}, {"rot": -2}, {"off": 65},
                {"off": -1}, {"rows": -1}, {"T": 5, "pos": None}, {"T": 1 << 31}, {"H": 1 << 21},
                {"strides": (ctypes.c_int64 * 4)(-1, 128, 512, 128)}):
        assert call(**bad) == lib.MXG_ERR_SHAPE, bad
    assert call(T=5) == lib.MXG_ERR_DEVICE                  # positions may name any rows
    assert call(layout=3) == lib.MXG_ERR_FMT and call(layout=-1) == lib.MXG_ERR_FMT
    assert call(dt=3) == lib.MXG_ERR_FMT and call(flags=4) == lib.MXG_ERR_FLAGS
    for name in ("X", "Y", "cos", "sin"):
        assert call(**{name: None}) == lib.MXG_ERR_NULL, name
    assert call(strides=None) == lib.MXG_ERR_NULL
    for bad in ({"X": GOOD + 1}, {"Y": GOOD + 1}, {"cos": GOOD + 2}, {"sin": GOOD + 2}, {"pos": GOOD + 2},
                {"pos": GOOD + 4, "flags": 2}):
        assert call(**bad) == lib.MXG_ERR_ALIGN, bad
    assert call(X=None, T=0) == lib.MXG_OK and call(X=None, H=0) == lib.MXG_OK
    assert call(cos=None, sin=None, rot=0, off=0) == lib.MXG_ERR_DEVICE


def test_norm_refusals(lib):
    fwd, bwd = lib._lib.mxgemm_qk_norm_rope, lib._lib.mxgemm_qk_norm_rope_backward
    need = lib._lib.mxgemm_qk_norm_rope_backward_workspace_bytes(4, 128)
    assert need > 0 and lib._lib.mxgemm_qk_norm_rope_backward_workspace_bytes(-1, 128) == 0

    def forward(bufs=(GOOD,) * 9, T=4, Hq=4, Hk=2, D=128, rot=64, off=0, rows=4, layout=0, dt=1, wdt=1, flags=0):
        return fwd(*bufs, STRIDES, T, Hq, Hk, D, rot, off, rows, 1e-6, layout, dt, wdt, flags, None)

    def backward(bufs=(GOOD,) * 13, T=4, Hq=4, Hk=2, D=128, rot=64, off=0, rows=4, layout=0, dt=1, wdt=1, flags=0,
                 ws=GOOD, nws=need):
        return bwd(*bufs, STRIDES, T, Hq, Hk, D, rot, off, rows, 1e-6, layout, dt, wdt, flags, ws, nws, None)
    for call, count in ((forward, 9), (backward, 13)):
        assert call() == lib.MXG_ERR_DEVICE
        for bad in ({"T": -1}, {"Hq": -1}, {"Hk": -1}, {"D": 1025}, {"rot": 130}, {"off": 66}):
            assert call(**bad) == lib.MXG_ERR_SHAPE, bad
        assert call(wdt=0) == lib.MXG_ERR_DEVICE and call(wdt=2) == lib.MXG_ERR_FMT and call(layout=7) == lib.MXG_ERR_FMT
        assert call(flags=1) == lib.MXG_ERR_FLAGS            # the transpose is rope's
        for i in range(count):
            bufs = [GOOD] * count
            bufs[i] = None
            want = lib.MXG_ERR_DEVICE if i == count - 1 else lib.MXG_ERR_NULL    # positions may be missing
            assert call(bufs=bufs) == want, i
            bufs[i] = GOOD + 1
            assert call(bufs=bufs) == lib.MXG_ERR_ALIGN, i
    assert backward(ws=None) == lib.MXG_ERR_NULL and backward(nws=need - 1) == lib.MXG_ERR_SHAPE
    assert backward(ws=GOOD + 8) == lib.MXG_ERR_ALIGN
    assert forward(bufs=[None] * 9, T=0) == lib.MXG_OK


def test_python_refusals(lib):
    import torch
    x = torch.zeros(4, 32)
    E = lib.MxgemmValueError
    for bad in (lambda: lib.block128_quantize(x.double()), lambda: lib.block128_quantize(x[0]),
                lambda: lib.block128_quantize(x, fmt=2), lambda: lib.block128_quantize(x, rows=False),
                lambda: lib.block128_quantize(x.t()), lambda: lib.block128_quantize(x, out=(None, None, None, None)),
                lambda: lib.block128_quantize(x[:1].expand(4, 32))):
        with pytest.raises(E):
            bad()
    q = torch.zeros(4, 32, dtype=torch.float8_e4m3fn)
    s = torch.ones(1, 4)
    sq = torch.ones(1, 1)
    for bad in (lambda: lib.block128_gemm(x, s, q, sq), lambda: lib.block128_gemm(q, s, q, s),
                lambda: lib.block128_gemm(q, s, q, sq, b_block=64), lambda: lib.block128_gemm(q, s.double(), q, sq),
                lambda: lib.block128_gemm(q, s, q[:, :16], sq), lambda: lib.block128_gemm(q, s, q, sq, c_dtype=torch.int8),
                lambda: lib.block128_gemm(q, s, q, sq, accumulate=True),
                lambda: lib.block128_gemm(q, s, q, sq, c=torch.zeros(4, 4).t()[:, :3]),
                lambda: lib.block128_gemm(q, torch.ones(1, 8)[:, ::2], q, sq)):
        with pytest.raises(E):
            bad()
    h = torch.zeros(3, 2, 8)
    cos = torch.zeros(3, 4)
    for bad in (lambda: lib.rope(h[0], cos, cos), lambda: lib.rope(h, cos, cos[:2]), lambda: lib.rope(h, cos.double(), cos),
                lambda: lib.rope(h, cos, cos, layout="other"), lambda: lib.rope(h, cos, cos, positions=torch.zeros(2)),
                lambda: lib.rope(h, cos, cos, positions=torch.zeros(3)), lambda: lib.rope(h.transpose(1, 2), cos, cos),
                lambda: lib.rope(h, cos, cos, out=h.half()), lambda: lib.rope(h, cos, None),
                lambda: lib.qk_norm_rope(h, h, torch.ones(8), torch.ones(7), cos, cos),
                lambda: lib.qk_norm_rope(h, h, torch.ones(8), torch.ones(8).half(), cos, cos),
                lambda: lib.qk_norm_rope(h, h.half(), torch.ones(8), torch.ones(8), cos, cos),
                lambda: lib.qk_norm_rope_backward(h, None, h, h, torch.ones(8), torch.ones(8), cos, cos)):
        with pytest.raises(E):
            bad()


def test_rope_tables(lib):
    cos, sin = lib.rope_table(50, 16, base=500.0, device="cpu")
    p, i = 37, 5
    a = p * 500.0 ** (-2 * i / 16)
    assert abs(float(cos[p, i]) - math.cos(a)) < 1e-7 and abs(float(sin[p, i]) - math.sin(a)) < 1e-7
    lin = lib.rope_table(50, 16, base=500.0, scaling="linear", factor=4.0, device="cpu")
    np.testing.assert_allclose(lin[0][::4][:12], cos[:12], atol=1e-7)
    ntk = lib.rope_table(401, 16, base=500.0, scaling="ntk", factor=8.0, device="cpu")
    np.testing.assert_allclose(ntk[0][:50, 0], cos[:, 0], atol=1e-7)                       # the fastest pair as it was
    slow = 500.0 ** (-14 / 16)
    np.testing.assert_allclose(ntk[1][400, 7], math.sin(400 * slow / 8), atol=1e-6)       # the slowest stretched by 8
    y = lib.rope_table(64, 128, scaling="yarn", factor=16.0, original_length=4096, device="cpu")
    m = 0.1 * math.log(16) + 1
    np.testing.assert_allclose(np.hypot(y[0], y[1]), m, rtol=1e-6)
    np.testing.assert_allclose(y[0][:, 0], m * np.cos(np.arange(64)), atol=1e-6)          # turns often: kept
    np.testing.assert_allclose(y[1][:, 63], m * np.sin(np.arange(64) * 10000.0 ** (-126 / 128) / 16), atol=1e-7)
    for bad in ({"rot": 15}, {"rot": 16, "scaling": "other"}, {"rot": 16, "factor": 0.0}, {"rot": 16, "length": -1}):
        with pytest.raises(lib.MxgemmValueError):
            lib.rope_table(**{"length": 4, "device": "cpu", **bad})


def test_more_heads_than_a_launch_has_waves(lib):
    f = lib._lib.mxgemm_rope
    for T, H, want in ((1 << 30, 1 << 6, lib.MXG_ERR_DEVICE), (1 << 30, (1 << 6) + 1, lib.MXG_ERR_SHAPE),
                       ((1 << 31) - 1, 1 << 20, lib.MXG_ERR_SHAPE)):
        assert f(GOOD, GOOD, GOOD, GOOD, GOOD, STRIDES, T, H, 128, 64, 0, 4, 0, 1, 0, None) == want, (T, H)


def test_sums_of_arguments_that_overflow(lib):
    """The end of the rotary part and the number of heads are not taken in arithmetic that overflows."""
    f, n = lib._lib.mxgemm_rope, lib._lib.mxgemm_qk_norm_rope
    for rot, off in ((64, (1 << 63) - 1), (64, (1 << 63) - 64), (1 << 62, 1 << 62), ((1 << 63) - 2, 2), (128, 1), (130, 0)):
        assert f(GOOD, GOOD, GOOD, GOOD, GOOD, STRIDES, 4, 4, 128, rot, off, 4, 0, 1, 0, None) == lib.MXG_ERR_SHAPE, (rot, off)
        assert n(*[GOOD] * 9, STRIDES, 4, 4, 2, 128, rot, off, 4, 1e-6, 0, 1, 1, 0, None) == lib.MXG_ERR_SHAPE, (rot, off)
    for hq, hk in ((1 << 62, 1 << 62), ((1 << 63) - 1, (1 << 63) - 1), (1 << 20, 1), (1, 1 << 20)):
        assert n(*[GOOD] * 9, STRIDES, 4, hq, hk, 128, 64, 0, 4, 1e-6, 0, 1, 1, 0, None) == lib.MXG_ERR_SHAPE, (hq, hk)


def test_workspaces_must_have_the_memory_they_count(lib):
    """An expanded tensor counts one element many times."""
    import torch
    ws = torch.zeros(1, dtype=torch.uint8).expand(1 << 30)
    q, s = torch.zeros(64, 7168, dtype=torch.float8_e4m3fn), torch.ones(56, 64)
    h, w = torch.zeros(3, 2, 16), torch.ones(16)
    x, xs = torch.zeros(32, 64, dtype=torch.float8_e4m3fn), torch.zeros(32, 2, dtype=torch.uint8)
    table = torch.zeros(32, 64, dtype=torch.bfloat16)
    out = tuple(torch.zeros(1) for _ in range(4))
    for bad in (lambda: lib.block128_gemm(q, s, q, s, b_block=1, workspace=ws),
                lambda: lib.qk_norm_rope_backward(h, h, h, h, w, w, workspace=ws),
                lambda: lib.projection_mxfp8(x, x, xs, xs, table, table, 1, 64, 64, workspace=ws, out=out)):
        with pytest.raises(lib.MxgemmValueError, match="workspace"):
            bad()


@pytest.mark.parametrize("length,rot,base,factor", [(4096, 64, 1e4, 4.0), (32768, 128, 1e6, 4.0), (65536, 128, 1e4, 4.0),
                                                    (131072, 128, 1e4, 4.0), (4096, 128, 500.0, 4.0), (8192, 32, 1e4, 16.0),
                                                    (1 << 20, 128, 100.0, 2.0), (100, 16, 1e4, 8.0)])
def test_yarn_ramp(lib, length, rot, base, factor):
    """Every pair's frequency, read off position 1 of the table, against turns = length base^(-2i/rot) / (2 pi): kept above
    32 turns, divided by the factor below one, the ramp between the pairs where the (real) pair index has 32 turns and
    one, those rounded outwards."""
    cos, sin = lib.rope_table(2, rot, base=base, scaling="yarn", factor=factor, original_length=length, device="cpu")
    got = np.arctan2(sin[1].double().numpy(), cos[1].double().numpy())
    index = lambda turns: math.log(length / (2 * math.pi * turns)) * rot / (2 * math.log(base))  # noqa: E731
    lo, hi = max(math.floor(index(32.0)), 0), min(math.ceil(index(1.0)), rot - 1)
    for i in range(rot // 2):
        freq = base ** (-2 * i / rot)
        turns = length * freq / (2 * math.pi)
        part = min(max((i - lo) / (hi - lo), 0.0), 1.0) if hi > lo else float(i > lo)
        want = freq * (1 - part) + freq / factor * part
        # float32 sine and cosine: 2^-24 of their length in either, and in the angle
        assert abs(got[i] - want) <= 2.0 ** -23, (i, turns)
        if turns >= 32:
            assert abs(got[i] - freq) <= 2.0 ** -23
        if turns < 1:
            assert part > 0.9, (i, turns)
        assert part < 1 or turns < 1 or i >= hi


def test_missing_weights_and_scales(lib):
    import torch
    h, w = torch.zeros(3, 2, 8), torch.ones(8)
    q, s = torch.zeros(4, 32, dtype=torch.float8_e4m3fn), torch.ones(1, 4)
    for bad in (lambda: lib.qk_norm_rope(h, h, w, None), lambda: lib.qk_norm_rope(h, h, None, w), lambda: lib.qk_norm_rope(h, None, None, None),
                lambda: lib.qk_norm_rope_backward(h, h, h, h, w, None), lambda: lib.qk_norm_rope_backward(h, h, h, h, None, w),
                lambda: lib.block128_gemm(q, None, q, s, b_block=1), lambda: lib.block128_gemm(q, s, q, None)):
        with pytest.raises(lib.MxgemmValueError) as e:
            bad()
        assert e.value.status == lib.MXG_ERR_NULL


def test_outputs_whose_rows_lie_on_each_other(lib):
    """An expanded output would be written by many rows at once; inputs may be expanded."""
    rope, norm, back = lib._lib.mxgemm_rope, lib._lib.mxgemm_qk_norm_rope, lib._lib.mxgemm_qk_norm_rope_backward
    good = [512, 128]
    arr = lambda s: (ctypes.c_int64 * len(s))(*s)  # noqa: E731

    def call(x, y, T=4, H=4):
        return (rope(GOOD, GOOD, GOOD, GOOD, GOOD, arr(x + y), T, H, 128, 64, 0, 4, 0, 1, 0, None),
                norm(*[GOOD] * 9, arr(x + x + good + y), T, 4, H, 128, 64, 0, 4, 1e-6, 0, 1, 1, 0, None),
                norm(*[GOOD] * 9, arr(x + x + y + good), T, H, 4, 128, 64, 0, 4, 1e-6, 0, 1, 1, 0, None),
                back(*[GOOD] * 13, arr(x * 4 + good + y), T, 4, H, 128, 64, 0, 4, 1e-6, 0, 1, 1, 0, GOOD, 1 << 30, None),
                back(*[GOOD] * 13, arr(x * 4 + y + good), T, H, 4, 128, 64, 0, 4, 1e-6, 0, 1, 1, 0, GOOD, 1 << 30, None))
    for y in ([0, 128], [512, 0], [127, 1024], [512, 127], [128, 128]):
        assert call(good, y) == (lib.MXG_ERR_SHAPE,) * 5, y
    for x, y, T, H in (([0, 0], good, 4, 4), (good, [128, 512], 4, 4), (good, [0, 128], 1, 4), (good, [512, 0], 4, 1),
                       (good, [0, 0], 1, 1), (good, [128, 4096], 4, 4)):
        assert call(x, y, T, H) == (lib.MXG_ERR_DEVICE,) * 5, (x, y)
