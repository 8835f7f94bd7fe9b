"""Refusals of the products with what follows them and on rows in groups, before any device work (no GPU needed)."""

import ctypes
import os

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


def ends(lib, bias=None, gate=None, residual=None, preact=None, ldgate=128, ldresidual=128, ldpreact=128, act=0, bias_dtype=0):
    return lib._Ends(bias, gate, residual, preact, ldgate, ldresidual, ldpreact, act, bias_dtype)


def test_linear_refusals(lib):
    f = lib._lib.mxgemm_block128_linear

    def call(A=GOOD, SA=GOOD, B=GOOD, SB=GOOD, C=GOOD, ldc=128, M=64, N=128, K=256, fa=0, fb=0, ct=1, flags=0, ws=GOOD,
             nws=1 << 40, e=None, **kw):
        return f(A, SA, B, SB, C, ldc, M, N, K, fa, fb, ct, ctypes.byref(e or ends(lib, **kw)), flags, ws, nws, None)
    assert call() == lib.MXG_ERR_DEVICE                      # valid; no GPU owns these pointers here
    assert call(bias=GOOD, bias_dtype=1, gate=GOOD, residual=GOOD, preact=GOOD, act=4) == lib.MXG_ERR_DEVICE
    assert f(GOOD, GOOD, GOOD, GOOD, GOOD, 128, 64, 128, 256, 0, 0, 1, None, 0, GOOD, 1 << 40, None) == lib.MXG_ERR_NULL
    for bad in ({"M": -1}, {"N": -1, "ldc": 0}, {"K": -16}, {"ldc": 127}, {"K": 1 << 23}, {"ldc": (1 << 21) + 1},
                {"gate": GOOD, "ldgate": 127}, {"residual": GOOD, "ldresidual": 0}, {"preact": GOOD, "ldpreact": (1 << 21) + 1}):
        assert call(**bad) == lib.MXG_ERR_SHAPE, bad
    for bad in ({"act": 5}, {"act": -1}, {"bias": GOOD, "bias_dtype": 2}, {"fa": 2}, {"ct": 3}):
        assert call(**bad) == lib.MXG_ERR_FMT, bad
    for flags in (1, 2, 256, 512):
        assert call(flags=flags) == lib.MXG_ERR_FLAGS
    assert call(ldgate=0, ldresidual=-5, ldpreact=1 << 40, bias_dtype=9) == lib.MXG_ERR_DEVICE  # of tensors that are not there
    for bad in ({"K": 100}, {"gate": GOOD + 1}, {"residual": GOOD + 1}, {"preact": GOOD + 1}, {"bias": GOOD + 1, "bias_dtype": 1},
                {"bias": GOOD + 2, "bias_dtype": 0}, {"C": GOOD + 1}, {"A": GOOD + 8}):
        assert call(**bad) == lib.MXG_ERR_ALIGN, bad
    assert call(bias=GOOD + 2, bias_dtype=1) == lib.MXG_ERR_DEVICE
    for name in ("A", "SA", "B", "SB", "C"):
        assert call(**{name: None}) == lib.MXG_ERR_NULL, name
    assert call(A=None, M=0) == lib.MXG_OK and call(C=None, N=0, ldc=0) == lib.MXG_OK
    assert call(A=None, SA=None, B=None, SB=None, K=0) == lib.MXG_ERR_DEVICE                # an empty sum is work
    need = lib._lib.mxgemm_block128_workspace_bytes(64, 1024, 7168, 1, 1)
    assert need > 0
    assert call(N=1024, K=7168, ldc=1024, ws=None) == lib.MXG_ERR_NULL
    assert call(N=1024, K=7168, ldc=1024, nws=need - 1) == lib.MXG_ERR_SHAPE


def test_activation_backward_refusals(lib):
    f = lib._lib.mxgemm_activation_backward

    def call(DY=GOOD, Z=GOOD, GATE=None, DZ=GOOD, DGATE=None, DBIAS=None, lds=(128,) * 5, M=4096, N=128, act=2, dt=1, flags=0,
             ws=GOOD, nws=1 << 40):
        return f(DY, Z, GATE, DZ, DGATE, DBIAS, None if lds is None else (ctypes.c_int64 * 5)(*lds), M, N, act, dt, flags, ws, nws, None)
    assert call() == lib.MXG_ERR_DEVICE and call(GATE=GOOD, DGATE=GOOD, DBIAS=GOOD) == lib.MXG_ERR_DEVICE
    for bad in ({"M": -1}, {"N": -1}, {"M": 1 << 31}, {"N": 1 << 31}, {"lds": (127, 128, 128, 128, 128)}, {"lds": (128, 0, 128, 128, 128)},
                {"lds": (128, 128, 128, 1 << 41, 128)}):
        assert call(**bad) == lib.MXG_ERR_SHAPE, bad
    assert call(lds=(128, 128, 0, 128, 0)) == lib.MXG_ERR_DEVICE                            # of a gate that is not there
    assert call(act=5) == lib.MXG_ERR_FMT and call(act=-1) == lib.MXG_ERR_FMT and call(dt=3) == lib.MXG_ERR_FMT
    assert call(flags=1) == lib.MXG_ERR_FLAGS
    for bad in ({"DY": None}, {"Z": None}, {"DZ": None}, {"GATE": GOOD}, {"DGATE": GOOD}, {"lds": None}):
        assert call(**bad) == lib.MXG_ERR_NULL, bad
    for bad in ({"DY": GOOD + 1}, {"DZ": GOOD + 1}, {"DBIAS": GOOD + 2}, {"DBIAS": GOOD, "ws": GOOD + 8}):
        assert call(**bad) == lib.MXG_ERR_ALIGN, bad
    need = lib._lib.mxgemm_activation_backward_workspace_bytes(4096, 128)
    assert need > 0 and lib._lib.mxgemm_activation_backward_workspace_bytes(100, 128) == 0
    assert call(DBIAS=GOOD, ws=None) == lib.MXG_ERR_NULL and call(DBIAS=GOOD, nws=need - 1) == lib.MXG_ERR_SHAPE
    assert call(ws=None, nws=0) == lib.MXG_ERR_DEVICE
    assert call(DY=None, Z=None, DZ=None, N=0) == lib.MXG_OK


def test_group_blocks(lib):
    from oracle import feed_forward as F
    for rows in (0, 1, 5, 127, 128, 129, 1000, 8192, 1 << 24):
        for groups in (0, 1, 2, 7, 128, 1024):
            assert lib.group_blocks(rows, groups) == F.group_blocks(rows, groups)
    assert lib.group_blocks(-1, 2) == lib.group_blocks(5, -1) == lib.group_blocks(5, 1025) == lib.group_blocks((1 << 24) + 1, 1) == 0


def test_quantize_grouped_refusals(lib):
    f = lib._lib.mxgemm_block128_quantize_grouped

    def call(X=GOOD, ldx=256, off=GOOD, Q=GOOD, S=GOOD, QT=GOOD, ST=GOOD, T=64, E=4, K=256, dt=1, fmt=0, flags=0):
        return f(X, ldx, off, Q, S, QT, ST, T, E, K, dt, fmt, flags, None)
    assert call() == lib.MXG_ERR_DEVICE and call(Q=None, S=None) == lib.MXG_ERR_DEVICE
    for bad in ({"T": -1}, {"E": -1}, {"K": -1}, {"ldx": 255}, {"T": (1 << 24) + 1}, {"E": 1025}, {"K": 1 << 31, "ldx": 1 << 31}):
        assert call(**bad) == lib.MXG_ERR_SHAPE, bad
    assert call(dt=3) == lib.MXG_ERR_FMT and call(fmt=2) == lib.MXG_ERR_FMT
    assert call(flags=lib.MXG_QUANT_SQUARE) == lib.MXG_ERR_FLAGS and call(flags=512) == lib.MXG_ERR_FLAGS
    for bad in ({"X": None}, {"off": None}, {"QT": None}, {"ST": None}, {"Q": None}, {"S": None}):
        assert call(**bad) == lib.MXG_ERR_NULL, bad
    for bad in ({"X": GOOD + 1}, {"Q": GOOD + 8}, {"QT": GOOD + 8}, {"ST": GOOD + 2}, {"off": GOOD + 2},
                {"off": GOOD + 4, "flags": lib.MXG_GROUP_OFFSETS64}):
        assert call(**bad) == lib.MXG_ERR_ALIGN, bad
    assert call(off=GOOD + 4) == lib.MXG_ERR_DEVICE
    assert call(X=None, T=0) == lib.MXG_OK and call(X=None, K=0, ldx=0) == lib.MXG_OK
    assert call(E=0, QT=None, ST=None) == lib.MXG_ERR_DEVICE                                # the rows' codes are work


def test_grouped_refusals(lib):
    f = lib._lib.mxgemm_block128_grouped

    def call(A=GOOD, SA=GOOD, B=GOOD, SB=GOOD, off=GOOD, C=GOOD, ldc=128, T=64, E=4, N=128, K=256, fa=0, fb=0, ct=1, flags=0,
             e=None, **kw):
        return f(A, SA, B, SB, off, C, ldc, T, E, N, K, fa, fb, ct, None if e is False else ctypes.byref(ends(lib, **kw)), flags, None)
    assert call() == lib.MXG_ERR_DEVICE and call(e=False) == lib.MXG_ERR_DEVICE
    assert call(gate=GOOD, preact=GOOD, act=1, flags=256 | 512 | 1024) == lib.MXG_ERR_DEVICE
    for bad in ({"T": -1}, {"E": -1}, {"N": -1, "ldc": 0}, {"K": 0}, {"K": -16}, {"ldc": 127}, {"T": (1 << 24) + 1}, {"E": 1025},
                {"K": 1 << 23}, {"ldc": (1 << 21) + 1}, {"gate": GOOD, "ldgate": 127}, {"T": 1 << 24, "N": 1 << 20, "ldc": 1 << 20}):
        assert call(**bad) == lib.MXG_ERR_SHAPE, bad
    for bad in ({"fa": 2}, {"fb": 3}, {"ct": 3}, {"act": 5}):
        assert call(**bad) == lib.MXG_ERR_FMT, bad
    for bad in ({"flags": 1}, {"flags": 2}, {"bias": GOOD}, {"residual": GOOD}):
        assert call(**bad) == lib.MXG_ERR_FLAGS, bad
    for bad in ({"K": 100}, {"A": GOOD + 8}, {"C": GOOD + 1}, {"off": GOOD + 2}, {"gate": GOOD + 1}, {"off": GOOD + 4, "flags": 256}):
        assert call(**bad) == lib.MXG_ERR_ALIGN, bad
    for name in ("A", "SA", "B", "SB", "C", "off"):
        assert call(**{name: None}) == lib.MXG_ERR_NULL, name
    assert call(A=None, T=0) == lib.MXG_OK and call(C=None, N=0, ldc=0) == lib.MXG_OK
    assert call(A=None, SA=None, B=None, SB=None, E=0) == lib.MXG_ERR_DEVICE


def test_weight_gradient_refusals(lib):
    f = lib._lib.mxgemm_block128_grouped_weight_gradient

    def call(A=GOOD, SA=GOOD, B=GOOD, SB=GOOD, off=GOOD, C=GOOD, ldc=128, blocks=3, E=4, M=64, N=128, fa=0, fb=0, flags=0,
             ws=GOOD, nws=1 << 40):
        return f(A, SA, B, SB, off, C, ldc, blocks, E, M, N, fa, fb, flags, ws, nws, None)
    assert call() == lib.MXG_ERR_DEVICE and call(flags=256 | lib.MXG_B128_ACCUMULATE) == lib.MXG_ERR_DEVICE
    for bad in ({"blocks": -1}, {"E": -1}, {"M": -1}, {"N": -1, "ldc": 0}, {"ldc": 127}, {"blocks": 1 << 16}, {"E": 1025},
                {"ldc": (1 << 21) + 1}, {"M": 1 << 31}, {"E": 1024, "M": 1 << 20, "N": 1 << 20, "ldc": 1 << 20}):
        assert call(**bad) == lib.MXG_ERR_SHAPE, bad
    assert call(fa=2) == lib.MXG_ERR_FMT and call(fb=2) == lib.MXG_ERR_FMT
    assert call(flags=1) == lib.MXG_ERR_FLAGS and call(flags=512) == lib.MXG_ERR_FLAGS
    for name in ("A", "SA", "B", "SB", "C", "off"):
        assert call(**{name: None}) == lib.MXG_ERR_NULL, name
    for bad in ({"A": GOOD + 8}, {"SB": GOOD + 2}, {"C": GOOD + 2}, {"off": GOOD + 2}):
        assert call(**bad) == lib.MXG_ERR_ALIGN, bad
    need = lib._lib.mxgemm_block128_grouped_weight_gradient_workspace_bytes(80, 1, 64, 128)
    assert need > 0 and lib._lib.mxgemm_block128_grouped_weight_gradient_workspace_bytes(3, 4, 64, 128) == 0
    assert call(blocks=80, E=1, ws=None) == lib.MXG_ERR_NULL and call(blocks=80, E=1, nws=need - 1) == lib.MXG_ERR_SHAPE
    assert call(blocks=80, E=1, ws=GOOD + 8) == lib.MXG_ERR_ALIGN and call(ws=None, nws=0) == lib.MXG_ERR_DEVICE
    assert call(C=None, E=0) == lib.MXG_OK and call(C=None, M=0) == lib.MXG_OK and call(C=None, N=0, ldc=0) == lib.MXG_OK


def test_wrappers_refuse_host_tensors(lib):
    """Tensors on the host are refused, whatever else is right; wrong shapes and types are, too, where they are seen first."""
    import torch
    a, sa = torch.zeros(8, 256).to(torch.float8_e4m3fn), torch.ones(2, 8)
    b, sb = torch.zeros(3, 64, 256).to(torch.float8_e4m3fn), torch.ones(3, 1, 2)
    off = torch.tensor([0, 2, 2, 8])
    x = torch.zeros(8, 64)
    for call in (lambda: lib.block128_linear(a, sa, b[0], sb[0]), lambda: lib.block128_grouped_gemm(a, sa, b, sb, off),
                 lambda: lib.activation_backward(x, x, "silu", x, True),
                 lambda: lib.block128_quantize(x, cols=True, offsets=off),
                 lambda: lib.block128_grouped_weight_gradient(b[0, :, :128].contiguous(), torch.ones(1, 64), a[:, :128].contiguous(),
                                                              torch.ones(1, 8), off)):
        with pytest.raises(lib.MxgemmRuntimeError) as e:
            call()
        assert e.value.status == lib.MXG_ERR_DEVICE
