"""How the products with what follows them and on rows in groups are called: the short way of the wrappers against the long
one, other streams, captured graphs, offsets that are wrong, refusals, inputs past 32 bits, and the example that runs them
together."""

import os
import sys

import numpy as np
import pytest
import torch

from test_gpu_bind import same, slow  # noqa: F401
from test_gpu_large_counts import need, over, repeats
from test_gpu_streams import check as check_streams

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    import block_scaled_precision_e4m3_amd as lib
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    assert lib._torch().fast is not None, "_bind.so is not built"
    return lib


def rand(*shape, seed=0):
    return torch.randn(*shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))


def offsets(*sizes, head=0, dtype=torch.int32):
    return torch.tensor([head] + (head + np.cumsum(sizes)).tolist(), dtype=dtype, device="cuda")


def operands(lib, m, n, k, groups=None, seed=0):
    a, sa, _, _ = lib.block128_quantize(rand(m, k, seed=seed))
    b, sb, _, _ = lib.block128_quantize(rand(*(() if groups is None else (groups,)), n, k, seed=seed + 1) / k ** 0.5, square=True)
    return a, sa, b, sb


def all_same(got, want):
    got, want = (t if isinstance(t, tuple) else (t,) for t in (got, want))
    assert len(got) == len(want)
    for g, w in zip(got, want):
        same(g, w)


# --- the short way --------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_short_and_long_way(lib, slow, dtype):  # noqa: F811
    f = lib._torch().fast
    for m, n, k in ((3, 136, 256), (128, 1000, 4096), (300, 200, 272)):
        a, sa, b, sb = operands(lib, m, n, k)
        bias, g, r = rand(n, seed=2), rand(m, n, seed=3).to(dtype), rand(m, n + 8, seed=4).to(dtype)[:, :n]
        for args in ((None, None, None, None, False), (bias, "gelu", g, r, True), (bias.to(dtype), "relu", None, r, 1), (None, "silu", g, None, 0)):
            all_same(f.linear(a, sa, b, sb, *args, dtype, None), slow(lambda: lib.block128_linear(a, sa, b, sb, *args, c_dtype=dtype)))
        c = torch.zeros(m, n + 4, device="cuda", dtype=dtype)[:, :n]
        assert f.linear(a, sa, b, sb, None, None, None, None, False, None, c) is c
        all_same(c, slow(lambda: lib.block128_linear(a, sa, b, sb, c_dtype=dtype)))
        dy, z = rand(m, n, seed=5).to(dtype), rand(m, n, seed=6).to(dtype)
        for args in ((None, None, False), ("silu", g, True), ("gelu_tanh", r, False), ("gelu", None, 1)):
            all_same(f.activation_backward(dy, z, *args), slow(lambda: lib.activation_backward(dy, z, *args)))
    for sizes in ((0, 3, 1), (90, 0, 200)):
        for index in (torch.int32, torch.int64):
            t = sum(sizes) + 5
            off = offsets(*sizes, head=2, dtype=index)
            a, sa, b, sb = operands(lib, t, 136, 256, 3)
            g, x = rand(t, 136, seed=3).to(dtype), rand(t, 200, seed=4).to(dtype)
            for args in ((None, None, False), ("silu", g, True)):
                all_same(f.grouped(a, sa, b, sb, off, *args, dtype, None), slow(lambda: lib.block128_grouped_gemm(a, sa, b, sb, off, *args, c_dtype=dtype)))
            c = [torch.full((t, 136), 3, device="cuda", dtype=dtype) for _ in range(2)]
            got = f.grouped(a, sa, b, sb, off, None, None, True, None, c[0])
            assert got[0] is c[0]
            all_same(got, slow(lambda: lib.block128_grouped_gemm(a, sa, b, sb, off, preact=True, c=c[1])))
            for rows, fmt, pow2 in ((True, 0, False), (False, 1, True)):
                all_same(f.quantize_grouped(x, off, fmt, rows, pow2),
                         slow(lambda: lib.block128_quantize(x, fmt, rows, True, pow2=pow2, offsets=off)))
            _, _, p, sp = lib.block128_quantize(x, cols=True, offsets=off)
            _, _, q, sq = lib.block128_quantize(g, fmt=1, cols=True, offsets=off)
            same(f.grouped_weight_gradient(p, sp, q, sq, off, None, False), slow(lambda: lib.block128_grouped_weight_gradient(p, sp, q, sq, off)))
            c = [torch.ones(3, 200, 136, device="cuda") for _ in range(2)]
            assert f.grouped_weight_gradient(p, sp, q, sq, off, c[0], True) is c[0]
            same(c[0], slow(lambda: lib.block128_grouped_weight_gradient(p, sp, q, sq, off, c[1], True)))


def test_short_way_leaves_the_rest_to_the_checks(lib):
    f = lib._torch().fast
    a, sa, b, sb = operands(lib, 5, 64, 256, 2)
    off, x = offsets(2, 3), rand(5, 64).bfloat16()
    lin = (a, sa, b[0], sb[0])
    for bad in (lambda: f.linear(*lin, None, "other", None, None, False, None, None), lambda: f.linear(*lin, None, 1, None, None, False, None, None),
                lambda: f.linear(*lin, x[0, :63].contiguous(), None, None, None, False, None, None),
                lambda: f.linear(*lin, None, None, x.float(), None, False, None, None),
                lambda: f.linear(*lin, None, None, x[:4], None, False, None, None), lambda: f.linear(*lin, None, None, x.t().contiguous().t(), None, False, None, None),
                lambda: f.linear(*lin, None, None, x[:1].expand(5, 64), None, False, None, None),
                lambda: f.linear(*lin, None, None, None, x.cpu(), False, None, None), lambda: f.linear(*lin, None, None, None, None, False, torch.float64, None),
                lambda: f.linear(*lin, x[0].clone().requires_grad_(), None, None, None, False, None, None),
                lambda: f.linear(a, sa, b, sb, None, None, None, None, False, None, None),
                lambda: f.grouped(a, sa, b, sb, off[:2], None, None, False, None, None), lambda: f.grouped(a, sa, b, sb, off.float(), None, None, False, None, None),
                lambda: f.grouped(a, sa, b, sb, off.cpu(), None, None, False, None, None), lambda: f.grouped(a, sa, b, sb, None, None, None, False, None, None),
                lambda: f.grouped(a, sa[:1], b, sb, off, None, None, False, None, None),
                lambda: f.activation_backward(x, x.float(), None, None, False), lambda: f.activation_backward(x, x[:4], None, None, False),
                lambda: f.activation_backward(x, x, "no", None, False), lambda: f.activation_backward(x[0], x[0], None, None, False),
                lambda: f.quantize_grouped(x.double(), off, 0, True, False), lambda: f.quantize_grouped(x, off[None], 0, True, False),
                lambda: f.grouped_weight_gradient(a, sa, a, sa, off, None, True)):
        assert bad() is None


def test_refusals_say_what_is_wrong(lib):
    a, sa, b, sb = operands(lib, 6, 64, 256, 2)
    off, x = offsets(2, 4), rand(6, 64).bfloat16()
    _, _, q, s = lib.block128_quantize(x, cols=True, offsets=off)
    for status, call in ((lib.MXG_ERR_FMT, lambda: lib.block128_linear(a, sa, b[0], sb[0], activation="tanh")),
                         (lib.MXG_ERR_FMT, lambda: lib.block128_linear(a, sa, b[0], sb[0], activation=["relu"])),
                         (lib.MXG_ERR_SHAPE, lambda: lib.block128_linear(a, sa, b[0], sb[0], bias=x[0, :60].contiguous())),
                         (lib.MXG_ERR_FMT, lambda: lib.block128_linear(a, sa, b[0], sb[0], bias=x[0].half())),
                         (lib.MXG_ERR_ALIGN, lambda: lib.block128_linear(a, sa, b[0], sb[0], gate=x[:1].expand(6, 64))),
                         (lib.MXG_ERR_SHAPE, lambda: lib.block128_linear(a, sa, b[0], sb[0], residual=x[:5])),
                         (lib.MXG_ERR_FMT, lambda: lib.block128_linear(a, sa, b[0], sb[0], c=x.float(), c_dtype=torch.bfloat16)),
                         (lib.MXG_ERR_FLAGS, lambda: lib.block128_linear(a, sa, b[0], sb[0], residual=x.clone().requires_grad_())),
                         (lib.MXG_ERR_FLAGS, lambda: lib.block128_linear(a, sa, b[0], sb[0], bias=x[0].clone().requires_grad_())),
                         (lib.MXG_ERR_FLAGS, lambda: lib.block128_grouped_gemm(a, sa, b, sb, off, gate=x.clone().requires_grad_())),
                         (lib.MXG_ERR_FLAGS, lambda: lib.activation_backward(x.clone().requires_grad_(), x)),
                         (lib.MXG_ERR_NULL, lambda: lib.block128_grouped_gemm(a, sa, b, sb, None)),
                         (lib.MXG_ERR_SHAPE, lambda: lib.block128_grouped_gemm(a, sa, b, sb, off[:2])),
                         (lib.MXG_ERR_FMT, lambda: lib.block128_grouped_gemm(a, sa, b, sb, off.float())),
                         (lib.MXG_ERR_ALIGN, lambda: lib.block128_grouped_gemm(a, sa, b, sb, off.repeat(2)[::2][:3])),
                         (lib.MXG_ERR_SHAPE, lambda: lib.block128_grouped_gemm(a, sa, b[0], sb[0], off)),
                         (lib.MXG_ERR_FLAGS, lambda: lib.block128_quantize(x, offsets=off)),
                         (lib.MXG_ERR_FLAGS, lambda: lib.block128_quantize(x, cols=True, square=True, offsets=off)),
                         (lib.MXG_ERR_SHAPE, lambda: lib.block128_quantize(x[None], cols=True, offsets=off)),
                         (lib.MXG_ERR_SHAPE, lambda: lib.block128_grouped_weight_gradient(q, s, q[:, :128].contiguous(), s[:1], off)
                          if q.shape[1] > 128 else lib.block128_grouped_weight_gradient(q, s, q[:, :64].contiguous(), s, off)),
                         (lib.MXG_ERR_SHAPE, lambda: lib.block128_grouped_weight_gradient(q, s[:, :60].contiguous(), q, s, off)),
                         (lib.MXG_ERR_NULL, lambda: lib.block128_grouped_weight_gradient(q, s, q, s, off, accumulate=True)),
                         (lib.MXG_ERR_FMT, lambda: lib.block128_grouped_weight_gradient(q, s, q, s, off, torch.zeros(2, 64, 64, device="cuda").bfloat16())),
                         (lib.MXG_ERR_SHAPE, lambda: lib.block128_grouped_weight_gradient(q, s, q, s, off, torch.zeros(3, 64, 64, device="cuda"))),
                         (lib.MXG_ERR_NULL, lambda: lib.activation_backward(x, x, gate=x, out=(x, None))),
                         (lib.MXG_ERR_SHAPE, lambda: lib.activation_backward(x, x, gate=x, out=(x, x))),
                         (lib.MXG_ERR_SHAPE, lambda: lib.activation_backward(x, x[:5])),
                         (lib.MXG_ERR_ALIGN, lambda: lib.activation_backward(x[:1].expand(6, 64), x))):
        with pytest.raises(lib.MxgemmError) as e:
            call()
        assert e.value.status == status, e.value
    with torch.no_grad():  # nothing is lost here
        lib.block128_linear(a, sa, b[0], sb[0], residual=x.clone().requires_grad_())
        lib.activation_backward(x.clone().requires_grad_(), x)


def test_given_outputs_count_as_changed(lib):
    a, sa, b, sb = operands(lib, 6, 64, 256, 2)
    off = offsets(2, 4)
    c = rand(6, 64)
    for call in (lambda: lib.block128_linear(a, sa, b[0], sb[0], c=c), lambda: lib.block128_grouped_gemm(a, sa, b, sb, off, c=c),
                 lambda: lib.activation_backward(c, c, out=(c, None)),
                 lambda: lib.block128_linear(a, sa, b[0], sb[0], c=c, stream=torch.cuda.current_stream()),
                 lambda: lib.block128_grouped_gemm(a, sa, b, sb, off, c=c, stream=torch.cuda.current_stream())):
        before = c._version
        call()
        assert c._version > before


# --- streams and graphs ---------------------------------------------------------------

def test_other_streams(lib):
    a, sa, b, sb = operands(lib, 1000, 1024, 512)
    g = rand(1000, 1024, seed=3).bfloat16()
    check_streams(lambda **kw: lib.block128_linear(a, sa, b, sb, activation="silu", gate=g, preact=True, **kw))
    dy = rand(1000, 1024, seed=4).bfloat16()
    check_streams(lambda **kw: lib.activation_backward(dy, g, "silu", dy, True, **kw),
                  [lib._lib.mxgemm_activation_backward_workspace_bytes(1000, 1024)])
    p, sp, w, sw = operands(lib, 64, 512, 7168)
    check_streams(lambda **kw: (lib.block128_linear(p, sp, w, sw, **kw),), [lib._lib.mxgemm_block128_workspace_bytes(64, 512, 7168, 1, 1)])
    off = offsets(300, 0, 500, head=100)
    a, sa, b, sb = operands(lib, 1000, 1024, 512, 3)
    check_streams(lambda **kw: lib.block128_grouped_gemm(a, sa, b, sb, off, "silu", g, True, **kw))
    check_streams(lambda **kw: lib.block128_quantize(g, cols=True, offsets=off, **kw))
    _, _, q, s = lib.block128_quantize(g, cols=True, offsets=off)
    check_streams(lambda **kw: (lib.block128_grouped_weight_gradient(q, s, q, s, off, **kw),))
    off = offsets(6000)
    _, _, q, s = lib.block128_quantize(rand(6000, 200), cols=True, offsets=off)
    scratch = lib._lib.mxgemm_block128_grouped_weight_gradient_workspace_bytes(q.shape[1] // 128, 1, 200, 200)
    assert scratch > 0
    check_streams(lambda **kw: (lib.block128_grouped_weight_gradient(q, s, q, s, off, **kw),), [scratch])


def test_in_a_graph(lib):
    """Captured once and replayed with other values and other group sizes, with eager work between the replays."""
    T, E, n, k = 400, 6, 264, 272
    g = torch.Generator().manual_seed(3)
    x, w = rand(T, k).bfloat16(), rand(E, n, k, seed=1) / k ** 0.5
    wq, ws, _, _ = lib.block128_quantize(w, square=True)
    gate = rand(T, n, seed=2).bfloat16()
    off = offsets(100, 0, 50, 50, 100, 90)

    def work():
        q, s, qt, st = lib.block128_quantize(x, cols=True, offsets=off)
        y, z = lib.block128_grouped_gemm(q, s, wq, ws, off, "silu", gate, True)
        few = lib.block128_grouped_gemm(q[:8], s[:, :8].contiguous(), wq, ws, off, "gelu")
        dz, dgate, dbias = lib.activation_backward(y, z, "silu", gate, True)
        _, _, gt, gst = lib.block128_quantize(dz, 1, rows=False, cols=True, offsets=off)
        dw = lib.block128_grouped_weight_gradient(gt, gst, qt, st, off)
        dense, kept = lib.block128_linear(q, s, wq[0], ws[0], gate[0], "gelu_tanh", gate, gate, True)
        return q.float(), s, qt.float(), st, y, z, few, dz, dgate, dbias, dw, dense, kept
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for step in range(4):
        x.copy_(rand(T, k, seed=10 + step))
        sizes = torch.multinomial(torch.rand(E, generator=g), T - 7 * step, replacement=True, generator=g).bincount(minlength=E)
        off.copy_(torch.cat((torch.tensor([step]), step + sizes.cumsum(0))).int())
        want = work()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_two_calls_at_once(lib):
    """Calls on two streams share nothing."""
    a, sa, b, sb = operands(lib, 64, 512, 7168)
    dy = rand(3000, 512, seed=4)
    off = offsets(20, 0, 44)
    p, sp, w, sw = operands(lib, 64, 512, 7168, 3)
    calls = (lambda: (lib.block128_linear(a, sa, b, sb, activation="silu"),), lambda: lib.activation_backward(dy, dy, "gelu", None, True),
             lambda: (lib.block128_grouped_gemm(p, sp, w, sw, off),))
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                got.append((i % 3, calls[i % 3]()))
    torch.cuda.synchronize()
    for i, outs in got:
        for x, y in zip(outs, want[i]):
            assert (x is None) == (y is None) and (x is None or torch.equal(x, y))


# --- offsets that are wrong -----------------------------------------------------------

BAD = ([-5, 3, 10], [0, 50, 20], [0, 10, 1 << 30], [40, 40, 0], [1 << 30, -(1 << 30), 7], [30, 0, 30, 0, 30, 0, 30], [0] * 9, [40] * 9)


def units(off, T, per, most):
    """What the kernels make of offsets, in Python: every group's (start, rows, first unit), each of them held in bounds."""
    at = [min(max(v, 0), T) for v in off]
    out, end = [], 0
    for lo, hi in zip(at, at[1:]):
        rows = max(hi - lo, 0)
        out.append((lo, rows, min(end, most)))
        end += -(-rows // per)
    return out, min(end, most)


@pytest.mark.parametrize("case", range(len(BAD)))
def test_wrong_offsets_stay_in_bounds(lib, case):
    """Offsets that decrease or lie outside give wrong rows, which nobody reads, and write nothing outside the outputs."""
    T, n, k = 40, 72, 144
    off = BAD[case]
    E = len(off) - 1
    for start, rows, first in units(off, T, 16, 1 << 20)[0]:  # held in bounds by what the kernels do with them
        assert 0 <= start <= T and 0 <= rows <= T - start
    a, sa, b, sb = operands(lib, T, n, k, E)
    for index in (torch.int32, torch.int64):
        o = torch.tensor(off, dtype=index, device="cuda")
        guard = torch.full((T + 64, n), 7.0, device="cuda")
        lib.block128_grouped_gemm(a, sa, b, sb, o, c=guard[32:32 + T])
        x = rand(T, k)
        G = lib.group_blocks(T, E)
        qt, st = torch.full((k + 8, 128 * G), 1, dtype=torch.uint8, device="cuda"), torch.full((G + 8, k), 7.0, device="cuda")
        lib.block128_quantize(x, rows=False, cols=True, offsets=o, out=(None, None, qt[4:4 + k].view(F8), st[4:4 + G]))
        dw = torch.full((E + 2, k, k), 7.0, device="cuda")
        q, s = qt[4:4 + k].view(F8), st[4:4 + G]
        lib.block128_grouped_weight_gradient(q, s, q, s, o, dw[1:1 + E])
        torch.cuda.synchronize()
        assert torch.all(guard[:32] == 7) and torch.all(guard[32 + T:] == 7)
        assert torch.all(qt[:4] == 1) and torch.all(qt[4 + k:] == 1) and torch.all(st[:4] == 7) and torch.all(st[4 + G:] == 7)
        assert torch.all(dw[0] == 7) and torch.all(dw[1 + E:] == 7)


# --- past 32 bits ---------------------------------------------------------------------

@pytest.fixture
def memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def test_weights_past_32_bits(lib, memory):
    need(30)
    E, n, k = 160, 4096, 7168  # 4.7 GB of codes
    one, scale, _, _ = lib.block128_quantize(rand(n, k), square=True)
    b = torch.empty(E, n, k, dtype=torch.uint8, device="cuda")
    b.zero_()
    b = b.view(F8)
    b[E - 1].view(torch.uint8).copy_(one.view(torch.uint8))
    sb = scale.expand(E, -1, -1).contiguous()
    for m in (3, 700):
        a, sa, _, _ = lib.block128_quantize(rand(m, k, seed=2))
        off = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
        off[E] = m
        off[E - 1] = m - m // 2
        off[1:E - 1] = m - m // 2  # half the rows to the first group, whose weight is zero, and half to the last
        y = lib.block128_grouped_gemm(a, sa, b, sb, off)
        want = lib.block128_grouped_gemm(a[m - m // 2:], sa[:, m - m // 2:].contiguous(), one[None], scale[None], offsets(m // 2))
        assert not y[:m - m // 2].any()
        # another tile may add the blocks of K in the same order, block by block: the same float32 sums
        assert torch.equal(y[m - m // 2:], want)


def test_rows_past_32_bits(lib, memory):
    """K = 128: one block, whose sum does not depend on the tile."""
    need(60)
    T, n, k = 600000, 4096, 128  # 2.5e9 values of C
    part, p = rand(512, k), 512
    aq, asc, _, _ = lib.block128_quantize(part)
    a, sa = over(aq.view(torch.uint8), T).view(F8), over(asc.t().contiguous(), T).t().contiguous()
    b, sb, _, _ = lib.block128_quantize(rand(n, k, seed=1), square=True)
    gate = rand(p, n, seed=2).bfloat16()
    big = over(gate, T)
    want = lib.block128_linear(aq, asc, b, sb, activation="silu", gate=gate, preact=True)
    y, z = lib.block128_linear(a, sa, b, sb, activation="silu", gate=big, preact=True)
    assert repeats(y, want[0]) and repeats(z, want[1])
    del y, z
    y = lib.block128_grouped_gemm(a, sa, b[None].expand(3, -1, -1).contiguous(), sb[None].expand(3, -1, -1).contiguous(),
                                  offsets(512 * 700, 0, T - 512 * 700, dtype=torch.int64), "silu", big)
    assert repeats(y, want[0])
    dz, dgate, _ = lib.activation_backward(big, y, "gelu", big, True)
    small = lib.activation_backward(gate, want[0], "gelu", gate)
    assert repeats(dz, small[0]) and repeats(dgate, small[1])


def test_codes_past_32_bits(lib, memory):
    need(60)
    T, k = 600064, 7168  # 4.3 GB of codes
    part = rand(256, k).bfloat16()
    x = over(part, T)
    off = offsets(128 * 2000, 0, T - 128 * 2000)
    q, s, qt, st = lib.block128_quantize(x, cols=True, offsets=off)
    want = lib.block128_quantize(part, cols=True)
    assert repeats(q, want[0]) and repeats(s.t().contiguous(), want[1].t().contiguous())
    blocks = -(-T // 128)
    assert repeats(st[:blocks], want[3]) and not st[blocks:].any()
    for col in (0, 4095, k - 1):
        assert repeats(qt[col, :T].view(torch.uint8).view(-1, 128), want[2][col].view(torch.uint8).view(-1, 128))
        assert not qt[col, T:].view(torch.uint8).any()


@pytest.mark.parametrize("m", [1, 2])
def test_few_long_rows_of_gradients(lib, memory, m):
    """More columns than a launch's 2^32 work items take 8 at a time and 64 to a row."""
    need(40)
    dy = rand(1, 1 << 20).bfloat16().repeat(m, 513)
    z = torch.ones_like(dy)
    z[:, -5:] = -1
    dz, _, dbias = lib.activation_backward(dy, z, "relu", bias=True)
    assert torch.equal(dz[:, :-5], dy[:, :-5]) and not dz[:, -5:].any()
    assert torch.equal(dbias[:-5], m * dy[0, :-5].float()) and not dbias[-5:].any()


def test_gradients_past_32_bits(lib, memory):
    need(60)
    E, m, n = 70, 8192, 8192  # 4.7e9 values
    x = rand(E, m)
    off = torch.arange(E + 1, device="cuda", dtype=torch.int32)
    _, _, a, sa = lib.block128_quantize(x, rows=False, cols=True, offsets=off)
    c = lib.block128_grouped_weight_gradient(a, sa, a, sa, off)
    for e in (0, 33, E - 1):
        one = lib.block128_grouped_weight_gradient(a[:, 128 * e:128 * e + 128].contiguous(), sa[e:e + 1], a[:, 128 * e:128 * e + 128].contiguous(),
                                                   sa[e:e + 1], offsets(1))
        assert torch.equal(c[e], one[0])


# --- together -------------------------------------------------------------------------

@pytest.mark.parametrize("sizes", [{}, dict(hidden=272, inner=400, tokens=33, sizes=(1, 0, 40), behind=0),
                                   dict(hidden=256, inner=2048, tokens=1, sizes=(0, 0, 130), behind=64)])
def test_feed_forward(sizes):
    """Each operand's codes are off by at most 1/16 / sqrt(3) of a value in root mean square (uniform rounding at the coarse
    end of a binade), 0.037, and a product of two by sqrt(2) of that.  y has gone through the gate's and the up
    product, which both enter h, and the down product: sqrt(6), 0.089.  A gradient of gate or up has besides those of h its
    own chain: dy and down, then the gradient's and x's codes, with the forward pass's error in z and u: sqrt(10), 0.115; dx
    has two of them: the same.  The slope of silu turns an error of z into one of up to 1.1 of it (its second derivative
    is below 0.5): within the same sum."""
    import feed_forward
    for name, e in feed_forward.check(**sizes).items():
        assert e < (0.089 if name.endswith("y") else 0.115), (name, e)


def test_layer_follows_its_weights():
    import feed_forward
    torch.manual_seed(3)
    layer = feed_forward.Experts(3, 256, 128)
    x, off = rand(50, 256).bfloat16(), offsets(20, 0, 30)
    with torch.no_grad():
        first = layer(x, off)
        layer.down.mul_(2)
        assert torch.equal(layer(x, off), 2 * first)  # codes of a doubled weight are the same, scales twice
