"""Products with bias, activation, gate and residual, their gradients, and rows in groups, on the GPU against float64.

Tolerances.  With S = sum |a||b| a product's value p is off by (K/16 + 4 K/128 + 4) 2^-24 S, for a 16-bit C by 2^-10 S
more (what the 8-bit products may drop): dz.  A bias adds 2^-24 |z|.  An activation's slope is below 1.13 (gelu's and
gelu_tanh's largest), so dz moves it by 1.13 dz at most, and its own arithmetic by A |act|:
A = 2^-15 for 16-bit results: |u| 2^-24 of the exponential's argument with its second rounding, |u| at most 88 before e^-u leaves float32,
together 2^-16.4; 2^-22 of hardware exponential and reciprocal, 4.7e-6 of the tail's polynomial;
A = 2^-20 for float32: 4e-7 of the polynomial and eight roundings of 2^-24 in the products, division and exponential.
What float32 cannot hold of e^-u is below 2^-126 |z|.  Gate and residual add two roundings of 2^-24, and the result is
rounded once: u, half a step of its type relative to it (2^-8, 2^-11; float32's is in the roundings counted), or half of the
smallest subnormal.
"""

import numpy as np
import pytest
import torch

from oracle import block128 as B
from oracle import feed_forward as F

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {torch.float32: 2.0 ** -23, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
A = {torch.float32: 2.0 ** -20, torch.bfloat16: 2.0 ** -15, torch.float16: 2.0 ** -15}
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}
F8 = (torch.float8_e4m3fn, torch.float8_e5m2)


@pytest.fixture(scope="module")
def lib():
    import block_scaled_precision_e4m3_amd as lib
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return lib


def rand(*shape, seed=0):
    return torch.randn(*shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))


def wide(codes, scales, block):
    """float64 values of codes (R, K) with scales (K blocks, R), or (R blocks, K blocks)."""
    r, k = torch.arange(codes.shape[0], device="cuda"), torch.arange(codes.shape[1], device="cuda") // 128
    s = scales.double()
    return codes.float().double() * (s[k][:, r].t() if block == 1 else s[r // 128][:, k])


def matmul(x, w):
    return x @ w.t().contiguous()


def act64(z, kind):
    value, slope = F.activation(z.cpu().numpy(), kind)
    return torch.from_numpy(value).cuda(), torch.from_numpy(slope).cuda()


def padded(t, pad, off=0):
    """The values of t in rows that are further apart, from an element that need not be aligned."""
    buf = torch.empty(t.shape[0], t.shape[1] + pad + off, device="cuda", dtype=t.dtype)
    buf.fill_(7)
    view = buf[:, off:off + t.shape[1]]
    view.copy_(t)
    return view


def close(got, want, bound, what):
    """Element by element; NaN where and only where the reference has it."""
    got = got.double()
    assert got.shape == want.shape
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN elsewhere"
    off = torch.where(got == want, 0.0, (got - want).abs())
    worst = (off / bound).nan_to_num(0.0)
    at = int(worst.argmax()) if worst.numel() else 0
    if worst.numel():
        i, j = divmod(at, worst.shape[-1])
        assert worst.max().item() <= 1, (f"{what}: {worst.max().item():.3g} of the bound at ({i}, {j}) of {tuple(got.shape)}: "
                                         f"{got.reshape(-1)[at].item()} for {want.reshape(-1)[at].item()}")


def ends(p, S, K, dtype, bias, kind, gate, residual):
    """((y, its bound), (z, its bound)) of products p with S = sum |a||b|."""
    dz = (K / 16 + 4 * K / 128 + 4) * 2.0 ** -24 * S + (2.0 ** -10 * S if dtype != torch.float32 else 0)
    z = p if bias is None else p + bias.double()
    dz = dz + 2.0 ** -24 * z.abs()
    y, _ = act64(z, kind)
    dy = dz * (1.13 if kind else 1) + (A[dtype] * y.abs() + 2.0 ** -126 * z.abs() if kind else 0)
    if gate is not None:
        y, dy = y * gate.double(), dy * gate.double().abs()
        dy = dy + 2.0 ** -24 * y.abs()
    if residual is not None:
        y = y + residual.double()
        dy = dy + 2.0 ** -24 * y.abs()
    return (y, dy + U[dtype] * (y.abs() + dy) + TINY[dtype]), (z, dz + U[dtype] * (z.abs() + dz) + TINY[dtype])


def operands(lib, m, n, k, fa=0, fb=0, seed=0, groups=None):
    a, sa, _, _ = lib.block128_quantize(rand(m, k, seed=seed), fmt=fa)
    lead = () if groups is None else (groups,)
    b, sb, _, _ = lib.block128_quantize(rand(*lead, n, k, seed=seed + 1) / k ** 0.5, fmt=fb, square=True)
    return a, sa, b, sb


# --- linear ---------------------------------------------------------------------------

def check_linear(lib, m, n, k, dtype, bias=True, kind=None, gate=False, residual=False, preact=False, fa=0, fb=0, pad=None,
                 bias_f32=False, seed=0):
    print(f"linear {m}x{n}x{k} {dtype} bias {bias} {kind} gate {gate} residual {residual} preact {preact} {fa}{fb} {pad}", flush=True)
    a, sa, b, sb = operands(lib, m, n, k, fa, fb, seed)
    tb = (0.5 * rand(n, seed=seed + 2)).to(torch.float32 if bias_f32 else dtype) if bias else None
    tg = rand(m, n, seed=seed + 3).to(dtype) if gate else None
    tr = (2 * rand(m, n, seed=seed + 4)).to(dtype) if residual else None
    c = None
    if pad:
        tg, tr = (t if t is None else padded(t, *pad) for t in (tg, tr))
        c = padded(torch.zeros(m, n, device="cuda", dtype=dtype), *pad)
    x, w = wide(a, sa, 1), wide(b, sb, 128)
    (y, by), (z, bz) = ends(matmul(x, w), matmul(x.abs(), w.abs()), k, dtype, tb, kind, tg, tr)
    out = lib.block128_linear(a, sa, b, sb, tb, kind, tg, tr, preact, dtype, c)
    torch.cuda.synchronize()
    got, kept = out if preact else (out, None)
    if pad:
        assert got is c
        whole = c._base
        assert torch.all(whole[:, :pad[1]] == 7) and torch.all(whole[:, pad[1] + n:] == 7), "a write beside the columns"
    close(got, y, by, "y")
    if preact:
        assert kept.shape == (m, n) and kept.dtype == dtype
        close(kept, z, bz, "z")
    return got


SIZES = [(1, 24, 16), (1, 7168, 2048), (3, 129, 400), (16, 500, 1040), (17, 1024, 272), (32, 64, 2048), (33, 200, 272),
         (300, 500, 400), (512, 4096, 272), (1000, 4096, 272), (2100, 4100, 272), (2048, 4096, 144), (128, 1000, 4096)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear_sizes(lib, m, n, k, dtype):
    check_linear(lib, m, n, k, DT[dtype], True, "gelu", True, True, True)
    check_linear(lib, m, n, k, DT[dtype], False, "silu", True, False, False, seed=5)
    check_linear(lib, m, n, k, DT[dtype], True, None, False, True, False, seed=9)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("kind", F.ACTIVATIONS)
@pytest.mark.parametrize("m,n,k", [(7, 96, 256), (130, 264, 256)])
def test_linear_options(lib, m, n, k, kind, dtype):
    for mask in range(16):
        check_linear(lib, m, n, k, DT[dtype], bool(mask & 1), kind, bool(mask & 2), bool(mask & 4), bool(mask & 8),
                     bias_f32=bool(mask & 8), seed=mask)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("fa", (0, 1))
@pytest.mark.parametrize("fb", (0, 1))
def test_linear_formats(lib, fa, fb, dtype):
    for m, n, k in ((5, 96, 144), (200, 300, 272), (512, 4096, 144), (1000, 4096, 144), (2100, 4104, 144)):
        check_linear(lib, m, n, k, DT[dtype], True, "silu", True, True, True, fa, fb)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("pad", [(8, 0), (8, 8), (3, 0), (5, 1)])
def test_linear_strides_and_alignment(lib, dtype, pad):
    for m, n, k in ((4, 104, 256), (90, 264, 144), (600, 1001, 144), (2100, 4096, 144)):
        check_linear(lib, m, n, k, DT[dtype], True, "gelu_tanh", True, True, True, pad=pad)


@pytest.mark.parametrize("dtype", list(DT))
def test_linear_into_its_own_residual_and_gate(lib, dtype):
    """The output in place of the residual or the gate gives the same bits."""
    for m, n, k in ((2, 96, 256), (128, 1000, 4096), (300, 264, 272), (2100, 4096, 144)):
        print(f"in place {m}x{n}x{k}", flush=True)
        a, sa, b, sb = operands(lib, m, n, k)
        r = rand(m, n, seed=3).to(DT[dtype])
        want = lib.block128_linear(a, sa, b, sb, residual=r, c_dtype=r.dtype)
        got = r.clone()
        assert lib.block128_linear(a, sa, b, sb, residual=got, c=got) is got
        assert torch.equal(got, want)
        want = lib.block128_linear(a, sa, b, sb, activation="silu", gate=r, c_dtype=r.dtype)
        got = r.clone()
        lib.block128_linear(a, sa, b, sb, activation="silu", gate=got, c=got)
        assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", list(DT))
def test_linear_without_anything_is_the_product(lib, dtype):
    for m, n, k in ((1, 96, 256), (33, 264, 272), (128, 1000, 4096), (600, 1000, 272), (2100, 4096, 272)):
        a, sa, b, sb = operands(lib, m, n, k)
        assert torch.equal(lib.block128_linear(a, sa, b, sb, c_dtype=DT[dtype]), lib.block128_gemm(a, sa, b, sb, c_dtype=DT[dtype]))


def test_linear_empty(lib):
    for m, n in ((0, 64), (3, 0)):
        a, sa, b, sb = operands(lib, m, n, 128)
        y, z = lib.block128_linear(a, sa, b, sb, bias=torch.ones(n, device="cuda"), preact=True, activation="relu")
        assert y.shape == z.shape == (m, n)
    # an empty sum
    e = torch.empty
    a, sa = e(5, 0, device="cuda", dtype=F8[0]), e(0, 5, device="cuda")
    b, sb = e(9, 0, device="cuda", dtype=F8[0]), e(1, 0, device="cuda")
    bias, r = rand(9), rand(5, 9)
    y, z = lib.block128_linear(a, sa, b, sb, bias=bias, activation="silu", residual=r, preact=True, c_dtype=torch.float32)
    assert torch.equal(z, bias.expand(5, 9))
    close(y, act64(bias.double().expand(5, 9), "silu")[0] + r.double(), 2.0 ** -20 * (r.double().abs() + 9), "y")


@pytest.mark.parametrize("kind", F.ACTIVATIONS)
@pytest.mark.parametrize("dtype", list(DT))
def test_activations_over_their_range(lib, kind, dtype):
    """Values that come through the bias alone, from the smallest to where the activations have long been straight."""
    t = DT[dtype]
    x = torch.cat([torch.linspace(-30, 30, 4001), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e-3, -1e-3, 100.0, -100.0, 6e4, -6e4])])
    if t != torch.float16:
        x = torch.cat([x, torch.tensor([1e15, -1e15, 1e30, -1e30, 3e38, -3e38])])
    x = torch.nn.functional.pad(x, (0, -x.numel() % 8)).to(t).cuda()
    n = x.numel()
    for m, k in ((1, 0), (2, 16), (40, 16)):
        a, b = torch.zeros(m, k, device="cuda").to(F8[0]), torch.zeros(n, k, device="cuda").to(F8[0])
        sa, sb = torch.ones(-(-k // 128), m, device="cuda"), torch.ones(-(-n // 128), -(-k // 128), device="cuda")
        y = lib.block128_linear(a, sa, b, sb, bias=x, activation=kind, c_dtype=t)
        want = act64(x.double(), kind)[0].expand(m, n)
        close(y, want, (A[t] + U[t]) * want.abs() + TINY[t] + 2.0 ** -126 * x.double().abs(), f"{kind}")


def test_linear_non_finite(lib):
    """An infinity or NaN reaches the elements of its row, gate or residual, and no others."""
    for m in (3, 70, 300):
        a, sa, b, sb = operands(lib, m, 136, 256)
        r, g = rand(m, 136), rand(m, 136)
        r[2, 5], g[1, 7] = float("nan"), float("inf")
        y = lib.block128_linear(a, sa, b, sb, activation="relu", gate=g, residual=r, c_dtype=torch.float32)
        bad = torch.zeros_like(r, dtype=torch.bool)
        bad[2, 5] = bad[1, 7] = True
        assert torch.equal(~torch.isfinite(y), bad)


# --- gradients ------------------------------------------------------------------------

def check_backward(lib, m, n, dtype, kind, gate, bias, pad=None, seed=0):
    print(f"backward {m}x{n} {dtype} {kind} gate {gate} bias {bias} {pad}", flush=True)
    dy, z = rand(m, n, seed=seed).to(dtype), (2 * rand(m, n, seed=seed + 1)).to(dtype)
    g = rand(m, n, seed=seed + 2).to(dtype) if gate else None
    if pad:
        dy, z, g = (t if t is None else padded(t, *pad) for t in (dy, z, g))
    dz, dgate, dbias = lib.activation_backward(dy, z, kind, g, bias)
    torch.cuda.synchronize()
    assert (dgate is None) == (g is None) and (dbias is None) == (not bias)
    value, slope = act64(z.double(), kind)
    # the slope's parts are below 1.13 each (s, z s (1 - s) and their kind), so its error is A and roundings of them
    err = (A[dtype] + 2.0 ** -22) * 2.5 if kind else 0.0
    d = dy.double()
    t = d.abs() * (1 if g is None else g.double().abs())
    want = d * slope * (1 if g is None else g.double())
    bound = t * err + 2.0 ** -22 * want.abs()
    close(dz, want, bound + U[dtype] * (want.abs() + bound) + TINY[dtype], "dz")
    if gate:
        wg = d * value
        bg = A[dtype] * wg.abs() + 2.0 ** -22 * wg.abs() + d.abs() * z.double().abs() * 2.0 ** -126
        close(dgate, wg, bg + U[dtype] * (wg.abs() + bg) + TINY[dtype], "dgate")
    if bias:
        assert dbias.dtype == torch.float32
        # a sum of m float32 values in any order
        close(dbias[None], want.sum(0)[None], (bound.sum(0) + m * 2.0 ** -24 * want.abs().sum(0) + TINY[dtype])[None], "dbias")
    return dz, dgate, dbias


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_bias_gradient_keeps_float32(lib, dtype):
    """One z down each column and dy of one, so that a slope's error adds up.  gelu's slope is off by less than 2^-21 (4e-7 of
    a tail that is at most a half, and roundings of 2^-24 of numbers below 1.13), and the sum of m of them by less than
    m 2^-24 of it."""
    m, n = 4, 800
    z = torch.linspace(-4, 4, n).to(dtype)
    dbias = lib.activation_backward(torch.ones(m, n, dtype=dtype, device="cuda"), z.expand(m, n).contiguous().cuda(), "gelu",
                                    bias=True)[2].cpu().double()
    want = m * torch.from_numpy(F.activation(z.double().numpy(), "gelu")[1])
    off = (dbias - want).abs() - m * (2.0 ** -21 + 2.0 ** -24 * want.abs())
    assert off.max() < 0, (off.max(), z[off.argmax()])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("m,n", [(1, 1), (1, 7), (3, 8), (5, 100), (40, 2048), (333, 65), (129, 513), (700, 24), (64, 24576),
                                 (2500, 1030), (9000, 16)])
def test_backward_sizes(lib, m, n, dtype):
    check_backward(lib, m, n, DT[dtype], "silu", True, True)
    check_backward(lib, m, n, DT[dtype], "gelu", False, True, seed=4)
    check_backward(lib, m, n, DT[dtype], "gelu_tanh", False, False, seed=8)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("kind", F.ACTIVATIONS)
def test_backward_activations(lib, kind, dtype):
    for gate in (False, True):
        check_backward(lib, 70, 264, DT[dtype], kind, gate, True)
        for pad in ((8, 8), (5, 1)):
            check_backward(lib, 70, 264, DT[dtype], kind, gate, True, pad)


@pytest.mark.parametrize("dtype", list(DT))
def test_backward_in_place_and_again(lib, dtype):
    """Outputs in place of inputs, and a second call, give the same bits."""
    for m, n in ((3, 40), (300, 1000), (5000, 136)):
        dy, z, g = (rand(m, n, seed=i).to(DT[dtype]) for i in range(3))
        want = lib.activation_backward(dy, z, "gelu", g, True)
        again = lib.activation_backward(dy, z, "gelu", g, True)
        assert all(torch.equal(a, b) for a, b in zip(want, again))
        for outs in ((0, 1), (0, 2), (1, 2), (1, 0)):
            args = [dy.clone(), z.clone(), g.clone()]
            got = lib.activation_backward(args[0], args[1], "gelu", args[2], True, out=(args[outs[0]], args[outs[1]]))
            assert got[0] is args[outs[0]] and all(torch.equal(a, b) for a, b in zip(got, want))


def test_backward_empty(lib):
    e = torch.empty(0, 40, device="cuda", dtype=torch.bfloat16)
    dz, dgate, dbias = lib.activation_backward(e, e, "silu", e, True)
    assert dz.shape == dgate.shape == (0, 40) and torch.equal(dbias, torch.zeros(40, device="cuda"))
    e = torch.empty(5, 0, device="cuda")
    assert lib.activation_backward(e, e, None, None, True)[2].shape == (0,)


@pytest.mark.parametrize("kind", F.ACTIVATIONS[1:])
def test_backward_is_the_forward_differentiated(lib, kind):
    """dz and dgate against differences of the forward call's own float32 values (relu away from its corner).  The values
    carry 2^-20 of |act| < 6, over a step of 2^-4 2^-15.4 of it; the differences themselves are off by h^2/6 times a third
    derivative, which for these activations is below 2."""
    m, n, h = 4, 256, 2.0 ** -4
    x = torch.linspace(-4, 4, n, device="cuda")
    if kind == "relu":
        x = torch.where(x.abs() < 2 * h, 2.5 * h, x)
    a, b = torch.zeros(m, 16, device="cuda").to(F8[0]), torch.zeros(n, 16, device="cuda").to(F8[0])
    sa, sb = torch.ones(1, m, device="cuda"), torch.ones(2, 1, device="cuda")
    g, dy = rand(m, n, seed=1), rand(m, n, seed=2)

    def f(z):
        return lib.block128_linear(a, sa, b, sb, bias=z, activation=kind, gate=g, c_dtype=torch.float32).double()
    dz, dgate, _ = lib.activation_backward(dy, x.expand(m, n).contiguous(), kind, g)
    slope = dy.double() * (f(x + h) - f(x - h)) / (2 * h)
    scale = (dy * g).abs().double()
    close(dz, slope, scale * (2 * h * h / 6 + 6 * 2.0 ** -20 / h) + 1e-6, "dz")
    ratio = dy.double() * f(x) / g.double()
    close(dgate, ratio, ratio.abs() * 2.0 ** -18 + 1e-6, "dgate")


# --- rows in groups -------------------------------------------------------------------

def sizes_of(T, E, seed, empty=0.2):
    """Group sizes that add up to T, some of them zero."""
    rng = np.random.default_rng(seed)
    w = rng.exponential(1, E) * (rng.random(E) > empty)
    if w.sum() == 0:
        w[0] = 1
    return rng.multinomial(T, w / w.sum()).tolist()


def offsets_of(sizes, head=0, dtype=torch.int32):
    return torch.tensor([head] + (head + np.cumsum(sizes)).tolist(), dtype=dtype, device="cuda")


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("sizes,k,head,tail", [([1], 1, 0, 0), ([5], 128, 0, 0), ([0, 3, 0], 130, 2, 1), ([128, 128], 264, 0, 0),
                                               ([127, 129, 1], 96, 130, 5), ([300, 0, 0, 41, 128], 500, 0, 200),
                                               ([1] * 70, 40, 1, 3), ([0] * 5, 64, 3, 4), ([2] * 700 + [0] * 300, 24, 0, 0)])
def test_quantize_grouped_bit_exact(lib, sizes, k, head, tail, dtype):
    T = sum(sizes) + head + tail
    print(f"grouped quantise {sizes[:5]} x{len(sizes)} {k} {head} {tail}", flush=True)
    rng = np.random.default_rng(T + k)
    x = torch.from_numpy((rng.standard_normal((T, k)) * np.exp2(rng.integers(-4, 5, (T, k)))).astype(np.float32)).to(DT[dtype])
    for fmt in (0, 1):
        for rows in (True, False):
            off = offsets_of(sizes, head, torch.int64 if rows else torch.int32)
            pow2 = fmt == 1 and rows
            got = lib.block128_quantize(x.cuda(), fmt, rows=rows, cols=True, pow2=pow2, offsets=off)
            want = F.quantize_grouped(x.float().numpy(), off.tolist(), fmt, rows, pow2)
            for name, g, w in zip(("q", "s", "qt", "st"), got, want):
                assert (g is None) == (w is None)
                if g is None:
                    continue
                g = (g.view(torch.uint8) if name[0] == "q" else g).cpu().numpy()
                bad = np.argwhere(g != w)
                assert g.shape == w.shape and len(bad) == 0, f"{name}: {len(bad)} differ, first {bad[:4].tolist()}"


def test_quantize_grouped_of_one_group_is_the_plain_one(lib):
    x = rand(300, 520).bfloat16()
    q, s, qt, st = lib.block128_quantize(x, cols=True, offsets=offsets_of([300]))
    want = lib.block128_quantize(x, cols=True)
    assert torch.equal(q.view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(s, want[1]) and torch.equal(st, want[3])
    assert torch.equal(qt[:, :304].view(torch.uint8), want[2].view(torch.uint8)) and not qt[:, 304:].float().any()


def test_quantize_grouped_strided_and_given_outputs(lib):
    x = padded(rand(200, 136), 5, 1)
    off = offsets_of([50, 0, 120], 7)
    want = lib.block128_quantize(x.contiguous(), cols=True, offsets=off)
    for i, t in enumerate(want):
        assert torch.equal(lib.block128_quantize(x, cols=True, offsets=off)[i].view(torch.uint8), t.view(torch.uint8))
    out = tuple(torch.empty_like(t) for t in want)
    got = lib.block128_quantize(x, cols=True, offsets=off, out=out)
    assert all(a is b and torch.equal(a.view(torch.uint8), t.view(torch.uint8)) for a, b, t in zip(got, out, want))


def check_grouped(lib, sizes, n, k, dtype, head=0, tail=0, kind=None, gate=False, preact=False, fa=0, fb=0, pad=None,
                  index=torch.int32, seed=0):
    T, E = sum(sizes) + head + tail, len(sizes)
    print(f"grouped {sizes[:6]} x{E} T {T} {n}x{k} {dtype} {kind} gate {gate} preact {preact} {fa}{fb} {pad} {head} {tail}", flush=True)
    a, sa, b, sb = operands(lib, T, n, k, fa, fb, seed, E)
    off = offsets_of(sizes, head, index)
    g = rand(T, n, seed=seed + 3).to(dtype) if gate else None
    c = None
    if pad:
        g = None if g is None else padded(g, *pad)
        c = padded(torch.full((T, n), 5, device="cuda", dtype=dtype), *pad)
    out = lib.block128_grouped_gemm(a, sa, b, sb, off, kind, g, preact, dtype, c)
    torch.cuda.synchronize()
    got, kept = out if preact else (out, None)
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[head:head + sum(sizes)] = False
    assert torch.all(got[rest] == (5 if pad else 0)), "rows of no group"
    if preact:
        assert torch.all(kept[rest] == 0), "kept rows of no group"
    if pad:
        whole = c._base
        assert torch.all(whole[:, :pad[1]] == 7) and torch.all(whole[:, pad[1] + n:] == 7), "a write beside the columns"
    lo = head
    for e, m in enumerate(sizes):
        if m:
            at = slice(lo, lo + m)
            x, w = wide(a[at], sa[:, at], 1), wide(b[e], sb[e], 128)
            (y, by), (z, bz) = ends(matmul(x, w), matmul(x.abs(), w.abs()), k, dtype, None, kind, None if g is None else g[at], None)
            close(got[at], y, by, f"y of group {e}")
            if preact:
                close(kept[at], z, bz, f"z of group {e}")
        lo += m
    return got


GROUPS = [([1], 24, 16, 0, 0), ([1] * 8, 200, 272, 0, 3), ([0, 1, 0, 0, 2, 0], 96, 2048, 2, 0), ([16, 17, 1], 520, 400, 0, 0),
          ([40, 3, 0, 90], 200, 272, 0, 5), (sizes_of(300, 4, 1), 500, 400, 10, 10), (sizes_of(1100, 4, 2), 2100, 144, 0, 0),
          (sizes_of(2100, 4, 3, 0), 2050, 272, 0, 7), (sizes_of(2100, 4, 4, 0), 4100, 144, 0, 0),
          (sizes_of(4200, 5, 5), 4096, 144, 9, 0), (sizes_of(900, 300, 6), 136, 144, 0, 0), ([1] * 1000 + [0] * 24, 40, 144, 0, 0)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("case", range(len(GROUPS)))
def test_grouped_sizes(lib, case, dtype):
    sizes, n, k, head, tail = GROUPS[case]
    check_grouped(lib, sizes, n, k, DT[dtype], head, tail)
    check_grouped(lib, sizes, n, k, DT[dtype], head, tail, "silu", True, True, index=torch.int64, seed=7)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("kind", F.ACTIVATIONS)
def test_grouped_options(lib, kind, dtype):
    for gate in (False, True):
        for preact in (False, True):
            check_grouped(lib, [3, 0, 9, 1], 104, 256, DT[dtype], 0, 2, kind, gate, preact)
            check_grouped(lib, [70, 0, 150], 264, 144, DT[dtype], 1, 0, kind, gate, preact)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("fa", (0, 1))
@pytest.mark.parametrize("fb", (0, 1))
def test_grouped_formats(lib, fa, fb, dtype):
    for case in (1, 3, 5, 6, 7, 9):
        sizes, n, k, head, tail = GROUPS[case]
        check_grouped(lib, sizes, n, k, DT[dtype], head, tail, fa=fa, fb=fb)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("pad", [(8, 8), (5, 1)])
def test_grouped_strides_and_alignment(lib, dtype, pad):
    for sizes, n in (([3, 0, 5], 104), ([70, 0, 150], 265), (sizes_of(4200, 5, 5), 4096)):
        check_grouped(lib, sizes, n, 144, DT[dtype], 4, 3, "gelu_tanh", True, True, pad=pad)


def test_grouped_of_one_group_is_the_linear_call(lib):
    for m, n, k in ((40, 264, 272), (600, 1000, 272)):
        a, sa, b, sb = operands(lib, m, n, k)
        g = rand(m, n).bfloat16()
        got = lib.block128_grouped_gemm(a, sa, b[None].contiguous(), sb[None].contiguous(), offsets_of([m]), "silu", g)
        want = lib.block128_linear(a, sa, b, sb, activation="silu", gate=g)
        assert torch.equal(got, want)


def test_grouped_without_groups_or_rows(lib):
    a, sa, b, sb = operands(lib, 6, 64, 128, groups=0)
    y, z = lib.block128_grouped_gemm(a, sa, b, sb, offsets_of([]), preact=True)
    assert y.shape == (6, 64) and not y.any() and not z.any()
    c = torch.ones(6, 64, device="cuda")
    assert lib.block128_grouped_gemm(a, sa, b, sb, offsets_of([]), c=c) is c and torch.all(c == 1)
    a, sa, b, sb = operands(lib, 0, 64, 128, groups=3)
    assert lib.block128_grouped_gemm(a, sa, b, sb, offsets_of([0, 0, 0])).shape == (0, 64)
    # rows, but all of them of no group
    for m in (6, 400):
        a, sa, b, sb = operands(lib, m, 64, 128, groups=3)
        assert not lib.block128_grouped_gemm(a, sa, b, sb, offsets_of([0, 0, 0], m // 2)).any()


def check_weight_gradient(lib, sizes, m, n, head=0, tail=0, fa=1, fb=0, pad=0, index=torch.int32, seed=0):
    T, E = sum(sizes) + head + tail, len(sizes)
    print(f"weight gradient {sizes[:6]} x{E} T {T} {m}x{n} {fa}{fb} pad {pad} {head} {tail}", flush=True)
    off = offsets_of(sizes, head, index)
    dy, x = rand(T, m, seed=seed), rand(T, n, seed=seed + 1)
    _, _, a, sa = lib.block128_quantize(dy, fa, rows=False, cols=True, offsets=off)
    _, _, b, sb = lib.block128_quantize(x, fb, rows=False, cols=True, offsets=off)
    c = None
    if pad:
        c = torch.full((E, m, n + pad), 7.0, device="cuda")[:, :, :n]
    got = lib.block128_grouped_weight_gradient(a, sa, b, sb, off, c)
    torch.cuda.synchronize()
    assert got.shape == (E, m, n) and got.dtype == torch.float32
    if pad:
        assert got is c and torch.all(c._base[:, :, n:] == 7), "a write beside the columns"
    base = rand(E, m, n, seed=seed + 2)
    added = lib.block128_grouped_weight_gradient(a, sa, b, sb, off, base.clone(), accumulate=True)
    at = 0
    for e, rows in enumerate(sizes):
        nb = -(-rows // 128)
        if rows == 0:
            assert not got[e].any() and torch.equal(added[e], base[e])
        else:
            p, q = wide(a[:, 128 * at:128 * (at + nb)], sa[at:at + nb], 1), wide(b[:, 128 * at:128 * (at + nb)], sb[at:at + nb], 1)
            want, S = matmul(p, q), matmul(p.abs(), q.abs())
            bound = (nb * 8 + 4 * nb + 4) * 2.0 ** -24 * S + 2.0 ** -126
            close(got[e], want, bound, f"group {e}")
            close(added[e], want + base[e].double(), bound + 2.0 ** -24 * (want + base[e].double()).abs(), f"added to, group {e}")
        at += nb
    return got


@pytest.mark.parametrize("sizes,m,n,head,tail", [([1], 8, 16, 0, 0), ([0, 5, 0], 100, 70, 1, 1), ([128, 127, 129], 130, 300, 0, 0),
                                                 (sizes_of(900, 4, 1), 200, 300, 0, 30), (sizes_of(900, 4, 2), 1000, 1000, 5, 0),
                                                 (sizes_of(1500, 4, 3), 2000, 2001, 0, 0), (sizes_of(3000, 6, 4), 4000, 2000, 0, 0),
                                                 (sizes_of(600, 250, 5), 40, 72, 0, 0), ([3] * 1024, 16, 24, 0, 0),
                                                 # few tiles: the blocks in parts, some of them empty
                                                 ([4000], 70, 130, 3, 0), ([3000, 0, 200, 1], 200, 101, 0, 0), ([5000, 700], 500, 300, 0, 9)])
def test_weight_gradient_sizes(lib, sizes, m, n, head, tail):
    check_weight_gradient(lib, sizes, m, n, head, tail)
    check_weight_gradient(lib, sizes, m, n, head, tail, pad=3, index=torch.int64, seed=5)


@pytest.mark.parametrize("fa", (0, 1))
@pytest.mark.parametrize("fb", (0, 1))
def test_weight_gradient_formats(lib, fa, fb):
    for case in ((([300, 0, 41], 72, 136)), (sizes_of(900, 4, 2), 1000, 1000), (sizes_of(1500, 4, 3), 2000, 2000)):
        check_weight_gradient(lib, *case, fa=fa, fb=fb)


def test_weight_gradient_without_rows(lib):
    e = torch.empty
    for blocks in (0, 2):
        off = torch.zeros(4, dtype=torch.int32, device="cuda")
        a, sa = torch.zeros(40, 128 * blocks, device="cuda").to(F8[0]), e(blocks, 40, device="cuda")
        got = lib.block128_grouped_weight_gradient(a, sa, a, sa, off)
        assert got.shape == (3, 40, 40) and not got.any()
        c = torch.ones(3, 40, 40, device="cuda")
        lib.block128_grouped_weight_gradient(a, sa, a, sa, off, c, accumulate=True)
        assert torch.all(c == 1)
    assert lib.block128_grouped_weight_gradient(a, sa, a, sa, torch.zeros(1, dtype=torch.int64, device="cuda")).shape == (0, 40, 40)
