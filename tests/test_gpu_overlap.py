"""Outputs of the products with what follows them and of the activation's gradients on their inputs: the same rows, other rows."""

import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def lib():
    import block_scaled_precision_e4m3_amd as lib
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return lib


def rand(*shape, seed=0):
    return torch.randn(*shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))


def operands(lib, m, n, k, groups=None):
    a, sa, _, _ = lib.block128_quantize(rand(m, k))
    lead = () if groups is None else (groups,)
    b, sb, _, _ = lib.block128_quantize(rand(*lead, n, k, seed=1) / k ** 0.5, square=True)
    return a, sa, b, sb


def shaped(buffer, m, n, ld, first=0):
    return torch.as_strided(buffer, (m, n), (ld, 1), first)


def refused(lib, call):
    with pytest.raises(lib.MxgemmValueError) as e:
        call()
    assert e.value.status == lib.MXG_ERR_SHAPE


# (64, 512, 7168) divides K in 16 bits and float32; (5, 300, 272) has few rows, (700, 520, 272) odd tile ends
SIZES = [(5, 300, 272), (64, 512, 7168), (700, 520, 272), (513, 333, 144), (1024, 2048, 256)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear_in_place(lib, m, n, k, dtype):
    dt = DT[dtype]
    operand = operands(lib, m, n, k)
    bias, gate, residual = (0.5 * rand(n, seed=2)).to(dt), rand(m, n, seed=3).to(dt), rand(m, n, seed=4).to(dt)
    for kind in ("silu", "gelu"):
        for g, r in ((gate, residual), (gate, None), (None, residual)):
            want, z = lib.block128_linear(*operand, bias, kind, g, r, preact=True, c_dtype=dt)
            for name in ("gate", "residual"):
                own = {"gate": g, "residual": r}
                if own[name] is None:
                    continue
                c = own[name] = own[name].clone()
                got, kept = lib.block128_linear(*operand, bias, kind, own["gate"], own["residual"], preact=True, c=c)
                assert got is c and torch.equal(c, want) and torch.equal(kept, z), (kind, name)
        # both at once
        want = lib.block128_linear(*operand, bias, kind, gate, gate, c_dtype=dt)
        c = gate.clone()
        assert torch.equal(lib.block128_linear(*operand, bias, kind, c, c, c=c), want)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("sizes,n,k", [((3, 0, 1, 2), 300, 272), ((100, 0, 300, 31), 520, 272), ((40, 17), 333, 144),
                                       ((700, 900), 2048, 256)])
def test_grouped_in_place(lib, sizes, n, k, dtype):
    dt, T = DT[dtype], sum(sizes) + 9
    operand = operands(lib, T, n, k, len(sizes))
    at = torch.tensor([0, *sizes]).cumsum(0).int().cuda()
    gate = rand(T, n, seed=3).to(dt)
    for kind in ("silu", "gelu"):
        want, z = lib.block128_grouped_gemm(*operand, at, kind, gate, preact=True, c_dtype=dt)
        c = gate.clone()
        got, kept = lib.block128_grouped_gemm(*operand, at, kind, c, preact=True, c=c)
        rows = sum(sizes)
        assert got is c and torch.equal(c[:rows], want[:rows]) and torch.equal(kept, z)
        assert torch.equal(c[rows:], gate[rows:])


@pytest.mark.parametrize("dtype", list(DT))
def test_halves_of_one_matrix(lib, dtype):
    """Rows side by side in one buffer lie between each other and not on each other."""
    m, n, k, dt = 300, 520, 272, DT[dtype]
    operand = operands(lib, m, n, k)
    both = rand(m, 3 * n, seed=5).to(dt)
    gate, residual, c = both[:, :n], both[:, n:2 * n], both[:, 2 * n:]
    want = lib.block128_linear(*operand, None, "silu", gate.contiguous(), residual.contiguous(), c_dtype=dt)
    assert torch.equal(lib.block128_linear(*operand, None, "silu", gate, residual, c=c), want)
    dy = rand(m, n, seed=6).to(dt)
    want = lib.activation_backward(dy, gate.contiguous(), "gelu", residual.contiguous())
    out = torch.empty(m, 2 * n, device="cuda", dtype=dt)
    lib.activation_backward(dy, gate, "gelu", residual, out=(out[:, :n], out[:, n:]))
    assert torch.equal(out[:, :n], want[0]) and torch.equal(out[:, n:], want[1])


def test_a_single_row_has_no_row_distance(lib):
    operand = operands(lib, 1, 64, 128)
    gate = rand(1, 64, seed=3).bfloat16()
    want = lib.block128_linear(*operand, None, "silu", gate)
    c = gate.clone()
    assert torch.equal(lib.block128_linear(*operand, None, "silu", shaped(c, 1, 64, 900), c=c), want)


def test_linear_refuses_other_rows(lib):
    m, n, k = 40, 64, 128
    operand = operands(lib, m, n, k)
    for stream in (None, torch.cuda.current_stream()):
        buffer = rand(4 * m * n, seed=7).bfloat16()
        before = buffer.clone()
        c = shaped(buffer, m, n, n)
        for other in (shaped(buffer, m, n, n, n), shaped(buffer, m, n, n, 8), shaped(buffer, m, n, 2 * n),
                      shaped(buffer, m, n, n, (m - 1) * n + n - 1), shaped(buffer, m, n, n + 8, 16)):
            refused(lib, lambda: lib.block128_linear(*operand, gate=other, c=c, stream=stream))
            refused(lib, lambda: lib.block128_linear(*operand, residual=other, c=c, stream=stream))
            refused(lib, lambda: lib.block128_linear(*operand, gate=other, residual=c, c=c, stream=stream))
        refused(lib, lambda: lib.block128_linear(*operand, bias=buffer[m * n - n:m * n], c=c, stream=stream))
        torch.cuda.synchronize()
        assert torch.equal(buffer, before)
    # the codes and scales themselves
    a, sa, b, sb = operands(lib, m, 32, k)
    refused(lib, lambda: lib.block128_linear(a, sa, b, sb, c=a.view(torch.bfloat16)[:, :32]))
    a, sa, b, sb = operands(lib, 1, 16, 4096)
    refused(lib, lambda: lib.block128_linear(a, sa, b, sb, c=sa.view(1, -1)[:, :16]))
    refused(lib, lambda: lib.block128_linear(a, sa, b, sb, c=sb[:, :16]))


def test_grouped_refuses_other_rows(lib):
    m, n, k = 40, 64, 128
    operand = operands(lib, m, n, k, 3)
    at = torch.tensor([0, 10, 10, 35], device="cuda", dtype=torch.int32)
    buffer = rand(4 * m * n, seed=7).bfloat16()
    before = buffer.clone()
    c = shaped(buffer, m, n, n)
    for other in (shaped(buffer, m, n, n, n), shaped(buffer, m, n, n, 8), shaped(buffer, m, n, 2 * n)):
        for stream in (None, torch.cuda.current_stream()):
            refused(lib, lambda: lib.block128_grouped_gemm(*operand, at, gate=other, c=c, stream=stream))
    assert torch.equal(buffer, before)


def test_kept_inputs_of_the_activation_are_their_own(lib):
    """The C entry points take preact from the caller."""
    m, n, k = 40, 64, 128
    a, sa, b, sb = operands(lib, m, n, k)
    buffer, bias = rand(4 * m * n, seed=7).bfloat16(), rand(n, seed=8)
    c = buffer[:m * n]
    at = torch.tensor([0, 10, 35], device="cuda", dtype=torch.int32)
    ab, sab = torch.stack((b, b)), torch.stack((sb, sb))

    def linear(z, gate=None, ldz=n):
        e = lib._Ends(bias.data_ptr(), gate, None, z, n, n, ldz, 2, 0)
        return lib._lib.mxgemm_block128_linear(a.data_ptr(), sa.data_ptr(), b.data_ptr(), sb.data_ptr(), c.data_ptr(), n, m, n, k,
                                               0, 0, 1, ctypes.byref(e), 0, None, 0, None)

    def grouped(z, gate=None, ldz=n):
        e = lib._Ends(None, gate, None, z, n, n, ldz, 2, 0)
        return lib._lib.mxgemm_block128_grouped(a.data_ptr(), sa.data_ptr(), ab.data_ptr(), sab.data_ptr(), at.data_ptr(),
                                                c.data_ptr(), n, m, 2, n, k, 0, 0, 1, ctypes.byref(e), 0, None)
    free = buffer[m * n:].data_ptr()
    for f in (linear, grouped):
        assert f(free) == lib.MXG_OK and f(free, free + 2 * m * n) == lib.MXG_OK
        assert f(c.data_ptr()) == lib.MXG_ERR_SHAPE
        assert f(free - 2) == lib.MXG_ERR_SHAPE
        assert f(free, free) == lib.MXG_ERR_SHAPE
        assert f(a.data_ptr()) == lib.MXG_ERR_SHAPE and f(sa.data_ptr()) == lib.MXG_ERR_SHAPE
    assert linear(bias.data_ptr()) == lib.MXG_ERR_SHAPE and grouped(at.data_ptr()) == lib.MXG_ERR_SHAPE
    torch.cuda.synchronize()


@pytest.mark.parametrize("m,n", [(300, 200), (20, 4096)])
def test_gradients_refuse_other_rows(lib, m, n):
    buffer = rand(6 * m * n, seed=9).bfloat16()
    dy, z, gate = (shaped(buffer, m, n, n, i * m * n) for i in range(3))
    dz, dgate = (shaped(buffer, m, n, n, i * m * n) for i in (3, 4))
    before = buffer.clone()
    for stream in (None, torch.cuda.current_stream()):
        def call(dz, dgate):
            return lib.activation_backward(dy, z, "silu", gate, True, (dz, dgate), stream=stream)
        for i in range(3):
            for other in (shaped(buffer, m, n, n, i * m * n + 1), shaped(buffer, m, n, n, i * m * n + n), shaped(buffer, m, n, 2 * n, i * m * n)):
                refused(lib, lambda: call(other, dgate))
                refused(lib, lambda: call(dz, other))
        for other in (shaped(buffer, m, n, n, 3 * m * n + 1), shaped(buffer, m, n, n, 4 * m * n - 1), dz):
            refused(lib, lambda: call(dz, other))
        assert torch.equal(buffer, before)
    want = lib.activation_backward(dy, z, "silu", gate, True)
    for a, b in ((0, 1), (1, 2), (2, 0), (3, 0)):
        buffer.copy_(before)
        out = [shaped(buffer, m, n, n, i * m * n) for i in (a, b)]
        got = lib.activation_backward(dy, z, "silu", gate, True, out)
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_gradients_refuse_sums_on_other_tensors(lib):
    """The C entry point takes dbias and its workspace from the caller; two outputs in one there too."""
    m, n = 2000, 64
    t = [rand(m, n, seed=i) for i in range(5)]
    need = lib._lib.mxgemm_activation_backward_workspace_bytes(m, n)
    assert need > 0
    ws, dbias = torch.empty(need, device="cuda", dtype=torch.uint8), torch.empty(n, device="cuda")

    def call(dz=t[3], dgate=t[4], dbias=dbias, ws=ws):
        return lib._lib.mxgemm_activation_backward(t[0].data_ptr(), t[1].data_ptr(), t[2].data_ptr(), dz.data_ptr(), dgate.data_ptr(),
                                                   dbias.data_ptr(), (ctypes.c_int64 * 5)(*[n] * 5), m, n, 2, 0, 0, ws.data_ptr(),
                                                   ws.numel() * ws.element_size(), None)
    assert call() == lib.MXG_OK
    assert call(dgate=t[3]) == lib.MXG_ERR_SHAPE
    for other in t:
        assert call(dbias=other[m - 1]) == lib.MXG_ERR_SHAPE and call(ws=other[4:]) == lib.MXG_ERR_SHAPE
    assert call(dbias=ws.view(torch.float32)[:n]) == lib.MXG_ERR_SHAPE
    torch.cuda.synchronize()


def test_weight_gradient_refuses_its_operands(lib):
    at = torch.tensor([0, 100, 228], device="cuda")
    _, _, a, sa = lib.block128_quantize(rand(228, 64), rows=False, cols=True, offsets=at)
    _, _, b, sb = lib.block128_quantize(rand(228, 16, seed=1), rows=False, cols=True, offsets=at)
    large = torch.empty(2 * 64 * 16 + sa.numel() + sb.numel(), device="cuda")
    c, tail = large[:2 * 64 * 16].view(2, 64, 16), large[2 * 64 * 16:]
    want = lib.block128_grouped_weight_gradient(a, sa, b, sb, at)
    scales = tail[:sa.numel()].view(sa.shape).copy_(sa)
    assert torch.equal(lib.block128_grouped_weight_gradient(a, scales, b, sb, at, c=c), want)
    scales = large[2 * 64 * 16 - 1:][:sa.numel()].view(sa.shape)
    refused(lib, lambda: lib.block128_grouped_weight_gradient(a, scales, b, sb, at, c=c))
    # b (N, 128 G) for an output (2, 64, 16) of the same bytes and more
    codes = torch.zeros(4 * c.numel(), device="cuda", dtype=torch.uint8)
    inside = codes[:b.numel()].view(b.shape).view(b.dtype)
    refused(lib, lambda: lib.block128_grouped_weight_gradient(a, sa, inside, sb, at, c=codes.view(torch.float32).view(2, 64, 16)))
