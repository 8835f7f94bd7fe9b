"""Calls on another stream than the current one, while that one still has work queued on memory which Python has freed:
new outputs and workspaces must not lie there."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import block_scaled_precision_e4m3_amd as lib
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return lib


def normal(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def nbytes(t):
    return t.numel() * t.element_size()


def raw(t):
    return t.contiguous().reshape(-1).view(torch.uint8)


def check(call, scratch=()):
    """call(stream=s) gives what it gives on the current stream, and work that was queued before it keeps its memory.

    The current stream has some milliseconds of work (additions on 256 MB) and then fills buffers that have been freed by
    then, of the sizes of call's outputs and of `scratch`; what they were filled with is read back from them."""
    want = [t.clone() for t in call() if t is not None]
    sizes = [nbytes(t) for t in want] + list(scratch)
    busy = torch.zeros(1 << 26, device="cuda")
    for handle in (False, True):
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        # reserved here, so that the calls that follow allocate without waiting for the card
        del [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes][:]
        kept = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
        for _ in range(60):
            busy.add_(1)
        buffers = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
        for b, k in zip(buffers, kept):
            b.fill_(0x5A)
            for _ in range(3):
                busy.add_(1)
            k.copy_(b)
        del b, buffers
        got = call(stream=s.cuda_stream if handle else s)
        s.synchronize()
        torch.cuda.synchronize()
        for g, w in zip([t for t in got if t is not None], want):
            assert torch.equal(raw(g), raw(w))
        for k in kept:
            assert torch.all(k == 0x5A).item()
        # and when they are freed while the current stream still reads them, the next call there leaves them alone
        for _ in range(60):
            busy.add_(1)
        copies = [g.clone() for g in got if g is not None]
        del g, got
        again = call(stream=s)
        torch.cuda.synchronize()
        for c, w in zip(copies, want):
            assert torch.equal(raw(c), raw(w))
        del again


def test_quantize(lib):
    x = normal(1000, 2048).bfloat16()
    check(lambda **kw: lib.block128_quantize(x, cols=True, **kw))


@pytest.mark.parametrize("m,n,k", [(1000, 1024, 512), (64, 512, 7168)])
def test_product(lib, m, n, k):
    a, sa, _, _ = lib.block128_quantize(normal(m, k))
    b, sb, _, _ = lib.block128_quantize(normal(n, k, seed=1), square=True)
    need = lib._lib.mxgemm_block128_workspace_bytes(m, n, k, 1, lib.MXG_DT_BF16)
    assert (need > 0) == (m == 64)
    check(lambda **kw: (lib.block128_gemm(a, sa, b, sb, **kw),), [need] if need else [])


def test_rope(lib):
    x = normal(1000, 8, 128).bfloat16()
    cos, sin = lib.rope_table(1000, 128)
    check(lambda **kw: (lib.rope(x, cos, sin, **kw),))


def test_norm_and_backward(lib):
    q, k, w = normal(1000, 8, 128).bfloat16(), normal(1000, 2, 128, seed=1).bfloat16(), normal(128, seed=2).bfloat16()
    cos, sin = lib.rope_table(1000, 128)
    check(lambda **kw: lib.qk_norm_rope(q, k, w, w, cos, sin, **kw))
    need = lib._lib.mxgemm_qk_norm_rope_backward_workspace_bytes(1000, 128)
    check(lambda **kw: lib.qk_norm_rope_backward(q, k, q, k, w, w, cos, sin, **kw), [need])


def test_default_stream_by_its_handle(lib):
    """0 is the default stream's handle, also where another one is current."""
    x = normal(100, 8, 128).bfloat16()
    cos, sin = lib.rope_table(100, 128)
    want = lib.rope(x, cos, sin)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = lib.rope(x, cos, sin, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_mx_quantize_and_gemm_amax(lib):
    M, N, K = 512, 768, 1024
    x, w = normal(M, K), normal(N, K, seed=1)
    check(lambda **kw: lib.mx_quantize(x, **kw))
    (a, sfa), (b, sfb) = lib.mx_quantize(x), lib.mx_quantize(w)
    a, b = a.view(torch.float8_e4m3fn), b.view(torch.float8_e4m3fn)
    check(lambda **kw: lib.gemm_amax(a, b, sfa, sfb, **kw))
    check(lambda **kw: lib.gemm_amax(a, b, sfa, sfb, c_major="m", accumulate=True, **kw))
    rowwise = torch.randint(120, 130, (M, K // 32), dtype=torch.uint8, device="cuda")
    check(lambda **kw: (lib.sf_from_rowwise(rowwise, K, **kw),))


def test_projection(lib):
    tokens, heads, d, qr, K = 256, 4, 192, 64, 512
    code = lambda *s: torch.randint(0, 120, s, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)  # noqa: E731
    scale = lambda *s: torch.randint(120, 130, s, dtype=torch.uint8, device="cuda")  # noqa: E731
    x, w, xs, ws = code(tokens, K), code(heads * d, K), scale(tokens, K // 32), scale(heads * d, K // 32)
    cos, sin = normal(tokens, qr).bfloat16(), normal(tokens, qr, seed=1).bfloat16()
    need = lib._lib.mxgemm_projection_workspace_bytes(tokens, heads, d, K)
    check(lambda **kw: lib.projection_mxfp8(x, w, xs, ws, cos, sin, heads, d, qr, **kw), [need])
    check(lambda **kw: lib.projection_mxfp8_noalloc(x, w, xs, ws, cos, sin, heads, d, qr, **kw))
    sfa, sfb = lib.sf_from_rowwise(xs, K), lib.sf_from_rowwise(ws, K)
    check(lambda **kw: lib.gemm_rope_mxfp8(x, w, sfa, sfb, cos, sin, tokens, heads, d, qr, K, **kw))
    y = normal(tokens, heads * d)
    check(lambda **kw: lib.proj_rope_mxfp8(y, cos, sin, heads, d, qr, **kw))
