"""rope and qk_norm_rope under autograd: their gradients are the backward entry points' and, in float32, those of the same
formula in torch; what they write into a caller's tensor is known to autograd."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import block_scaled_precision_e4m3_amd as lib
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return lib


def normal(*shape, seed=0, dtype=torch.float32):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def leaf(t):
    return t.detach().clone().requires_grad_()


def formula(x, w, cos, sin, eps=1e-6):
    """float64, pairs in halves over the whole head."""
    x = x.double()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.double()
    c, s = cos.double()[:len(x), None], sin.double()[:len(x), None]
    a, b = x.chunk(2, -1)
    return torch.cat((a * c - b * s, b * c + a * s), -1)


@pytest.mark.parametrize("layout", ["half", "interleaved", "interleaved_to_half"])
@pytest.mark.parametrize("transpose", [False, True])
def test_rope(lib, layout, transpose):
    cos, sin = lib.rope_table(50, 64)
    pos = torch.arange(9, device="cuda") * 5
    for dtype in (torch.float32, torch.bfloat16):
        x, g = leaf(normal(9, 3, 128, dtype=dtype)), normal(9, 3, 128, seed=1, dtype=dtype)
        y = lib.rope(x, cos, sin, pos, layout, 32, transpose)
        with torch.no_grad():
            assert y.requires_grad and torch.equal(y, lib.rope(x, cos, sin, pos, layout, 32, transpose))
        y.backward(g)
        assert torch.equal(x.grad, lib.rope(g, cos, sin, pos, layout, 32, not transpose))


def test_gradients_of_the_formula(lib):
    """Float32 sums of at most 2 D terms forward and 3 D back, for rows and gradients of unit size: 2^-24 (3 D + 32) of the
    magnitudes, below 8; a weight's gradient adds those of all heads and tokens, 4 2^-24 of 30 heads of those."""
    cos, sin = lib.rope_table(10, 64)
    q, k, wq, wk = leaf(normal(10, 3, 64)), leaf(normal(10, 2, 64, seed=1)), leaf(normal(64, seed=2)), leaf(normal(64, seed=3))
    gq, gk = normal(10, 3, 64, seed=4), normal(10, 2, 64, seed=5)
    tol = (3 * 64 + 32) * 2.0 ** -24 * 8
    yq, yk = lib.qk_norm_rope(q, k, wq, wk, cos, sin)
    got = torch.autograd.grad((yq, yk), (q, k, wq, wk), (gq, gk))
    ref = torch.autograd.grad((formula(q, wq, cos, sin), formula(k, wk, cos, sin)), (q, k, wq, wk), (gq.double(), gk.double()))
    for i, (a, b) in enumerate(zip(got, ref)):
        assert (a - b).abs().max() <= tol * (1 if i < 2 else 30)
    (got,), (ref,) = (torch.autograd.grad(f(q), q, gq.to(t)) for f, t in ((lambda x: lib.rope(x, cos, sin), torch.float32),
                                                                           (lambda x: formula(x, None, cos, sin), torch.float64)))
    assert (got - ref).abs().max() <= 3 * 2.0 ** -24 * 8


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_norm_is_the_backward_entry(lib, dtype):
    cos, sin = lib.rope_table(20, 32)
    qkv = leaf(normal(11, 7, 128, dtype=dtype))
    wq, wk = leaf(normal(128, seed=2, dtype=dtype)), leaf(normal(128, seed=3, dtype=dtype))
    gq, gk = normal(11, 4, 128, seed=4, dtype=dtype), normal(11, 2, 128, seed=5, dtype=dtype)
    how = dict(positions=None, eps=1e-5, layout="interleaved", rot_offset=96)
    q, k = qkv[:, :4], qkv[:, 4:6]             # views of a projection's output
    y = lib.qk_norm_rope(q, k, wq, wk, cos, sin, **how)
    torch.autograd.backward(y, (gq, gk))
    dq, dk, dwq, dwk = lib.qk_norm_rope_backward(gq, gk, q, k, wq, wk, cos, sin, **how)
    assert torch.equal(qkv.grad[:, :4], dq) and torch.equal(qkv.grad[:, 4:6], dk) and not qkv.grad[:, 6:].any()
    assert torch.equal(wq.grad, dwq.to(dtype)) and torch.equal(wk.grad, dwk.to(dtype))
    # no keys, only one output used, an expanded gradient, weights that need none
    x = leaf(normal(5, 2, 128, dtype=dtype))
    lib.qk_norm_rope(x, None, wq.detach(), None)[0].sum().backward()
    one = torch.ones(5, 2, 128, device="cuda", dtype=dtype)
    assert torch.equal(x.grad, lib.qk_norm_rope_backward(one, None, x.detach(), None, wq.detach(), None)[0])
    x.grad = None
    lib.qk_norm_rope(x, x.detach(), wq.detach(), wk.detach())[0].sum().backward()
    assert torch.equal(x.grad, lib.qk_norm_rope_backward(one, one, x.detach(), x.detach(), wq.detach(), wk.detach())[0])


def test_on_another_stream(lib):
    cos, sin = lib.rope_table(9, 128)
    x, s = leaf(normal(9, 3, 128)), torch.cuda.Stream()
    torch.cuda.synchronize()
    y = lib.rope(x, cos, sin, stream=s)
    s.synchronize()
    g = normal(9, 3, 128, seed=1)
    assert torch.equal(torch.autograd.grad(y, x, g)[0], lib.rope(g, cos, sin, transpose=True))


def test_results_written_into_tensors(lib):
    """A result in a given tensor has no history: refused where one is needed.  What is written counts as a change."""
    cos, sin = lib.rope_table(9, 128)
    x, w = normal(9, 3, 128), normal(128)
    leaf_x, leaf_w, out = leaf(x), leaf(w), torch.empty_like(x)
    a, sa, _, _ = lib.block128_quantize(normal(9, 128))
    for bad in (lambda: lib.rope(leaf_x, cos, sin, out=out), lambda: lib.rope(x, cos, sin, out=leaf_x),
                lambda: lib.qk_norm_rope(leaf_x, None, w, None, out=(out, None)),
                lambda: lib.qk_norm_rope(x, None, leaf_w, None, out=[out, None]),
                lambda: lib.block128_gemm(a, sa, a, sa, b_block=1, c=leaf(torch.empty(9, 9, device="cuda")))):
        with pytest.raises(lib.MxgemmValueError):
            bad()
        with torch.no_grad():
            bad()
    calls = (lambda t: lib.rope(t, cos, sin, out=t), lambda t: lib.qk_norm_rope(t, None, w, None, out=(t, None)),
             lambda t: lib.qk_norm_rope_backward(x, None, x, None, w, None, out=(t, None)),
             lambda t: lib.block128_gemm(a, sa, a, sa, b_block=1, c=t.view(-1)[:81].view(9, 9)),
             lambda t: lib.block128_quantize(x[:, 0], out=(torch.empty_like(a), t.view(-1)[:9].view(1, 9), None, None)))
    fast = lib._torch().fast
    for use in (fast, None):
        lib._torch().fast = use
        try:
            for call in calls:
                y = leaf(x).exp()              # keeps its result for the backward pass
                call(y.detach())
                with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                    y.sum().backward()
                with torch.inference_mode():
                    call(x.clone())
        finally:
            lib._torch().fast = fast
