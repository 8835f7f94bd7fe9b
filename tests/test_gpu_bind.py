"""The torch wrappers' short way into the library (_bind.so) against the way through their own checks: the same results,
on the current stream, and None for whatever the checks must judge."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import block_scaled_precision_e4m3_amd as lib
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    assert lib._torch().fast is not None, "_bind.so is not built"
    return lib


def same(a, b):
    assert (a is None) == (b is None)
    if a is not None:
        assert a.shape == b.shape and a.dtype == b.dtype
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.fixture
def slow(lib, monkeypatch):
    """Calls f through the wrapper's checks."""
    def call(f):
        with monkeypatch.context() as m:
            m.setattr(lib._torch(), "fast", None)
            return f()
    return call


def inputs():
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, device="cuda", generator=g)  # noqa: E731
    return r


@pytest.mark.parametrize("shape", [(5, 272), (3, 40, 144)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantize(lib, slow, shape, dtype):
    x = inputs()(*shape).to(dtype)
    for kw in ({}, {"cols": True}, {"rows": False, "cols": True}, {"square": True, "cols": True}, {"pow2": True, "fmt": 1}):
        for a, b in zip(lib._torch().fast.quantize(x, kw.get("fmt", 0), kw.get("rows", True), kw.get("cols", False),
                                                   kw.get("square", False), kw.get("pow2", False)),
                        slow(lambda: lib.block128_quantize(x, **kw))):
            same(a, b)


def test_gemm(lib, slow):
    r = inputs()
    for lead in ((), (2,)):
        for m in (3, 40, 300):
            a, sa, _, _ = lib.block128_quantize(r(*lead, m, 1296))
            for block in (1, 128):
                b, sb, _, _ = lib.block128_quantize(r(*lead, 200, 1296), square=block == 128)
                for dtype in (None, torch.float32, torch.float16):
                    same(lib._torch().fast.gemm(a, sa, b, sb, block, dtype, None, False),
                         slow(lambda: lib.block128_gemm(a, sa, b, sb, block, dtype)))
                wide = torch.zeros(*lead, m, 208, device="cuda")
                c = wide[..., :200]
                assert lib._torch().fast.gemm(a, sa, b, sb, block, None, c, 1) is c
                same(c, slow(lambda: lib.block128_gemm(a, sa, b, sb, block, torch.float32)))


def test_rope_and_norm(lib, slow):
    r = inputs()
    x = r(7, 12, 128).bfloat16()
    q, k = x[:, :8], x[:, 8:10]
    w, w32 = r(128).bfloat16(), r(128)
    cos, sin = lib.rope_table(30, 64)
    fast = lib._torch().fast
    for pos in (None, torch.arange(7, device="cuda") * 3, torch.arange(7, device="cuda", dtype=torch.int32)):
        for layout in ("half", "interleaved", "interleaved_to_half"):
            for t in (False, True):
                same(fast.rope(x, cos, sin, pos, layout, 64, t, None), slow(lambda: lib.rope(x, cos, sin, pos, layout, 64, t)))
            for wq, wk in ((w, w), (w32, w32)):
                for a, b in zip(fast.qk_norm_rope(q, k, wq, wk, cos, sin, pos, layout, 32, 1e-5),
                                slow(lambda: lib.qk_norm_rope(q, k, wq, wk, cos, sin, pos, 1e-5, layout, 32))):
                    same(a, b)
                for a, b in zip(fast.qk_norm_rope_backward(q, k, q, k, wq, wk, cos, sin, pos, layout, 0, 1e-6),
                                slow(lambda: lib.qk_norm_rope_backward(q, k, q, k, wq, wk, cos, sin, pos, layout=layout))):
                    same(a, b)
    y = x.clone()
    assert fast.rope(y, cos, sin, None, "half", 0, False, y) is y
    same(y, slow(lambda: lib.rope(x, cos, sin)))
    same(fast.qk_norm_rope(q, None, w, None, None, None, None, "half", 0, 1e-6)[0],
         slow(lambda: lib.qk_norm_rope(q, None, w, None))[0])


def test_leaves_the_rest_to_the_checks(lib):
    r = inputs()
    x = r(5, 3, 128)
    cos, sin = lib.rope_table(9, 64)
    f = lib._torch().fast
    for bad in (lambda: f.rope(x.cpu(), cos, sin, None, "half", 0, False, None), lambda: f.rope(x, cos, None, None, "half", 0, False, None),
                lambda: f.rope(x, cos, sin, None, "other", 0, False, None), lambda: f.rope(x, cos.cpu(), sin, None, "half", 0, False, None),
                lambda: f.rope(x.transpose(1, 2), cos, sin, None, "half", 0, False, None), lambda: f.rope(x[:, :, ::2], cos, sin, None, "half", 0, False, None),
                lambda: f.rope(x, cos, sin, torch.zeros(4, device="cuda"), "half", 0, False, None), lambda: f.rope(1, cos, sin, None, "half", 0, False, None),
                lambda: f.rope(x, cos, sin, None, "half", 0, False, x.half()), lambda: f.rope(x, cos, sin),
                lambda: f.quantize(x.double(), 0, True, False, False, False), lambda: f.quantize(x, 3, True, False, False, False),
                lambda: f.quantize(x, 0, False, False, False, False), lambda: f.quantize(x.transpose(1, 2), 0, True, False, False, False),
                lambda: f.gemm(x, x, x, x, 128, None, None, False),
                lambda: f.qk_norm_rope(x, x.half(), x[0, 0], x[0, 0], cos, sin, None, "half", 0, 1e-6),
                lambda: f.qk_norm_rope(x, x, x[0, 0, :64], x[0, 0], cos, sin, None, "half", 0, 1e-6),
                lambda: f.qk_norm_rope(x, x, x[0, 0], x[0, 0], cos, sin, None, "half", 0, "1")):
        assert bad() is None
    with pytest.raises(lib.MxgemmValueError):
        lib.rope(x, cos, sin, rot_offset=65)
    with pytest.raises(lib.MxgemmValueError):
        f.rope(x, cos, sin, None, "half", 65, False, None)
    assert f.rope(x, cos, sin, None, "half", 1 << 70, False, None) is None
    assert f.quantize(x, 1 << 32, True, False, False, False) is None


def test_current_stream(lib):
    """Calls follow torch's current stream: a long chain on another one is waited for by what comes after it there."""
    s = torch.cuda.Stream()
    x = torch.zeros(4096, 8, 128, device="cuda")
    cos, sin = lib.rope_table(4096, 128)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        y = x
        for _ in range(200):
            y = y + 1.0
        z = lib.rope(y, cos, sin)
    s.synchronize()
    same(z, lib.rope(y, cos, sin))
    assert torch.all(y == 200).item()
