"""The wrappers next to autograd: what they write into a caller's tensor is known to it."""

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


def test_results_written_into_tensors(lib):
    """What is written into a caller's tensor counts as a change."""
    cos, sin = lib.rope_table(9, 128)
    x, w = normal(9, 3, 128), normal(128)
    a, sa, _, _ = lib.block128_quantize(normal(9, 128))
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
