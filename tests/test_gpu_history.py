"""What the wrappers refuse because its gradient or tangent would be lost, on the GPU: there the short way comes first."""

import pytest
import torch
import torch.autograd.forward_ad as forward

from test_history_host import FOLLOWED, calls, refuses

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    import block_scaled_precision_e4m3_amd as lib
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return lib


@pytest.mark.parametrize("which,name", FOLLOWED)
def test_followed_inputs(lib, which, name):
    f, args = calls(lib, "cuda")[which]
    f(**args)
    plain = args[name]
    args[name] = plain.clone().requires_grad_()
    assert refuses(lib, f, args)
    with torch.no_grad():
        f(**args)
    with forward.dual_level():
        args[name] = forward.make_dual(plain.clone(), torch.ones_like(plain))
        assert refuses(lib, f, args)
        with torch.no_grad():
            assert refuses(lib, f, args)
        args[name] = forward.unpack_dual(args[name]).primal
        f(**args)


def test_rotation_and_norm_of_dual_tensors(lib):
    """They have gradients of their own but no tangents, which torch says."""
    f, args = calls(lib, "cuda")["rope"]
    x, cos, sin = args["x"], args["cos"], args["sin"]
    w = torch.ones(64, device="cuda")
    with forward.dual_level():
        dual = forward.make_dual(x, torch.ones_like(x))
        with pytest.raises(NotImplementedError, match="jvp"):
            lib.rope(dual, cos, sin)
        with pytest.raises(NotImplementedError, match="jvp"):
            lib.qk_norm_rope(dual, None, w, None, cos, sin)
        assert torch.equal(lib.rope(x, cos, sin), x)


def test_layer_of_a_dual_tensor(lib):
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import feed_forward
    layer = feed_forward.FeedForward(64, 128)
    x = torch.randn(5, 64, device="cuda").bfloat16()
    with forward.dual_level():
        dual = forward.make_dual(x, torch.ones_like(x))
        with pytest.raises(NotImplementedError, match="jvp"):
            layer(dual)
        with torch.no_grad(), pytest.raises(lib.MxgemmError):
            layer(dual)
