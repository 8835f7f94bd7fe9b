"""What the wrappers refuse because its gradient or tangent would be lost, before any device work (no GPU needed)."""

import os

import pytest
import torch
import torch.autograd.forward_ad as forward

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F8 = torch.float8_e4m3fn
SCALES = ("sa", "sb")


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    if not os.path.exists(os.path.join(ROOT, "block_scaled_precision_e4m3_amd", "libmxgemm.so")):
        __graft_entry__.build()
    import block_scaled_precision_e4m3_amd as lib
    return lib


def calls(lib, device="cpu"):
    """Name -> (call, its arguments by name); every float one of them may be followed by autograd."""
    def zeros(*shape, dtype=torch.float32):
        return torch.zeros(*shape, device=device).to(dtype)
    m, n, k, groups = 16, 32, 128, 2
    bf = torch.bfloat16
    offsets = torch.tensor([0, 10, 16], device=device)
    a, b = zeros(m, k, dtype=F8), zeros(n, k, dtype=F8)
    linear = dict(a=a, sa=zeros(1, m), b=b, sb=zeros(1, 1), bias=zeros(n), gate=zeros(m, n, dtype=bf), residual=zeros(m, n, dtype=bf),
                  c=zeros(m, n, dtype=bf))
    grouped = dict(a=a, sa=zeros(1, m), b=zeros(groups, n, k, dtype=F8), sb=zeros(groups, 1, 1), offsets=offsets,
                   gate=zeros(m, n, dtype=bf), c=zeros(m, n, dtype=bf))
    deep = dict(a=zeros(m, 2 * 128, dtype=F8), sa=zeros(2, m), b=zeros(n, 2 * 128, dtype=F8), sb=zeros(2, n), offsets=offsets,
                c=zeros(groups, m, n))
    back = dict(dy=zeros(m, n), z=zeros(m, n), gate=zeros(m, n))
    heads = dict(x=zeros(m, 2, 64), cos=zeros(m, 32), sin=zeros(m, 32))
    return {"linear": (lib.block128_linear, linear), "grouped": (lib.block128_grouped_gemm, grouped),
            "weight_gradient": (lib.block128_grouped_weight_gradient, deep), "backward": (lib.activation_backward, back),
            "rope": (lib.rope, heads)}


FOLLOWED = [("linear", name) for name in ("sa", "sb", "bias", "gate", "residual", "c")]
FOLLOWED += [("grouped", name) for name in ("sa", "sb", "gate", "c")] + [("weight_gradient", name) for name in ("sa", "sb", "c")]
FOLLOWED += [("backward", name) for name in ("dy", "z", "gate")]


def refuses(lib, f, args):
    with pytest.raises(lib.MxgemmError) as e:
        f(**args)
    return e.value.status == lib.MXG_ERR_FLAGS


@pytest.mark.parametrize("which,name", FOLLOWED)
def test_inputs_that_require_gradients(lib, which, name):
    f, args = calls(lib)[which]
    assert not refuses(lib, f, args)       # of the device: nothing here is on one
    args[name] = args[name].requires_grad_()
    assert refuses(lib, f, args)
    with torch.no_grad():
        assert not refuses(lib, f, args)


@pytest.mark.parametrize("which,name", FOLLOWED)
def test_inputs_with_a_tangent(lib, which, name):
    f, args = calls(lib)[which]
    with forward.dual_level():
        assert not refuses(lib, f, args)
        args[name] = forward.make_dual(args[name], torch.ones_like(args[name]))
        assert refuses(lib, f, args)
        with torch.no_grad():              # does not end it
            assert refuses(lib, f, args)
        with forward._set_fwd_grad_enabled(False):
            assert not refuses(lib, f, args)
        args[name] = forward.unpack_dual(args[name]).primal
        assert not refuses(lib, f, args)


def test_rotation_of_a_dual_tensor(lib):
    """It has a gradient of its own, which torch asks for."""
    f, args = calls(lib)["rope"]
    with forward.dual_level():
        args["out"] = torch.zeros_like(args["x"])
        args["x"] = forward.make_dual(args["x"], torch.ones_like(args["x"]))
        assert refuses(lib, f, args)
