"""The example that runs the block-128 product, the norm and the rotary positions together, against float32 torch."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("sizes", [{}, dict(norm=False), dict(hidden=144, heads=5, kv_heads=5, head_dim=80, tokens=77, norm=False),
                                   dict(hidden=528, heads=3, kv_heads=1, head_dim=64, tokens=131),
                                   dict(hidden=256, heads=4, kv_heads=4, head_dim=192, tokens=5)])
def test_attention_input(sizes):
    """Each operand's codes are off by at most 1/16 of a value, in root mean square by no more than 1/16 / sqrt(3) (uniform
    rounding at the coarse end of a binade): two operands, independent, sqrt(2) of that, 0.051.  The gradients take the
    forward pass's error (through y, in the norm) besides their own two: sqrt(4), 0.073.  The weight gradients of the
    norms see y only; they are sums with both signs, for which nothing smaller than their largest term is promised, so
    they get the same bound times 2."""
    import attention_input
    for name, e in attention_input.check(**sizes).items():
        bound = 0.051 if name.split()[-1] in "qkv" else 0.073 if name in ("dx", "dweight") else 0.146
        assert e < bound, (name, e)


def test_expanded_gradients():
    """The gradients of a sum reach the layer as views of one number."""
    import torch

    import attention_input
    torch.manual_seed(2)
    layer = attention_input.AttentionInput(256, 2, 1, 64, 64)
    x = torch.randn(9, 256, device="cuda").bfloat16().requires_grad_()
    sum(o.sum() for o in layer(x)).backward()
    got = x.grad.clone()
    x.grad = None
    out = layer(x)
    torch.autograd.backward(out, [torch.ones_like(o) for o in out])
    assert torch.equal(got, x.grad)


def test_decode_step_in_a_graph():
    """A decode step captured once and replayed, with other work between the replays, gives the eager results."""
    import torch

    import attention_input
    torch.manual_seed(1)
    layer = attention_input.AttentionInput(512, 4, 2, 64, 128)
    x = torch.randn(2, 512, device="cuda").bfloat16()
    at = torch.tensor([3, 70], device="cuda")
    with torch.no_grad():
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            layer(x, at)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = layer(x, at)
        for step in range(4):
            x.copy_(torch.randn(2, 512, device="cuda"))
            at.add_(1)
            want = layer(x, at)
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, want):
                assert torch.equal(a, b)


def test_codes_follow_the_weight():
    """After an optimiser's step, and after load_state_dict, the layer gives what a layer made of those weights gives."""
    import torch

    import attention_input
    torch.manual_seed(3)
    layer, other = (attention_input.AttentionInput(256, 2, 1, 64, 64) for _ in range(2))
    x = torch.randn(9, 256, device="cuda").bfloat16()
    step = torch.optim.SGD(layer.parameters(), lr=0.5)
    before = layer(x)
    sum(o.float().square().sum() for o in before).backward()
    step.step()
    got = layer(x)
    assert not torch.equal(got[2], before[2])
    other.load_state_dict(layer.state_dict())
    with torch.no_grad():
        for a, b in zip(got, other(x)):
            assert torch.equal(a, b)
        layer.requantise()
        for a, b in zip(got, layer(x)):
            assert torch.equal(a, b)


def test_a_layer_of_inference_tensors():
    import torch

    import attention_input
    with torch.inference_mode():
        layer = attention_input.AttentionInput(256, 2, 1, 64, 64)
        x = torch.randn(9, 256, device="cuda").bfloat16()
        for a, b in zip(layer(x), layer(x)):
            assert torch.equal(a, b)


def test_positions_changed_between_the_passes():
    """autograd notices, as for any tensor that a backward pass needs."""
    import torch

    import attention_input
    layer = attention_input.AttentionInput(256, 2, 1, 64, 64)
    x, at = torch.randn(9, 256, device="cuda").bfloat16(), torch.arange(9, device="cuda")
    out = layer(x, at)
    at.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out[0].sum().backward()
