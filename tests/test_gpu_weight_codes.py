"""The examples' weight codes on streams other than their own, and in captured graphs."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture
def torch():
    import torch
    torch.manual_seed(4)
    return torch


def layers(torch):
    """Each example's layer with a call of it that gives one tensor."""
    import attention_input
    import feed_forward
    x = torch.randn(40, 256, device="cuda").bfloat16()
    ends = torch.tensor([0, 15, 15, 38], device="cuda")
    dense, experts = feed_forward.FeedForward(256, 400), feed_forward.Experts(3, 256, 400)
    heads = attention_input.AttentionInput(256, 2, 1, 64, 64)
    return ((dense, lambda: dense(x)), (experts, lambda: experts(x, ends)), (heads, lambda: torch.cat(heads(x), 1)))


def change(torch, layer, by):
    with torch.no_grad():
        for p in layer.parameters():
            if p.dim() > 1:
                p.add_(by)


@pytest.mark.parametrize("which", [0, 1, 2])
def test_codes_on_another_stream(torch, which):
    """A call on one stream makes the codes behind a long chain of other work; one on another stream takes them right after."""
    layer, call = layers(torch)[which]
    busy = torch.randn(4096, 4096, device="cuda")
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.no_grad():
        call()
        change(torch, layer, 0.25)
        first = [p.clone() for p in layer.parameters()]
        torch.cuda.synchronize()
        with torch.cuda.stream(one):
            for _ in range(20):
                busy = busy @ busy
                busy /= busy.abs().max()
            call()
        with torch.cuda.stream(two):
            got = call()
            change(torch, layer, 0.5)
            again = call()
        torch.cuda.synchronize()
        assert torch.equal(again, call()) and not torch.equal(again, got)
        for p, w in zip(layer.parameters(), first):
            p.copy_(w)
        assert torch.equal(got, call())


@pytest.mark.parametrize("which", [0, 1, 2])
def test_graph_without_gradients_follows_requantised_weights(torch, which):
    layer, call = layers(torch)[which]
    with torch.no_grad():
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call()
        for by in (0.0, 0.25, -0.125):
            change(torch, layer, by)
            layer.requantise()
            graph.replay()
            got = out.clone()
            assert torch.equal(got, call())
            change(torch, layer, 0.5)
            want = call()
            graph.replay()
            assert torch.equal(out, want) and not torch.equal(out, got)


@pytest.mark.parametrize("which", [0, 1, 2])
def test_graph_of_a_call_with_gradients_makes_its_own_codes(torch, which):
    layer, call = layers(torch)[which]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call().detach()
    with torch.no_grad():
        for by in (0.0, 0.25, -0.125):
            change(torch, layer, by)
            graph.replay()
            got = out.clone()
            assert torch.equal(got, call())


@pytest.mark.parametrize("which", [0, 1, 2])
def test_capture_refuses_codes_that_are_not_up_to_date(torch, which):
    layer, call = layers(torch)[which]
    with torch.no_grad():
        want = call()
        change(torch, layer, 0.25)
        graph = torch.cuda.CUDAGraph()
        with pytest.raises(RuntimeError, match="before the capture"):
            with torch.cuda.graph(graph):
                call()
        got = call()
        assert not torch.equal(got, want)
        layer.requantise()
        assert torch.equal(got, call())
