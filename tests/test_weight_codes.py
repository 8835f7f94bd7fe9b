"""When the examples' layers make their weights' codes anew, with a stand-in for the quantiser (no GPU needed)."""

import copy
import os
import pickle
import sys
import threading

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture
def made(monkeypatch):
    """The weights that have been quantised, in order; a weight's codes are copies of it."""
    import block_scaled_precision_e4m3_amd as mx
    made = []

    def stand_in(w, square, cols, out=None):
        assert square and cols and out is None and not torch.is_grad_enabled()
        made.append(w)
        return tuple(w.detach().clone() for _ in range(4))
    monkeypatch.setattr(mx, "block128_quantize", stand_in)
    return made


def layer():
    import feed_forward
    return feed_forward.FeedForward(32, 48, device="cpu")


def current(of):
    """Whether the layer's codes are those of its weights as they are."""
    return all(torch.equal(c, w) for codes, w in zip(of.codes(), (of.gate, of.up, of.down)) for c in codes)


def new(like):
    return torch.randn(like.shape).bfloat16()


@torch.no_grad()
def in_place(of):
    of.up.mul_(2)


def step(of):
    of.down.grad = torch.ones_like(of.down)
    torch.optim.SGD(of.parameters(), lr=1.0).step()


def replaced(of):
    of.gate = torch.nn.Parameter(new(of.gate))


def other_data(of):
    of.gate.data = new(of.gate)


def other_data_twice(of):
    """The memory of the first may be the allocator's for the third."""
    for _ in range(2):
        of.gate.data = new(of.gate)


def same_memory_other_tensor(of):
    with torch.no_grad():
        of.gate.mul_(3)
    of.gate = torch.nn.Parameter(of.gate.data)  # torch's count of its changes starts from zero


def loaded(of):
    of.load_state_dict(layer().state_dict())


def assigned(of):
    of.load_state_dict(layer().state_dict(), assign=True)


def swapped(of):
    a, b = of.gate, of.up
    of.gate, of.up = b, a


@pytest.mark.parametrize("change", [in_place, step, replaced, other_data, other_data_twice, same_memory_other_tensor, loaded,
                                    assigned, swapped])
def test_codes_are_those_of_the_weights(made, change):
    torch.manual_seed(0)
    of = layer()
    assert current(of) and len(made) == 3
    assert current(of) and len(made) == 3
    change(of)
    assert current(of) and len(made) == 6
    assert current(of) and len(made) == 6


def test_codes_after_a_change_that_torch_does_not_count(made):
    torch.manual_seed(1)
    of = layer()
    assert current(of)
    of.gate.data.add_(1)
    of.requantise()
    assert current(of)


def test_codes_of_inference_tensors_are_not_kept(made):
    torch.manual_seed(2)
    with torch.inference_mode():
        of = layer()
        assert current(of)
        of.gate.mul_(2)
        assert current(of) and len(made) == 6
        of.requantise()


def test_codes_made_in_inference_mode_serve_a_backward_pass(made):
    of = layer()
    with torch.inference_mode():
        codes = of.codes()
    assert not any(t.is_inference() for c in codes for t in c)
    assert of.codes()[0][0] is codes[0][0]


def test_copies_make_their_own_codes(made):
    torch.manual_seed(3)
    of = layer()
    of.codes()
    for other in (copy.deepcopy(of), pickle.loads(pickle.dumps(of))):
        before = len(made)
        assert current(other) and len(made) == before + 3
        in_place(other)
        assert current(other) and current(of)


def test_threads_make_codes_once(made):
    of = layer()
    at_once = threading.Barrier(4)
    got = []

    def call():
        at_once.wait()
        got.append(of.codes())
    threads = [threading.Thread(target=call) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 4 and len(made) == 3 and all(g[0][0] is got[0][0][0] for g in got)


def test_a_failed_quantisation_leaves_no_codes(made, monkeypatch):
    import block_scaled_precision_e4m3_amd as mx
    of = layer()
    of.codes()
    in_place(of)
    works = mx.block128_quantize

    def fails(*args, **kwargs):
        raise RuntimeError("no")
    monkeypatch.setattr(mx, "block128_quantize", fails)
    with pytest.raises(RuntimeError, match="no"):
        of.codes()
    with pytest.raises(RuntimeError, match="no"):
        of.codes()
    monkeypatch.setattr(mx, "block128_quantize", works)
    assert current(of)
