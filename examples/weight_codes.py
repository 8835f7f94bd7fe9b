"""Codes of a layer's weights, in both directions, kept from one call to the next.

A layer that multiplies by its weights' codes makes them once and again when the weights are no longer those: another
tensor in a weight's place, other memory behind it (``weight.data = t``, ``load_state_dict(assign=True)``, ``.to``), or a
change that torch counts (an optimiser's step, an in-place operation).  What torch does not count, an in-place operation on
``weight.data``, calls for ``make``.  Inference tensors, which have no such count, get new codes in every call.

Codes are made on the stream of the call that needs them; a call on another stream waits for that, and the memory of codes
that are replaced is not used again before it is through with them.

Captured into a graph, a call that may have a backward pass makes the codes inside the graph, so that every replay takes the
weights as they are.  One without (``torch.no_grad()``) takes the kept codes, which have to be up to date, and which are from
then on remade in place: after a change of the weights, ``make`` or another call brings them up to date for the next replay.
The layer has to live as long as the graph.
"""

import os
import sys
import threading
import weakref

import torch
from torch.multiprocessing.reductions import StorageWeakRef

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import block_scaled_precision_e4m3_amd as mx  # noqa: E402


class _Seen:
    """A weight as it was when its codes were made."""

    def __init__(self, w):
        # the weak reference to its memory keeps another one from being taken for it, not the memory
        self.tensor, self.storage = weakref.ref(w), StorageWeakRef(w.untyped_storage())
        self.at, self.changes, self.layout = w.data_ptr(), w._version, (w.shape, w.stride(), w.dtype)

    def is_still(self, w):
        return (self.tensor() is w and self.storage.cdata == w.untyped_storage()._cdata and self.at == w.data_ptr()
                and self.changes == w._version and self.layout == (w.shape, w.stride(), w.dtype))


class WeightCodes:
    """codes(*weights): for each weight what block128_quantize(weight, square=True, cols=True) gives."""

    def __init__(self):
        self.lock = threading.Lock()
        self.seen, self.kept = (), []
        self.captured, self.left_to_graphs = False, []
        self.stream = self.event = None

    def __deepcopy__(self, memo):
        return WeightCodes()

    def __reduce__(self):
        return WeightCodes, ()

    def __call__(self, *weights):
        capturing = weights[0].is_cuda and torch.cuda.is_current_stream_capturing()
        if any(w.is_inference() for w in weights) or (capturing and torch.is_grad_enabled()):
            return self._quantise(weights, [None] * len(weights))
        with self.lock:
            if len(self.seen) != len(weights) or not all(s.is_still(w) for s, w in zip(self.seen, weights)):
                if capturing:
                    raise RuntimeError("the weights' codes are not made or not up to date, and a graph would not keep them "
                                       "so: call the layer, or make its codes, before the capture")
                self._make(weights)
            elif weights[0].is_cuda:
                self._join(torch.cuda.current_stream(weights[0].device), capturing)
            self.captured |= capturing
            return list(self.kept)

    def make(self, *weights):
        """Makes the codes, whether the weights have changed or not."""
        if any(w.is_inference() for w in weights):
            return
        if weights[0].is_cuda and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("codes that are to be kept are not made inside a graph")
        with self.lock:
            self._make(weights)

    def _join(self, stream, capturing):
        """Lets a stream other than the codes' own read them."""
        if stream == self.stream:
            return
        if not capturing:  # a capture begins with the card at rest, and may not wait for what lies outside of it
            stream.wait_event(self.event)
        for t in self._tensors():
            t.record_stream(stream)

    def _tensors(self):
        return [t for codes in self.kept for t in codes]

    def _make(self, weights):
        old = [None] * len(weights)
        if self.captured:
            if len(self.seen) == len(weights) and all(s.layout == (w.shape, w.stride(), w.dtype) and k[0].device == w.device
                                                      for s, w, k in zip(self.seen, weights, self.kept)):
                old = self.kept
                self._join(torch.cuda.current_stream(weights[0].device), False)
            else:
                self.left_to_graphs.append(self.kept)
                self.captured = False
        self.seen = ()  # none, if the making fails
        self.kept = self._quantise(weights, old)
        if weights[0].is_cuda:
            self.stream = torch.cuda.current_stream(weights[0].device)
            self.event = self.stream.record_event()
        self.seen = tuple(_Seen(w) for w in weights)

    @staticmethod
    def _quantise(weights, out):
        # not as inference tensors, which no backward pass can keep
        with torch.inference_mode(False), torch.no_grad():
            return [mx.block128_quantize(w, square=True, cols=True, out=o) for w, o in zip(weights, out)]
