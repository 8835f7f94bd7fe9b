"""The feed-forward half of a layer on 8-bit codes, dense or with experts, forward and back.

    u = x Wu^T,   h = silu(x Wg^T) * u,   y = h Wd^T (+ x for the dense layer)

    dense:    block128_quantize, block128_gemm and block128_linear with activation, gate and residual
    experts:  rows in order of their experts: block128_quantize(offsets=...), block128_grouped_gemm with activation and gate,
              block128_grouped_weight_gradient

The backward pass quantises a gradient once for both directions, goes through the gate and the activation with
activation_backward, and makes the weights' gradients in float32.

    python examples/feed_forward.py      a training step of both, checked against float32 torch
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import block_scaled_precision_e4m3_amd as mx  # noqa: E402
from weight_codes import WeightCodes  # noqa: E402


class _Weights(torch.nn.Module):
    """gate, up (..., inner, hidden) and down (..., hidden, inner), bfloat16, with their codes in both directions, kept while
    the weights stay what they are (weight_codes.py); requantise() after changes that torch does not count (through .data)."""

    def __init__(self, lead, hidden, inner, device):
        super().__init__()
        self.gate, self.up = (torch.nn.Parameter((torch.randn(*lead, inner, hidden, device=device) / hidden ** 0.5).bfloat16())
                              for _ in range(2))
        self.down = torch.nn.Parameter((torch.randn(*lead, hidden, inner, device=device) / inner ** 0.5).bfloat16())
        self.kept = WeightCodes()

    def codes(self):
        return self.kept(self.gate, self.up, self.down)

    def requantise(self):
        self.kept.make(self.gate, self.up, self.down)


class FeedForward(_Weights):
    """y (T, hidden) = x + the feed-forward of x (T, hidden), bfloat16; hidden and inner multiples of 16."""

    def __init__(self, hidden, inner, device="cuda"):
        super().__init__((), hidden, inner, device)

    def forward(self, x):
        if torch.is_grad_enabled():
            return _FeedForward.apply(x, self.gate, self.up, self.down, self.codes())
        (g, gs, _, _), (w, ws, _, _), (d, ds, _, _) = self.codes()
        xq, xs, _, _ = mx.block128_quantize(x)
        h = mx.block128_linear(xq, xs, g, gs, activation="silu", gate=mx.block128_gemm(xq, xs, w, ws))
        hq, hs, _, _ = mx.block128_quantize(h)
        return mx.block128_linear(hq, hs, d, ds, residual=x)


class _FeedForward(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, up, down, codes):
        (g, gs, gt, gts), (w, ws, wt, wts), (d, ds, dt, dts) = codes
        xq, xs, xqt, xst = mx.block128_quantize(x, cols=True)
        u = mx.block128_gemm(xq, xs, w, ws)
        h, z = mx.block128_linear(xq, xs, g, gs, activation="silu", gate=u, preact=True)
        hq, hs, hqt, hst = mx.block128_quantize(h, cols=True)
        ctx.save_for_backward(z, u, xqt, xst, hqt, hst, gt, gts, wt, wts, dt, dts)
        return mx.block128_linear(hq, hs, d, ds, residual=x)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        z, u, xqt, xst, hqt, hst, gt, gts, wt, wts, dt, dts = ctx.saved_tensors
        dy = dy.contiguous()
        q, s, qt, st = mx.block128_quantize(dy, cols=True)
        ddown = mx.block128_gemm(qt, st, hqt, hst, b_block=1, c_dtype=torch.float32)
        dz, du, _ = mx.activation_backward(mx.block128_gemm(q, s, dt, dts), z, "silu", u)
        q, s, qt, st = mx.block128_quantize(dz, cols=True)
        dgate = mx.block128_gemm(qt, st, xqt, xst, b_block=1, c_dtype=torch.float32)
        dx = mx.block128_linear(q, s, gt, gts, residual=dy)
        q, s, qt, st = mx.block128_quantize(du, cols=True)
        dup = mx.block128_gemm(qt, st, xqt, xst, b_block=1, c_dtype=torch.float32)
        dx = mx.block128_linear(q, s, wt, wts, residual=dx, c=dx)
        return dx, dgate.to(z.dtype), dup.to(z.dtype), ddown.to(z.dtype), None


class Experts(_Weights):
    """y (T, hidden) of rows x (T, hidden) in order of their experts: expert e has rows offsets[e] to offsets[e + 1] (int32 or
    int64 on the device).  Rows of no expert give zeros."""

    def __init__(self, experts, hidden, inner, device="cuda"):
        super().__init__((experts,), hidden, inner, device)

    def forward(self, x, offsets):
        if torch.is_grad_enabled():
            return _Experts.apply(x, self.gate, self.up, self.down, self.codes(), offsets)
        (g, gs, _, _), (w, ws, _, _), (d, ds, _, _) = self.codes()
        xq, xs, _, _ = mx.block128_quantize(x)
        h = mx.block128_grouped_gemm(xq, xs, g, gs, offsets, activation="silu",
                                     gate=mx.block128_grouped_gemm(xq, xs, w, ws, offsets))
        hq, hs, _, _ = mx.block128_quantize(h)
        return mx.block128_grouped_gemm(hq, hs, d, ds, offsets)


class _Experts(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, up, down, codes, offsets):
        (g, gs, gt, gts), (w, ws, wt, wts), (d, ds, dt, dts) = codes
        xq, xs, xqt, xst = mx.block128_quantize(x, cols=True, offsets=offsets)
        u = mx.block128_grouped_gemm(xq, xs, w, ws, offsets)
        h, z = mx.block128_grouped_gemm(xq, xs, g, gs, offsets, activation="silu", gate=u, preact=True)
        hq, hs, hqt, hst = mx.block128_quantize(h, cols=True, offsets=offsets)
        ctx.save_for_backward(z, u, xqt, xst, hqt, hst, gt, gts, wt, wts, dt, dts, offsets)
        return mx.block128_grouped_gemm(hq, hs, d, ds, offsets)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        z, u, xqt, xst, hqt, hst, gt, gts, wt, wts, dt, dts, offsets = ctx.saved_tensors
        q, s, qt, st = mx.block128_quantize(dy.contiguous(), cols=True, offsets=offsets)
        ddown = mx.block128_grouped_weight_gradient(qt, st, hqt, hst, offsets)
        dz, du, _ = mx.activation_backward(mx.block128_grouped_gemm(q, s, dt, dts, offsets), z, "silu", u)
        q, s, qt, st = mx.block128_quantize(dz, cols=True, offsets=offsets)
        dgate = mx.block128_grouped_weight_gradient(qt, st, xqt, xst, offsets)
        dx = mx.block128_grouped_gemm(q, s, gt, gts, offsets)
        q, s, qt, st = mx.block128_quantize(du, cols=True, offsets=offsets)
        dup = mx.block128_grouped_weight_gradient(qt, st, xqt, xst, offsets)
        dx += mx.block128_grouped_gemm(q, s, wt, wts, offsets)
        return dx, dgate.to(z.dtype), dup.to(z.dtype), ddown.to(z.dtype), None, None


def plain(x, gate, up, down):
    """The feed-forward of x in float32 torch."""
    return (torch.nn.functional.silu(x @ gate.t()) * (x @ up.t())) @ down.t()


def off(a, b):
    return ((a.detach().float() - b.detach()).norm() / b.detach().norm()).item()


def check(hidden=512, inner=1024, tokens=300, sizes=(100, 0, 3, 260, 129), behind=5, seed=0):
    """Relative errors (Frobenius) of a training step's outputs and gradients of both layers against float32 torch.  A
    product of two operands with 4 significant bits is off by about 1/28 (examples/attention_input.py); what has gone through
    three of them one after the other, by about 1/28 times the root of their number."""
    torch.manual_seed(seed)
    errors = {}
    layer = FeedForward(hidden, inner)
    x = torch.randn(tokens, hidden, device="cuda").bfloat16().requires_grad_()
    y = layer(x)
    dy = torch.randn_like(y)
    y.backward(dy)
    with torch.no_grad():
        served = layer(x)
    ref_in = [t.detach().float().requires_grad_() for t in (x, layer.gate, layer.up, layer.down)]
    ref = plain(*ref_in) + ref_in[0]
    ref.backward(dy.float())
    errors["dense y"] = off(y, ref)
    errors["dense served y"] = off(served, ref)
    for name, a, b in zip(("dx", "dgate", "dup", "ddown"), (x, layer.gate, layer.up, layer.down), ref_in):
        errors["dense " + name] = off(a.grad, b.grad)

    experts = Experts(len(sizes), hidden, inner)
    ends = torch.tensor([0, *sizes]).cumsum(0)
    T = int(ends[-1]) + behind
    x = torch.randn(T, hidden, device="cuda").bfloat16().requires_grad_()
    y = experts(x, ends.int().cuda())
    dy = torch.randn_like(y)
    y.backward(dy)
    with torch.no_grad():
        served = experts(x, ends.int().cuda())
    ref_in = [t.detach().float().requires_grad_() for t in (x, experts.gate, experts.up, experts.down)]
    parts = [plain(ref_in[0][a:b], *(w[e] for w in ref_in[1:])) for e, (a, b) in enumerate(zip(ends[:-1], ends[1:]))]
    ref = torch.cat(parts + [torch.zeros(behind, hidden, device="cuda")])
    ref.backward(dy.float())
    errors["experts y"] = off(y, ref)
    errors["experts served y"] = off(served, ref)
    for name, a, b in zip(("dx", "dgate", "dup", "ddown"), (x, experts.gate, experts.up, experts.down), ref_in):
        errors["experts " + name] = off(a.grad, b.grad)
    return errors


if __name__ == "__main__":
    for name, e in check().items():
        print(f"{name:16s} relative error {e:.4f}")
