"""The input half of an attention layer on 8-bit codes: hidden states to the heads that attention takes, and back.

    x (T, hidden) -> codes in blocks of 1 x 128
                  -> product with the weight's codes (blocks of 128 x 128)      block128_quantize, block128_gemm
                  -> q, k: root-mean-square norm and rotary positions,          qk_norm_rope,
                     or only the positions; v as is                             rope

The backward pass turns the heads' gradients into the projection's (qk_norm_rope_backward, or rope's transpose), quantises those once for
both directions and runs two more products: the input's gradient over the weight's transposed codes, and the weight's
gradient, float32, over the tokens.

    python examples/attention_input.py      a training step and a decode step, checked against float32 torch
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import block_scaled_precision_e4m3_amd as mx  # noqa: E402
from weight_codes import WeightCodes  # noqa: E402


class AttentionInput(torch.nn.Module):
    """q (T, heads, D), k (T, kv_heads, D) and v (T, kv_heads, D) of hidden states x (T, hidden), bfloat16; norm: q and k
    are normed per head before the positions turn them.

    weight ((heads + 2 kv_heads) D, hidden) is kept in bfloat16 and in codes of both directions, kept while the weight stays
    what it is (weight_codes.py); requantise() after changes that torch does not count (through weight.data)."""

    def __init__(self, hidden, heads, kv_heads, head_dim, max_positions, rot=None, norm=True, eps=1e-6,
                 device="cuda"):
        super().__init__()
        self.heads, self.kv_heads, self.head_dim, self.eps = heads, kv_heads, head_dim, eps
        n = (heads + 2 * kv_heads) * head_dim
        self.weight = torch.nn.Parameter((torch.randn(n, hidden, device=device) / hidden ** 0.5).bfloat16())
        self.q_norm = torch.nn.Parameter(torch.ones(head_dim, device=device)) if norm else None
        self.k_norm = torch.nn.Parameter(torch.ones(head_dim, device=device)) if norm else None
        self.cos, self.sin = mx.rope_table(max_positions, rot or head_dim, device=device)
        self.kept = WeightCodes()
        self.requantise()

    @property
    def codes(self):
        return self.kept(self.weight)[0]

    def requantise(self):
        self.kept.make(self.weight)

    def split(self, y):
        """Views of the projection's output (T, (heads + 2 kv_heads) D)."""
        y = y.view(-1, self.heads + 2 * self.kv_heads, self.head_dim)
        return y.split((self.heads, self.kv_heads, self.kv_heads), 1)

    def positioned(self, q, k, positions):
        if self.q_norm is None:
            return mx.rope(q, self.cos, self.sin, positions), mx.rope(k, self.cos, self.sin, positions)
        return mx.qk_norm_rope(q, k, self.q_norm, self.k_norm, self.cos, self.sin, positions, eps=self.eps)

    def positioned_backward(self, dq, dk, q, k, q_norm, k_norm, positions, out):
        """Gradients of q and k into out; returns the norm weights'."""
        if q_norm is None:
            mx.rope(dq, self.cos, self.sin, positions, transpose=True, out=out[0])
            mx.rope(dk, self.cos, self.sin, positions, transpose=True, out=out[1])
            return None, None
        return mx.qk_norm_rope_backward(dq, dk, q, k, q_norm, k_norm, self.cos, self.sin, positions, eps=self.eps,
                                        out=out)[2:]

    def forward(self, x, positions=None):
        if torch.is_grad_enabled():
            return _AttentionInput.apply(x, self.weight, self.q_norm, self.k_norm, self, self.codes, positions)
        w, ws, _, _ = self.codes
        xq, xs, _, _ = mx.block128_quantize(x)
        q, k, v = self.split(mx.block128_gemm(xq, xs, w, ws))
        return *self.positioned(q, k, positions), v


class _AttentionInput(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, q_norm, k_norm, layer, codes, positions):
        w, ws, wt, wts = codes
        xq, xs, xqt, xst = mx.block128_quantize(x, cols=True)
        y = mx.block128_gemm(xq, xs, w, ws)
        q, k, v = layer.split(y)
        ctx.layer = layer
        ctx.save_for_backward(y, xqt, xst, q_norm, k_norm, wt, wts, positions)
        # a view of y may not leave: y is kept as it is for the backward pass
        return *layer.positioned(q, k, positions), v.clone()

    @staticmethod
    def backward(ctx, dq, dk, dv):
        layer = ctx.layer
        y, xqt, xst, q_norm, k_norm, wt, wts, positions = ctx.saved_tensors
        q, k, _ = layer.split(y)
        dq, dk = dq.contiguous(), dk.contiguous()  # an expanded gradient (of a sum) has no features side by side
        dy = torch.empty_like(y)
        gq, gk, gv = layer.split(dy)
        dqn, dkn = layer.positioned_backward(dq, dk, q, k, q_norm, k_norm, positions, (gq, gk))
        gv.copy_(dv)
        g, gs, gt, gts = mx.block128_quantize(dy, cols=True)
        dx = mx.block128_gemm(g, gs, wt, wts)
        dw = mx.block128_gemm(gt, gts, xqt, xst, b_block=1, c_dtype=torch.float32)
        return dx, dw.to(layer.weight.dtype), dqn, dkn, None, None, None


def plain(layer, x, weight, q_norm, k_norm, positions):
    """The same layer in float32 torch."""
    q, k, v = layer.split(x @ weight.t())
    rot = 2 * layer.cos.shape[1]
    p = torch.arange(len(x), device=x.device) if positions is None else positions
    c, s = layer.cos[p][:, None], layer.sin[p][:, None]

    def one(h, w):
        if w is not None:
            h = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + layer.eps) * w
        a, b = h[..., :rot // 2], h[..., rot // 2:rot]
        return torch.cat((a * c - b * s, b * c + a * s, h[..., rot:]), -1)
    return one(q, q_norm), one(k, k_norm), v


def check(hidden=1024, heads=8, kv_heads=2, head_dim=128, tokens=300, norm=True, seed=0):
    """Relative errors (Frobenius) of a training step's outputs and gradients, and of a decode step's outputs, against
    float32 torch.  The codes carry 4 significant bits (relative error at most 1/16 per value, about 1/40 in the mean
    square), so a product of two such operands is off by about 1/28."""
    torch.manual_seed(seed)
    layer = AttentionInput(hidden, heads, kv_heads, head_dim, 4096, norm=norm)
    x = torch.randn(tokens, hidden, device="cuda").bfloat16().requires_grad_()
    out = layer(x)
    grads = [torch.randn_like(o) for o in out]
    torch.autograd.backward(out, grads)
    mine = (x, layer.weight) + ((layer.q_norm, layer.k_norm) if norm else ())
    ref_in = [t.detach().float().requires_grad_() for t in mine] + ([] if norm else [None, None])
    ref = plain(layer, *ref_in, None)
    torch.autograd.backward(ref, [g.float() for g in grads])

    def off(a, b):
        return ((a.detach().float() - b.detach()).norm() / b.detach().norm()).item()
    errors = {n: off(a, b) for n, a, b in zip(("q", "k", "v"), out, ref)}
    errors.update({n: off(a.grad, b.grad) for n, a, b in zip(("dx", "dweight", "dq_norm", "dk_norm"), mine, ref_in)})
    at = torch.tensor([1000, 17, 4095], device="cuda")
    with torch.no_grad():
        step = layer(x[:3], at)
        ref = plain(layer, *[t if t is None else t.detach() for t in (ref_in[0][:3], *ref_in[1:])], at)
    errors.update({"decode " + n: off(a, b) for n, a, b in zip(("q", "k", "v"), step, ref)})
    return errors


if __name__ == "__main__":
    for name, e in check().items():
        print(f"{name:10s} relative error {e:.4f}")
