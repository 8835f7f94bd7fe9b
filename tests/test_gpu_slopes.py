"""Slopes of the activations and the bias' gradient to the last bits of float32, on the GPU against float64.

Bounds, h = 2^-24 (half a step of float32 relative to a value).  With u the sigmoid's argument, e = e^-u, s = 1 / (1 + e) and r = e s:
  e   is off by 2 h of the hardware's exponential, and by its argument's error: 3.2 h |u| of itself for what the hardware takes
      directly (the product with log2 of e, and that constant's 2^-26.2, which float32 results keep), and for gelu_tanh 3 h |u| more
      of u's own three roundings (a float32 result keeps them too while |u| < 80, but for h |u|);
  s   by that times r, h for 1 + e, and 2 h for the reciprocal (a division: h);
  r   by e's, s's, and h.
A slope s + z s r u' then is off by s times s' error and |z| s r u' times the errors of s and r, 4 h for u' (z^2, two
constants, a multiply-add) and 2 h for two products, and by h of itself, and by what float32 cannot hold of s: 2^-126 times its factors.  gelu's is off by 2^-21 (4e-7 of a tail that is at
most a half, and roundings of numbers below 1.13).  A sum of equal terms loses h of itself in every addition; the longest
chain of them is a lane's rows, the lanes of a column and the parts, of which 16 are added at a time.
"""

import numpy as np
import pytest
import torch

from oracle import feed_forward as F

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
H = 2.0 ** -24


@pytest.fixture(scope="module")
def lib():
    import block_scaled_precision_e4m3_amd as lib
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return lib


def slope_bound(z, kind, direct):
    """How far the slope at float64 z may be off."""
    slope = F.activation(z, kind)[1]
    if kind == "gelu":
        return np.full_like(z, 2.0 ** -21)
    if kind == "relu":
        return np.zeros_like(z)
    a = 2 * np.sqrt(2 / np.pi) if kind == "gelu_tanh" else 1.0
    u = a * (z + 0.044715 * z ** 3) if kind == "gelu_tanh" else z
    du = a * (1 + 3 * 0.044715 * z * z) if kind == "gelu_tanh" else np.ones_like(z)
    s, r = F.sigmoid(u), F.sigmoid(-u)
    own = np.where(direct | (np.abs(u) >= 80), 3.0, 1.0) if kind == "gelu_tanh" else 1.0
    of_e = 2 * H + np.abs(u) * H * ((3.2 if direct else 0) + own)
    of_s = of_e * r + 3 * H
    return s * of_s + np.abs(z) * s * r * du * (of_s + of_e + of_s + H + 6 * H) + H * np.abs(slope) + 2.0 ** -126 * (1 + np.abs(z) * du)


@pytest.mark.parametrize("kind", F.ACTIVATIONS[1:])
def test_float32_slopes(lib, kind):
    z = torch.linspace(-12, 12, 1 << 16)
    dz = lib.activation_backward(torch.ones(1, z.numel(), device="cuda"), z[None].cuda(), kind)[0][0].cpu().double().numpy()
    z = z.double().numpy()
    off, bound = np.abs(dz - F.activation(z, kind)[1]), slope_bound(z, kind, False)
    at = (off - bound).argmax()
    assert off[at] <= bound[at], (z[at], off[at], bound[at])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("kind", F.ACTIVATIONS[1:])
@pytest.mark.parametrize("m", [4, 256, 2500])
def test_bias_gradient_to_the_last_bits(lib, kind, m, dtype):
    """One z down each column and dy of one, so that the errors of a slope add up; 2500 rows are summed in many parts."""
    dtype, n = DT[dtype], 1600
    z = torch.linspace(-8, 8, n).to(dtype)
    assert (lib._lib.mxgemm_activation_backward_workspace_bytes(m, n) > 0) == (m == 2500)
    dbias = lib.activation_backward(torch.ones(m, n, dtype=dtype, device="cuda"), z.expand(m, n).contiguous().cuda(), kind,
                                    bias=True)[2].cpu().double().numpy()
    z = z.double().numpy()
    want = m * F.activation(z, kind)[1]
    # 4 to 256 rows: 64 lanes of a column with 4 rows each at most; 2500: 2 rows to a lane, 8 lanes, 157 parts
    chain = min(m, 4 + 64) if m <= 256 else 2 + 8 + 10 + 16
    off, bound = np.abs(dbias - want), m * slope_bound(z, kind, dtype != torch.float32) + chain * H * np.abs(want)
    at = (off - bound).argmax()
    assert off[at] <= bound[at], (z[at], off[at], bound[at])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("kind", F.ACTIVATIONS[1:])
def test_slopes_at_the_ends(lib, kind, dtype):
    """Where an exponential overflows or vanishes slopes are zero and one, and a NaN stays one (in relu's value: its slope is
    whether z is above zero)."""
    large = 6e4 if dtype == "f16" else 1e30
    z = torch.tensor([[-large, -1000.0, -100.0, 100.0, 1000.0, large, float("nan")]], device="cuda").to(DT[dtype])
    dz, dgate, _ = lib.activation_backward(torch.ones_like(z), z, kind, torch.ones_like(z))
    assert torch.equal(dz[0, :6].float(), torch.tensor([0.0, 0, 0, 1, 1, 1], device="cuda")) and bool(dz[0, 6].isnan()) == (kind != "relu")
    assert torch.equal(dgate[0, :6], z[0, :6].clamp(min=0)) and dgate[0, 6].isnan()
