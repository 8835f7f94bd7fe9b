"""Rotary positions and the per-head norm on the GPU, forward and backward, against float64.

Tolerances, with mag the sum of the magnitudes of an output's terms and u the rounding of its type (2^-24, 2^-8,
2^-11; float16 subnormals 2^-25): a rotation multiplies twice and adds once, 3 2^-24 mag; the norm's sum of squares
of D features, its root and quotient and the two products before the rotation, (D/2 + 16) 2^-24 mag; the backward's
second sum over D as well, (3 D/2 + 32) 2^-24 mag; a weight gradient adds the terms of all R rows, (R + D/2 + 32)
2^-24 times the sum of their magnitudes."""

import numpy as np
import pytest
import torch

from oracle import rope_heads as R

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
LAYOUTS = ["half", "interleaved", "interleaved_to_half"]


@pytest.fixture(scope="module")
def lib():
    import block_scaled_precision_e4m3_amd as lib
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return lib


def normal(shape, seed, dtype):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape).astype(np.float32)).to(dtype)


def f64(t):
    return t.double().cpu().numpy()


def close(got, ref, mag, factor, dtype, where=""):
    got = f64(got)
    err = factor * 2.0 ** -24 * mag
    lim = err + U[dtype] * (np.abs(ref) + err) + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    bad = ~(np.abs(got - ref) <= lim)
    assert not bad.any(), f"{where}: {int(bad.sum())} of {bad.size} outside, first {np.argwhere(bad)[:4].tolist()}"


def view(full, heads, at=0):
    """`heads` heads of a wider (T, all, D) buffer."""
    return full[:, at:at + heads]


SHAPES = [(1, 1, 2, 2, 0), (5, 3, 64, 64, 0), (33, 8, 128, 128, 0), (4, 40, 128, 64, 0), (70, 5, 192, 64, 128),
          (9, 7, 96, 96, 0), (6, 2, 256, 32, 224), (3, 1, 1024, 512, 256), (11, 3, 80, 48, 16), (7, 5, 100, 34, 3),
          (2, 2, 1023, 6, 1), (5, 9, 33, 32, 1), (1000, 3, 128, 128, 0), (8, 33, 48, 16, 8), (3, 4, 512, 512, 0)]


@pytest.mark.parametrize("T,H,D,rot,off", SHAPES)
def test_rope(lib, T, H, D, rot, off):
    print(f"rope {T}x{H}x{D} rot {rot} at {off}", flush=True)
    rng = np.random.default_rng(T + D)
    rows = T + 11
    cos, sin = lib.rope_table(rows, rot, base=100.0)
    pos = rng.integers(0, rows, T)
    for i, layout in enumerate(LAYOUTS):
        for dtype in DT.values():
            x = normal((T, H, D), i, dtype).cuda()
            for transpose in (False, True):
                p = torch.from_numpy(pos.astype(np.int64 if transpose else np.int32)).cuda()
                y = lib.rope(x, cos, sin, p, layout, off, transpose)
                ref, mag = R.rotate(f64(x), f64(cos)[pos], f64(sin)[pos], layout, off, transpose)
                close(y, ref, mag, 3, dtype, f"{layout} {dtype} {transpose}")
                keep = np.r_[0:off, off + rot:D]
                assert torch.equal(y[..., keep], x[..., keep])
                x2 = x.clone()
                assert lib.rope(x2, cos, sin, p, layout, off, transpose, out=x2) is x2 and torch.equal(x2, y)
    y = lib.rope(x, cos, sin, layout="half", rot_offset=off)
    ref, mag = R.rotate(f64(x), f64(cos)[:T], f64(sin)[:T], "half", off)
    close(y, ref, mag, 3, x.dtype, "without positions")


@pytest.mark.parametrize("D,rot,off,pad", [(128, 64, 0, 0), (128, 128, 0, 8), (192, 64, 128, 1), (64, 64, 0, 3)])
def test_rope_strides(lib, D, rot, off, pad):
    """Heads of a wider projection output, in and out, with any spacing, and what lies between them untouched."""
    T, H = 21, 6
    cos, sin = lib.rope_table(T, rot)
    for dtype in DT.values():
        for start in (0, 1, 8):
            full = normal((T, H + 3, D + pad + start), 5, dtype).cuda()
            x = full[:, 2:2 + H, start:start + D]
            wide = torch.full((T, H + 4, D + pad + start), 7.0, dtype=dtype, device="cuda")
            out = wide[:, 1:1 + H, start:start + D]
            for layout in LAYOUTS:
                lib.rope(x, cos, sin, layout=layout, rot_offset=off, out=out)
                ref, mag = R.rotate(f64(x), f64(cos), f64(sin), layout, off)
                close(out, ref, mag, 3, dtype, layout)
            rest = wide.clone()
            rest[:, 1:1 + H, start:start + D] = 7.0
            assert torch.all(rest == 7.0).item()
            # token and head axes exchanged
            xt = full.transpose(0, 1)[:, :, start:start + D][:T]
            ct, st = lib.rope_table(xt.shape[0], rot)
            ref, mag = R.rotate(f64(xt), f64(ct), f64(st), "half", off)
            close(lib.rope(xt, ct, st, rot_offset=off), ref, mag, 3, dtype, "transposed")


def test_rope_positions_outside_the_table_and_non_finite_features(lib):
    cos, sin = lib.rope_table(10, 64)
    for D in (128, 65):
        x = normal((6, 3, D), 1, torch.bfloat16).cuda()
        for dt in (torch.int32, torch.int64):
            p = torch.tensor([0, 9, 10, -1, 2 ** 31 - 1, 3], dtype=dt, device="cuda")
            y = lib.rope(x, cos, sin, p)
            bad = torch.tensor([False, False, True, True, True, False])
            assert torch.equal(torch.isnan(y[..., :64]).all(-1).all(-1).cpu(), bad)
            assert torch.equal(torch.isnan(y[..., :64]).any(-1).any(-1).cpu(), bad)
            assert torch.equal(y[..., 64:], x[..., 64:])
        x[1, 1, 100 % D if D > 100 else 64] = float("inf")     # a copied feature
        x[2, 0, 5] = float("nan")
        y = lib.rope(x, cos, sin)
        assert torch.isinf(y[1, 1]).sum() == 1 and not torch.isnan(y[1]).any()
        assert torch.isnan(y[2, 0]).sum() == 2 and torch.isnan(y[2, 0, [5, 37]]).all()


def test_empty(lib):
    cos, sin = lib.rope_table(4, 8)
    w = torch.ones(16, device="cuda")
    for T, H in ((0, 3), (3, 0)):
        x = torch.zeros(T, H, 16, device="cuda")
        assert lib.rope(x, cos, sin).shape == x.shape
        assert lib.qk_norm_rope(x, x, w, w, cos, sin)[0].shape == x.shape
        dq, dk, dwq, dwk = lib.qk_norm_rope_backward(x, x, x, x, w, w, cos, sin)
        assert dq.shape == x.shape and not dwq.any() and not dwk.any()


def norm_case(lib, T, Hq, Hk, D, rot, off, layout, dtype, w_dtype, seed, wide=True):
    full = (1.5 * normal((T, Hq + 2 * Hk, D), seed, torch.float32)).to(dtype).cuda()
    q, k = view(full, Hq), view(full, Hk, Hq)
    if not wide:
        q, k = q.contiguous(), k.contiguous()
    wq, wk = (1 + 0.2 * normal((D,), seed + 1, torch.float32)).to(w_dtype).cuda(), normal((D,), seed + 2, w_dtype).cuda()
    cos, sin = lib.rope_table(T + 20, rot, base=100.0)
    pos = np.random.default_rng(seed).integers(0, T + 20, T)
    return q, k, wq, wk, cos, sin, torch.from_numpy(pos.astype(np.int32)).cuda(), f64(cos)[pos], f64(sin)[pos]


NORMS = [(1, 1, 1, 2, 2, 0), (3, 32, 8, 128, 128, 0), (65, 4, 2, 64, 32, 0), (17, 5, 1, 192, 64, 128), (9, 3, 3, 96, 96, 0),
         (5, 2, 1, 100, 30, 5), (4, 1, 2, 1024, 64, 0), (6, 9, 2, 80, 16, 64), (3, 2, 2, 33, 0, 0), (700, 6, 2, 128, 64, 0),
         (2, 1, 1, 1, 0, 0), (4, 3, 1, 256, 256, 0), (4, 20, 5, 512, 256, 256)]


@pytest.mark.parametrize("T,Hq,Hk,D,rot,off", NORMS)
def test_norm_forward_and_backward(lib, T, Hq, Hk, D, rot, off):
    print(f"norm {T}x({Hq}+{Hk})x{D} rot {rot} at {off}", flush=True)
    for i, layout in enumerate(LAYOUTS):
        for j, dtype in enumerate(DT.values()):
            w_dtype = torch.float32 if (i + j) % 2 else dtype
            q, k, wq, wk, cos, sin, pos, c, s = norm_case(lib, T, Hq, Hk, D, rot, off, layout, dtype, w_dtype, i)
            where = f"{layout} {dtype}"
            yq, yk = lib.qk_norm_rope(q, k, wq, wk, cos, sin, pos, 1e-5, layout, off)
            for y, x, w in ((yq, q, wq), (yk, k, wk)):
                ref, mag = R.norm_rotate(f64(x), f64(w), c, s, layout, off, 1e-5)
                close(y, ref, mag, D / 2 + 16, dtype, where)
            q2, k2 = q.clone(), k.clone()
            lib.qk_norm_rope(q2, k2, wq, wk, cos, sin, pos, 1e-5, layout, off, out=(q2, k2))
            assert torch.equal(q2, yq) and torch.equal(k2, yk)
            gq, gk = normal(tuple(q.shape), 7, dtype).cuda(), normal(tuple(k.shape), 8, dtype).cuda()
            back = lib.qk_norm_rope_backward(gq, gk, q, k, wq, wk, cos, sin, pos, 1e-5, layout, off)
            for dx, dw, g, x, w in ((back[0], back[2], gq, q, wq), (back[1], back[3], gk, k, wk)):
                ref, dref, mag, dmag = R.norm_rotate_backward(f64(g), f64(x), f64(w), c, s, layout, off, 1e-5)
                close(dx, ref, mag, 1.5 * D + 32, dtype, where + " dx")
                close(dw, dref, dmag, T * x.shape[1] + D / 2 + 32, torch.float32, where + " dw")
            again = lib.qk_norm_rope_backward(gq, gk, q, k, wq, wk, cos, sin, pos, 1e-5, layout, off, out=(gq, gk))
            for a, b in zip(again, back):
                assert torch.equal(a, b)
            assert again[0] is gq


def test_norm_without_keys_or_rotation(lib):
    q = normal((12, 5, 128), 1, torch.bfloat16).cuda()
    w = normal((128,), 2, torch.bfloat16).cuda()
    y, none = lib.qk_norm_rope(q, None, w, None)
    one = np.ones((12, 0))
    ref, mag = R.norm_rotate(f64(q), f64(w), one, one, "half")
    close(y, ref, mag, 128 / 2 + 16, q.dtype)
    g = normal((12, 5, 128), 3, torch.bfloat16).cuda()
    dq, dk, dwq, dwk = lib.qk_norm_rope_backward(g, None, q, None, w, None)
    assert none is None and dk is None and dwk is None
    ref, dref, mag, dmag = R.norm_rotate_backward(f64(g), f64(q), f64(w), one, one, "half")
    close(dq, ref, mag, 1.5 * 128 + 32, q.dtype)
    close(dwq, dref, dmag, 60 + 96, torch.float32)


def test_norm_of_zero_and_extreme_rows(lib):
    """A zero row stays zero through eps; infinities and NaN stay in their row."""
    for D in (128, 66):
        q = normal((4, 3, D), 1, torch.float32)
        q[0, 0] = 0
        q[1, 1] = 1e-20
        q[2, 2, 3] = float("inf")
        q[3, 0, 4] = float("nan")
        q = q.cuda()
        w = torch.ones(D, device="cuda")
        cos, sin = lib.rope_table(4, 32)
        y = lib.qk_norm_rope(q, q, w, w, cos, sin)[0]
        assert not y[0, 0].any() and torch.isfinite(y[1]).all()
        assert torch.isnan(y[2, 2]).any() and torch.isfinite(y[2, :2]).all()
        assert torch.isnan(y[3, 0]).all() and torch.isfinite(y[3, 1:]).all()
        g = torch.ones_like(q)
        dq = lib.qk_norm_rope_backward(g, g, q, q, w, w, cos, sin)[0]
        assert torch.isfinite(dq[:2]).all() and torch.isfinite(dq[2, :2]).all() and torch.isnan(dq[3, 0]).all()


def test_norm_strided_outputs_and_gradients(lib):
    T, Hq, Hk = 19, 4, 2
    for D, pad in ((128, 8), (64, 1), (192, 0)):
        for dtype in DT.values():
            q, k, wq, wk, cos, sin, pos, c, s = norm_case(lib, T, Hq, Hk, D, 64, 0, "half", dtype, dtype, 3)
            wide = torch.full((T, Hq + Hk + 1, D + pad), 3.0, dtype=dtype, device="cuda")
            oq, ok = wide[:, :Hq, :D], wide[:, Hq + 1:, :D]
            lib.qk_norm_rope(q, k, wq, wk, cos, sin, pos, out=(oq, ok))
            for y, x, w in ((oq, q, wq), (ok, k, wk)):
                ref, mag = R.norm_rotate(f64(x), f64(w), c, s, "half")
                close(y, ref, mag, D / 2 + 16, dtype)
            assert torch.all(wide[:, Hq] == 3).item()
            assert pad == 0 or torch.all(wide[:, :, D:] == 3).item()
            g = normal((T, Hq + Hk, D + pad), 9, dtype).cuda()
            gq, gk = g[:, :Hq, :D], g[:, Hq:, :D]
            want = lib.qk_norm_rope_backward(gq.contiguous(), gk.contiguous(), q.contiguous(), k.contiguous(), wq, wk, cos, sin, pos)
            got = lib.qk_norm_rope_backward(gq, gk, q, k, wq, wk, cos, sin, pos, out=(oq, ok))
            for dx, ref, mag in ((got[0], *R.norm_rotate_backward(f64(gq), f64(q), f64(wq), c, s, "half")[::2]),
                                 (got[1], *R.norm_rotate_backward(f64(gk), f64(k), f64(wk), c, s, "half")[::2])):
                close(dx, ref, mag, 1.5 * D + 32, dtype)
            close(want[0], *R.norm_rotate_backward(f64(gq), f64(q), f64(wq), c, s, "half")[::2], 1.5 * D + 32, dtype)


def test_gradients_are_differences_of_the_forward(lib):
    """Directional derivatives: with h = 2^-7 the difference quotient of the float32 forward is within the third
    derivative's h^2 (bounded by 40 for rows of unit scale) and the forward's rounding over h of the gradient's."""
    T, H, D, h = 6, 2, 64, 2.0 ** -7
    q, k, wq, wk, cos, sin, pos, _, _ = norm_case(lib, T, H, H, D, 32, 32, "half", torch.float32, torch.float32, 4)
    gq, gk = normal((T, H, D), 5, torch.float32).cuda(), normal((T, H, D), 6, torch.float32).cuda()
    args = (cos, sin, pos, 1e-6, "half", 32)

    def loss(q, k, wq, wk):
        yq, yk = lib.qk_norm_rope(q, k, wq, wk, *args)
        return (yq.double() * gq.double()).sum() + (yk.double() * gk.double()).sum()
    grads = lib.qk_norm_rope_backward(gq, gk, q, k, wq, wk, *args)
    scale = float(gq.double().norm() + gk.double().norm())
    for i, x in enumerate((q, k, wq, wk)):
        v = normal(tuple(x.shape), 20 + i, torch.float32).cuda()
        v /= v.norm()
        at = [q, k, wq, wk]
        at[i] = x + h * v
        up = loss(*at)
        at[i] = x - h * v
        down = loss(*at)
        got = float((up - down) / (2 * h))
        want = float((grads[i].double() * v.double()).sum())
        tol = 40 * h * h * scale + (D / 2 + 16) * 2.0 ** -24 * scale * 8 / h
        assert abs(got - want) <= tol, (i, got, want, tol)


def test_graphs_and_streams(lib):
    q, k, wq, wk, cos, sin, pos, _, _ = norm_case(lib, 50, 8, 2, 128, 128, 0, "half", torch.bfloat16, torch.bfloat16, 2)
    gq, gk = normal((50, 8, 128), 5, torch.bfloat16).cuda(), normal((50, 2, 128), 6, torch.bfloat16).cuda()
    want = (lib.rope(q, cos, sin, pos), *lib.qk_norm_rope(q, k, wq, wk, cos, sin, pos),
            *lib.qk_norm_rope_backward(gq, gk, q, k, wq, wk, cos, sin, pos))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = (lib.rope(q, cos, sin, pos), *lib.qk_norm_rope(q, k, wq, wk, cos, sin, pos),
               *lib.qk_norm_rope_backward(gq, gk, q, k, wq, wk, cos, sin, pos))
    for _ in range(3):
        for t in got:
            t.fill_(1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    there = lib.qk_norm_rope_backward(gq, gk, q, k, wq, wk, cos, sin, pos, stream=s)
    s.synchronize()
    for a, b in zip(there, want[3:]):
        assert torch.equal(a, b)


def test_offsets_past_32_bits(lib):
    """Tokens that lie more than 2^32 bytes apart, read and written in place."""
    stride = (1 << 31) + 64
    flat = torch.zeros(stride + 4 * 128, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(flat, (2, 3, 128), (stride, 128, 1))
    x.copy_(normal((2, 3, 128), 1, torch.bfloat16))
    cos, sin = lib.rope_table(2, 128)
    keep = x.clone()
    y = lib.rope(x, cos, sin, out=x)
    ref, mag = R.rotate(f64(keep), f64(cos), f64(sin), "half")
    close(y, ref, mag, 3, torch.bfloat16)


@pytest.mark.parametrize("D,pad,rot,off", [(128, 8, 64, 0), (64, 1, 64, 0), (192, 0, 64, 128), (128, 3, 128, 0), (100, 1, 30, 5)])
def test_strides_do_not_change_results(lib, D, pad, rot, off):
    """Heads of any spacing and alignment, in and out, go through the same arithmetic as contiguous ones: equal bits."""
    T, Hq, Hk = 19, 4, 2
    for dtype in DT.values():
        for layout in LAYOUTS:
            q, k, wq, wk, cos, sin, pos, _, _ = norm_case(lib, T, Hq, Hk, D, rot, off, layout, dtype, dtype, 3)
            args = (cos, sin, pos, 1e-6, layout, off)
            g = normal((T, Hq + Hk, D + pad), 9, dtype).cuda()
            gq, gk = g[:, :Hq, :D], g[:, Hq:, :D]
            qc, kc, gqc, gkc = (t.contiguous() for t in (q, k, gq, gk))
            wide = torch.full((T, Hq + Hk + 1, D + pad), 3.0, dtype=dtype, device="cuda")
            out = wide[:, :Hq, :D], wide[:, Hq + 1:, :D]
            lib.qk_norm_rope(q, k, wq, wk, *args, out=out)
            for a, b in zip(out, lib.qk_norm_rope(qc, kc, wq, wk, *args)):
                assert torch.equal(a, b)
            got = lib.qk_norm_rope_backward(gq, gk, q, k, wq, wk, *args, out=out)
            for a, b in zip(got, lib.qk_norm_rope_backward(gqc, gkc, qc, kc, wq, wk, *args)):
                assert torch.equal(a, b)
            for transpose in (False, True):
                lib.rope(gq, cos, sin, pos, layout, off, transpose, out=out[0])
                assert torch.equal(out[0], lib.rope(gqc, cos, sin, pos, layout, off, transpose))
