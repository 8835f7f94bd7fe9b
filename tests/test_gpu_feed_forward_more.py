"""Calls of the feed-forward products that the other tests leave out: strided outputs that are added to or are the gate, as many
groups and rows as there may be, values that are not finite where they do not count, divided products in graphs."""

import pytest
import torch

import feed_forward_paths as P
from test_gpu_feed_forward import DT, F8, check_grouped, lib, offsets_of, operands, padded, rand, sizes_of  # noqa: F401

pytestmark = pytest.mark.gpu
NAN = 0x7F  # of both code formats


def along_tokens(lib, T, m, n, off, fa=1, fb=0):  # noqa: F811
    _, _, a, sa = lib.block128_quantize(rand(T, m), fa, rows=False, cols=True, offsets=off)
    _, _, b, sb = lib.block128_quantize(rand(T, n, seed=1), fb, rows=False, cols=True, offsets=off)
    return a, sa, b, sb


def equal(x, y):
    return torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))


@pytest.mark.parametrize("sizes,m,n,head,tail", [([70, 0, 300], 72, 100, 0, 3), (sizes_of(900, 4, 2), 1000, 1001, 5, 0),
                                                 (sizes_of(1500, 4, 3), 2000, 2000, 0, 0)] + [c for c, _ in P.DEEP])
def test_weight_gradient_added_to_a_strided_output(lib, sizes, m, n, head, tail):  # noqa: F811
    off = offsets_of(sizes, head)
    operand = along_tokens(lib, sum(sizes) + head + tail, m, n, off)
    base = rand(len(sizes), m, n, seed=2)
    want = lib.block128_grouped_weight_gradient(*operand, off, base.clone(), accumulate=True)
    for pad in (8, 3):
        whole = torch.full((len(sizes), m, n + pad), 7.0, device="cuda")
        c = whole[:, :, :n]
        c.copy_(base)
        assert lib.block128_grouped_weight_gradient(*operand, off, c, accumulate=True) is c
        assert torch.equal(c, want) and torch.all(whole[:, :, n:] == 7)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("sizes,n,k", [([3, 0, 1, 2], 304, 272), ([100, 0, 300, 31], 520, 272), ([40, 17], 333, 144), ([700, 900], 2048, 256)])
def test_grouped_into_a_strided_gate(lib, sizes, n, k, dtype):  # noqa: F811
    T = sum(sizes) + 9
    operand, off = operands(lib, T, n, k, groups=len(sizes)), offsets_of(sizes, 4)
    gate = rand(T, n, seed=3).to(DT[dtype])
    want = lib.block128_grouped_gemm(*operand, off, "silu", gate, c_dtype=DT[dtype])
    for pad in ((8, 8), (5, 1)):
        c = padded(gate, *pad)
        assert lib.block128_grouped_gemm(*operand, off, "silu", c, c=c) is c
        assert torch.equal(c[4:-5], want[4:-5]) and torch.equal(c[:4], gate[:4]) and torch.equal(c[-5:], gate[-5:])
        whole = c._base
        assert torch.all(whole[:, :pad[1]] == 7) and torch.all(whole[:, pad[1] + n:] == 7)


@pytest.mark.parametrize("dtype", list(DT))
def test_as_many_groups_as_there_may_be(lib, dtype):  # noqa: F811
    sizes = [40 + e % 3 for e in range(1023)] + [0]
    check_grouped(lib, sizes, 72, 144, DT[dtype], 3, 2, "silu", True, True)


def test_as_many_rows_as_there_may_be(lib):  # noqa: F811
    T, k, n = 1 << 24, 16, 16
    sizes = [1, 0, (1 << 23) - 5, 1 << 22, (1 << 22) - 200, 3]
    head, off = 128, offsets_of(sizes, 128, torch.int64)
    assert head + sum(sizes) < T
    x = rand(1 << 12, k).bfloat16().repeat(T >> 12, 1)
    q, s, qt, st = lib.block128_quantize(x, cols=True, offsets=off)
    want = lib.block128_quantize(x[:1 << 12].contiguous())
    assert equal(q.view(-1, 1 << 12, k)[-1], want[0]) and equal(q.view(-1, 1 << 12, k)[777], want[0])
    assert torch.equal(s.view(T >> 12, 1 << 12), want[1].expand(T >> 12, 1 << 12))
    block = 0
    for e, rows in enumerate(sizes):
        for at in {0, rows // 2, rows - 1} if rows else ():
            first = at // 128 * 128
            part = x[off[e] + first:off[e] + min(first + 128, rows)]
            _, _, c, t = lib.block128_quantize(part, rows=False, cols=True)
            to = block + first // 128
            assert equal(qt[:, 128 * to:128 * to + c.shape[1]], c) and torch.equal(st[to], t[0])
        block += -(-rows // 128)
    assert not st[block:].any() and not qt[:, 128 * block:].view(torch.uint8).any()
    with pytest.raises(lib.MxgemmValueError):
        lib.block128_quantize(torch.zeros(T + 1, 1, device="cuda", dtype=torch.bfloat16), cols=True, offsets=off)

    b, sb, _, _ = lib.block128_quantize(rand(len(sizes), n, k, seed=1), square=True)
    y = lib.block128_grouped_gemm(q, s, b, sb, off)
    assert not y[:head].any() and not y[head + sum(sizes):].any()
    lo = head
    for e, rows in enumerate(sizes):
        for at in {0, rows // 2, rows - 1} if rows else ():
            row = slice(lo + at, lo + at + 1)
            assert torch.equal(y[row], lib.block128_linear(q[row], s[:, row].contiguous(), b[e], sb[e]))
        lo += rows


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("sizes,n,k", [([3, 0, 5, 1], 96, 256), ([70, 0, 150, 33], 264, 272), ([700, 0, 900, 130], 2048, 144)])
def test_values_that_are_not_finite_stay_with_their_rows_and_experts(lib, sizes, n, k, dtype):  # noqa: F811
    """NaN in rows of no group, in the weights of a group without rows or of another, and in a row, its scale or its gate."""
    head, tail = 2, 6
    T, off = head + sum(sizes) + tail, offsets_of(sizes, head)
    a, sa, b, sb = operands(lib, T, n, k, groups=len(sizes))
    gate = rand(T, n, seed=3).to(DT[dtype])
    want = lib.block128_grouped_gemm(a, sa, b, sb, off, "silu", gate, True, c_dtype=DT[dtype])
    codes, weights, sa, sb, gate = a.view(torch.uint8).clone(), b.view(torch.uint8).clone(), sa.clone(), sb.clone(), gate.clone()
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[head:T - tail] = False
    codes[rest], gate[rest] = NAN, float("nan")
    sa[:, rest] = float("inf")
    weights[1] = NAN        # its group has no rows
    sb[1] = float("nan")
    got = lib.block128_grouped_gemm(codes.view(F8[0]), sa, weights.view(F8[0]), sb, off, "silu", gate, True, c_dtype=DT[dtype])
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    # one row's code, another one's scale, the weights of the last group
    spoilt = torch.zeros(T, dtype=torch.bool, device="cuda")
    spoilt[head], spoilt[head + 1] = True, True
    codes[head, 5], sa[0, head + 1] = NAN, float("nan")
    last = head + sum(sizes[:-1])
    weights[-1], spoilt[last:last + sizes[-1]] = NAN, True
    got = lib.block128_grouped_gemm(codes.view(F8[0]), sa, weights.view(F8[0]), sb, off, "silu", gate, True, c_dtype=DT[dtype])
    for x, y in zip(got, want):
        assert torch.equal(x[~spoilt], y[~spoilt]) and x[spoilt].isnan().all()


@pytest.mark.parametrize("sizes,m,n", [([70, 0, 300, 129], 72, 100), ([700, 0, 900, 1], 1000, 1000), ([6000, 0, 9000, 100], 70, 130)])
def test_values_that_are_not_finite_stay_with_their_expert(lib, sizes, m, n):  # noqa: F811
    head, tail = 3, 130
    off = offsets_of(sizes, head)
    x, y = rand(head + sum(sizes) + tail, m), rand(head + sum(sizes) + tail, n, seed=1)

    def quantised(t):
        return lib.block128_quantize(t, cols=True, offsets=off)
    clean = [quantised(t) for t in (x, y)]
    want = lib.block128_grouped_weight_gradient(*clean[0][2:], *clean[1][2:], off)
    # rows of no group
    for t in (x, y):
        t[:head], t[head + sum(sizes):] = float("nan"), float("inf")
    spoilt = [quantised(t) for t in (x, y)]
    for c, s in zip(clean, spoilt):
        assert equal(c[2], s[2]) and equal(c[3], s[3])
        assert equal(c[0][head:-tail], s[0][head:-tail]) and equal(c[1][:, head:-tail], s[1][:, head:-tail])
    # codes and scales behind the last group's blocks
    used = sum(-(-r // 128) for r in sizes)
    (_, _, a, sa), (_, _, b, sb) = spoilt
    for q, s in ((a, sa), (b, sb)):
        q.view(torch.uint8)[:, 128 * used:] = NAN
        s[used:] = float("nan")
    assert torch.equal(lib.block128_grouped_weight_gradient(a, sa, b, sb, off), want)
    # a token of the first expert
    a.view(torch.uint8)[4, 7] = NAN
    got = lib.block128_grouped_weight_gradient(a, sa, b, sb, off)
    assert got[0, 4].isnan().all() and torch.equal(got[1:], want[1:])
    got[0, 4] = want[0, 4]
    assert torch.equal(got, want)


def test_divided_products_in_graphs_that_share_a_workspace(lib):  # noqa: F811
    """Two graphs with one workspace, replayed one after the other with other values and group sizes and eager work between."""
    m, n, k = 64, 513, 7168
    a, sa, b, sb = operands(lib, m, n, k)
    r = rand(m, n, seed=3).bfloat16()
    off = offsets_of([6000, 0, 9000])
    x, y = rand(15000, 70).bfloat16(), rand(15000, 130, seed=1).bfloat16()
    _, _, p, sp = lib.block128_quantize(x, rows=False, cols=True, offsets=off)
    _, _, q, sq = lib.block128_quantize(y, rows=False, cols=True, offsets=off)
    need = max(lib._lib.mxgemm_block128_workspace_bytes(m, n, k, 1, 1), lib._lib.mxgemm_block128_workspace_bytes(m, n, k, 1, 0),
               lib._lib.mxgemm_block128_grouped_weight_gradient_workspace_bytes(p.shape[1] // 128, 3, 70, 130))
    scratch = torch.empty(need, dtype=torch.uint8, device="cuda")

    def one(**kw):
        return lib.block128_linear(a, sa, b, sb, None, "silu", None, r, True, **kw)

    def two(**kw):
        return (lib.block128_grouped_weight_gradient(p, sp, q, sq, off, **kw),
                lib.block128_linear(a, sa, b, sb, None, "gelu", c_dtype=torch.float32, **kw))
    graphs, outs = [], []
    for work in (one, two):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            work(workspace=scratch)
        torch.cuda.current_stream().wait_stream(side)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(work(workspace=scratch))
    for ends in ([6000, 0, 9000], [0, 15000, 0], [1, 2, 14000], [7000, 7000, 1000]):
        sa.mul_(1.25)
        r.add_(0.5)
        off.copy_(offsets_of(ends))
        for dst, src in (((p, sp), x), ((q, sq), y)):
            _, _, c, s = lib.block128_quantize(src, rows=False, cols=True, offsets=off)
            dst[0].copy_(c)
            dst[1].copy_(s)
        for graph, out, work in zip(graphs, outs, (one, two)):
            scratch.fill_(0xFF)
            graph.replay()
            assert all(torch.equal(g, w) for g, w in zip(out, work()))
