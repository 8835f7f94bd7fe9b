"""Workloads of a feed-forward layer's products on block-128 codes: inputs, plain forms, exact values, work of one pass.

Five operators carry such a layer, dense or with its rows grouped by expert, forward and back:

* ``quantise``: tokens in order of their experts to 8-bit codes with one float32 scale per block of 128, the blocks along
  the tokens starting afresh at every expert's first row;
* ``grouped``: the product of such rows with their own expert's weight, with an activation and a gate where asked for;
* ``weight_gradient``: one product over the tokens of each expert;
* ``linear``: a dense product with bias, activation, gate and residual;
* ``backward``: the gradients through bias, activation and gate.

``run`` computes them with elementary torch operations in 32 bits, or, where ``own`` is set, through the
package's entry points on the same inputs.
"""

import math

import torch

own = False

TINY = 448.0 * 2.0 ** -100     # the smallest block maximum that a scale is made of
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
CODE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
DTYPE = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
SIZE = {"float32": 4, "bfloat16": 2, "float16": 2}
LARGEST_FLOPS = 2 * 16384 * 4096 * 7168
LARGEST_WEIGHTS = 32 * 4096 * 7168
LARGEST_VALUES = 8192 * 8192


def _quantise(name, T, E, K, dtype, fmt, rows, index, spread, behind):
    return {"name": name, "op": "quantise", "T": T, "E": E, "K": K, "dtype": dtype, "fmt": fmt, "rows": rows,
            "index": index, "spread": spread, "behind": behind}


def _grouped(name, T, E, N, K, a_fmt, c_dtype, activation, gate, preact, index, spread, behind):
    return {"name": name, "op": "grouped", "T": T, "E": E, "N": N, "K": K, "a_fmt": a_fmt, "c_dtype": c_dtype,
            "activation": activation, "gate": gate, "preact": preact, "index": index, "spread": spread, "behind": behind}


def _weight_gradient(name, T, E, M, N, index, spread, behind):
    return {"name": name, "op": "weight_gradient", "T": T, "E": E, "M": M, "N": N, "index": index, "spread": spread,
            "behind": behind}


def _linear(name, M, N, K, c_dtype, bias, activation, gate, residual, preact):
    return {"name": name, "op": "linear", "M": M, "N": N, "K": K, "c_dtype": c_dtype, "bias": bias,
            "activation": activation, "gate": gate, "residual": residual, "preact": preact}


def _backward(name, M, N, dtype, activation, gate, bias):
    return {"name": name, "op": "backward", "M": M, "N": N, "dtype": dtype, "activation": activation, "gate": gate,
            "bias": bias}


def listed():
    return [
        # a training batch in order of its experts: one read gives the forward operand and the weight gradient's
        _quantise("quantise_experts", 8192, 32, 7168, "bfloat16", "e4m3", True, "int32", 0.5, 0),
        # gradients of a small batch, some experts without a row and rows behind the last one
        _quantise("quantise_experts_ragged", 333, 16, 2048, "float16", "e5m2", False, "int64", 2.0, 20),
        # one decoding step: eight rows that mostly meet eight different experts, whose weights are read once
        _grouped("experts_one_token", 8, 64, 2048, 7168, "e4m3", "bfloat16", "silu", True, False, "int32", 0.0, 0),
        # a long prompt over 32 experts, the gated half of their first products
        _grouped("experts_prompt", 16384, 32, 4096, 7168, "e4m3", "bfloat16", "silu", True, False, "int32", 0.5, 0),
        # input gradients of a training batch in the gradients' format, ragged
        _grouped("experts_input_gradient", 4001, 16, 7168, 2048, "e5m2", "float16", None, False, False, "int64", 1.0, 33),
        # the weights' gradients of a training batch
        _weight_gradient("experts_weight_gradient", 8192, 16, 4096, 2048, "int32", 0.5, 0),
        # those of a small batch, some experts without a row
        _weight_gradient("experts_weight_gradient_ragged", 500, 8, 2048, 1024, "int64", 2.0, 11),
        # the output projection of one sequence's next token, onto the residual stream
        _linear("linear_one_row", 1, 7168, 2048, "bfloat16", True, None, False, True, False),
        # a first product with bias and activation over ragged rows, its input to the activation kept for training
        _linear("linear_ragged", 4000, 7168, 2048, "float16", True, "gelu", False, False, True),
        # the gated half of a training batch's first products
        _linear("linear_gated", 8192, 8192, 4096, "bfloat16", False, "silu", True, False, True),
        # gradients through a small float32 layer
        _backward("backward_small", 40, 2048, "float32", "gelu_tanh", False, True),
        # gradients through the gated half of a training batch
        _backward("backward_gated", 8192, 8192, "bfloat16", "silu", True, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["quantise", "quantise", "grouped", "grouped", "grouped", "weight_gradient", "weight_gradient",
                     "linear", "linear", "linear", "backward", "backward"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float16", "float32"])
    activation = rng.choice([None, "relu", "silu", "silu", "gelu", "gelu_tanh"])
    index, spread = rng.choice(["int32", "int64"]), rng.choice([0.0, 0.5, 1.0, 2.0])
    if op == "quantise":
        K = _log(rng, 64, 7168)
        T = _log(rng, 1, min(16384, LARGEST_VALUES // K))
        case = _quantise("", T, _log(rng, 1, 256), K, dtype, rng.choice(["e4m3", "e4m3", "e5m2"]), rng.random() < 0.7,
                         index, spread, rng.choice([0, T // 9]))
    elif op == "grouped":
        K, N = 16 * _log(rng, 8, 448), _log(rng, 64, 8192)
        E = _log(rng, 1, min(256, LARGEST_WEIGHTS // (N * K)))
        # float32 takes the 16-bit matrix cores: half as much
        T = _log(rng, 1, max(1, min(16384, LARGEST_FLOPS // (2 * N * K * (2 if dtype == "float32" else 1)))))
        case = _grouped("", T, E, N, K, rng.choice(["e4m3", "e4m3", "e5m2"]), dtype, activation, rng.random() < 0.4,
                        rng.random() < 0.3, index, spread, rng.choice([0, T // 9]))
    elif op == "weight_gradient":
        M, N = _log(rng, 64, 7168), _log(rng, 64, 4096)
        E = _log(rng, 1, max(1, min(256, LARGEST_WEIGHTS // (4 * M * N))))
        T = _log(rng, 1, max(1, min(16384, LARGEST_FLOPS // (4 * M * N))))
        case = _weight_gradient("", T, E, M, N, index, spread, rng.choice([0, T // 9]))
    elif op == "linear":
        K, N = 16 * _log(rng, 8, 448), _log(rng, 64, 24576)
        M = _log(rng, 1, max(1, min(8192, LARGEST_FLOPS // (2 * N * K * (2 if dtype == "float32" else 1)))))
        case = _linear("", M, N, K, dtype, rng.random() < 0.6, activation, rng.random() < 0.3, rng.random() < 0.4,
                       rng.random() < 0.3)
    else:
        N = _log(rng, 64, 24576)
        M = _log(rng, 1, min(16384, LARGEST_VALUES // (N * (2 if dtype == "float32" else 1))))
        case = _backward("", M, N, dtype, activation, rng.random() < 0.4, rng.random() < 0.6)
    del case["name"]
    return case


# --- inputs ---------------------------------------------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _codes(x, fmt, rows):
    """Codes and scales that quantisation in blocks of rows x 128 gives for x (L, M, K), K a multiple of 16."""
    L, M, K = x.shape
    kb, mb = -(-K // 128), -(-M // rows)
    padded = torch.nn.functional.pad(x, (0, kb * 128 - K, 0, mb * rows - M)).view(L, mb, rows, kb, 128)
    scale = padded.abs().amax(dim=(2, 4)).clamp(min=TINY) / FMAX[fmt]
    q = (padded / scale[:, :, None, :, None]).clamp(-FMAX[fmt], FMAX[fmt]).to(CODE[fmt])
    q = q.view(L, mb * rows, kb * 128)[:, :M, :K].contiguous()
    return q, (scale.transpose(1, 2) if rows == 1 else scale).contiguous()


def _sizes(case, seed):
    """Rows of every expert: T - behind rows that fall to experts of unequal weight, with none for an eighth of them
    where spread is large."""
    g = torch.Generator().manual_seed(seed)
    E = case["E"]
    weight = torch.exp(case["spread"] * torch.randn(E, generator=g, dtype=torch.float64))
    if case["spread"] >= 2 and E >= 8:
        weight[torch.randperm(E, generator=g)[:E // 8]] = 0
    who = torch.multinomial(weight, case["T"] - case["behind"], replacement=True, generator=g)
    return torch.bincount(who, minlength=E).tolist()


def _group_blocks(T, E):
    """Blocks of 128 tokens that E groups of T rows in all may take, each starting with a block of its own."""
    return (T + 127 * min(E, T)) // 128


def _regroup(sizes, blocks):
    """For each column of the operand over tokens its row among the tokens, or -1."""
    at = torch.full((blocks, 128), -1, dtype=torch.int64)
    row = block = 0
    for n in sizes:
        nb = -(-n // 128)
        at[block:block + nb].view(-1)[:n] = torch.arange(row, row + n)
        row, block = row + n, block + nb
    return at.view(-1).cuda()


def _token_operand(x, sizes, fmt, blocks):
    """Codes (K, 128 blocks) and scales (blocks, K) of x (T, K) in blocks of 128 along each group's tokens."""
    at = _regroup(sizes, blocks)
    full = torch.where((at >= 0)[:, None], x[at.clamp(min=0)], 0.0).t().contiguous()
    q, s = _codes(full[None], fmt, 1)
    return q[0], s[0]


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    state = {"case": case}
    if "E" in case:
        state["sizes"] = _sizes(case, seed)
        ends = torch.tensor([0] + state["sizes"], dtype=torch.int64).cumsum(0)
        state["offsets"] = ends.to(torch.int32 if case["index"] == "int32" else torch.int64).cuda()
    if op == "quantise":
        # activations of unit size with a few channels that are much larger
        x = normal(case["T"], case["K"])
        x *= torch.exp(0.5 * normal(case["K"])) * (1 + 20 * (torch.rand(case["K"], generator=g, device="cuda") < 0.005))
        state["x"] = x.to(DTYPE[case["dtype"]])
        return state
    if op == "weight_gradient":
        T, M, N = case["T"], case["M"], case["N"]
        blocks = _group_blocks(T, case["E"])
        state["a"], state["sa"] = _token_operand(normal(T, M), state["sizes"], "e5m2", blocks)
        state["b"], state["sb"] = _token_operand(normal(T, N), state["sizes"], "e4m3", blocks)
        return state
    if op == "backward":
        dt = DTYPE[case["dtype"]]
        state["dy"], state["z"] = normal(case["M"], case["N"]).to(dt), normal(case["M"], case["N"]).to(dt)
        state["gate"] = normal(case["M"], case["N"]).to(dt) if case["gate"] else None
        return state
    N, K, dt = case["N"], case["K"], DTYPE[case["c_dtype"]]
    rows = case["T"] if op == "grouped" else case["M"]
    a, sa = _codes(normal(1, rows, K), case.get("a_fmt", "e4m3"), 1)
    state["a"], state["sa"] = a[0], sa[0]
    parts = [_codes(normal(1, N, K) / math.sqrt(K), "e4m3", 128) for _ in range(case.get("E", 1))]
    state["b"] = torch.cat([q.view(torch.uint8) for q, _ in parts]).view(CODE["e4m3"])
    state["sb"] = torch.cat([s for _, s in parts])
    state["gate"] = normal(rows, N).to(dt) if case["gate"] else None
    if op == "linear":
        state["b"], state["sb"] = state["b"][0], state["sb"][0]
        state["bias"] = (0.5 * normal(N)).to(dt) if case["bias"] else None
        state["residual"] = (2 * normal(rows, N)).to(dt) if case["residual"] else None
    return state


# --- plain forms ----------------------------------------------------------------------------------------------------

def _scaled(q, s, block):
    """float32 values of codes (R, K) with scales in blocks of block x 128."""
    R, K = q.shape
    s = s.t() if block == 1 else s.repeat_interleave(128, dim=0)[:R]
    return q.float() * s.repeat_interleave(128, dim=1)[:, :K]


def _sigmoid(z):
    e = torch.exp(-z.abs())
    return torch.where(z >= 0, 1 / (1 + e), e / (1 + e))


TANH = math.sqrt(2 / math.pi)


def _activate(z, kind):
    if kind is None:
        return z
    if kind == "relu":
        return torch.where(z > 0, z, 0.0)
    if kind == "silu":
        return z * _sigmoid(z)
    if kind == "gelu":
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    return z * _sigmoid(2 * TANH * (z + 0.044715 * z * z * z))


def _slope(z, kind):
    if kind is None:
        return torch.ones_like(z)
    if kind == "relu":
        return torch.where(z > 0, 1.0, 0.0)
    if kind == "silu":
        s = _sigmoid(z)
        return s * (1 + z * (1 - s))
    if kind == "gelu":
        return 0.5 * torch.erfc(-z * math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    s = _sigmoid(2 * TANH * (z + 0.044715 * z * z * z))
    return s * (1 + z * (1 - s) * 2 * TANH * (1 + 3 * 0.044715 * z * z))


def _plain_quantise(state):
    c, x = state["case"], state["x"]
    fmt, (T, K) = c["fmt"], x.shape
    blocks, kb, k16 = _group_blocks(T, c["E"]), -(-K // 128), -(-K // 16) * 16

    def block_scale(amax):
        return amax.clamp(min=TINY) / FMAX[fmt]

    def code(v, amax):
        # the quotient in 64 bits: values next to a border between codes
        return (v.double() * FMAX[fmt] / amax.clamp(min=TINY).double()).to(CODE[fmt])

    out = {}
    if c["rows"]:
        tiles = torch.nn.functional.pad(x.float(), (0, kb * 128 - K)).view(T, kb, 128)
        amax = tiles.abs().amax(dim=2)
        out["q"] = code(tiles, amax[..., None]).view(T, kb * 128)[:, :k16].contiguous()
        out["s"] = block_scale(amax).t().contiguous()
    qt = torch.zeros(K, 128 * blocks, dtype=CODE[fmt], device="cuda")
    st = torch.zeros(blocks, K, device="cuda")
    row = block = 0
    for n in state["sizes"]:
        nb = -(-n // 128)
        if n:
            part = torch.nn.functional.pad(x[row:row + n].float(), (0, 0, 0, 128 * nb - n)).view(nb, 128, K)
            amax = part.abs().amax(dim=1)
            qt[:, 128 * block:128 * (block + nb)] = code(part, amax[:, None]).view(128 * nb, K).t()
            st[block:block + nb] = block_scale(amax)
        row, block = row + n, block + nb
    out["qt"], out["st"] = qt, st
    return out


def _finish(z, c, state, rows=slice(None)):
    """(y, z), or y alone, of a product's values z."""
    dt = DTYPE[c["c_dtype"]]
    if state.get("bias") is not None:
        z = z + state["bias"].float()
    y = _activate(z, c["activation"])
    if state["gate"] is not None:
        y = y * state["gate"][rows].float()
    if state.get("residual") is not None:
        y = y + state["residual"].float()
    return (y.to(dt), z.to(dt)) if c["preact"] else y.to(dt)


def _plain_grouped(state):
    c = state["case"]
    T, N, dt = c["T"], c["N"], DTYPE[c["c_dtype"]]
    out = [torch.zeros(T, N, dtype=dt, device="cuda") for _ in range(2 if c["preact"] else 1)]
    row = 0
    for e, n in enumerate(state["sizes"]):
        if n:
            at = slice(row, row + n)
            a, b = _scaled(state["a"][at], state["sa"][:, at], 1), _scaled(state["b"][e], state["sb"][e], 128)
            done = _finish(a @ b.t().contiguous(), c, state, at)
            for o, d in zip(out, done if c["preact"] else (done,)):
                o[at] = d
        row += n
    return tuple(out) if c["preact"] else out[0]


def _plain_weight_gradient(state):
    c = state["case"]
    out = torch.zeros(c["E"], c["M"], c["N"], device="cuda")
    block = 0
    for e, n in enumerate(state["sizes"]):
        nb = -(-n // 128)
        if n:
            at, of = slice(128 * block, 128 * (block + nb)), slice(block, block + nb)
            a, b = _scaled(state["a"][:, at], state["sa"][of], 1), _scaled(state["b"][:, at], state["sb"][of], 1)
            out[e] = a @ b.t().contiguous()
        block += nb
    return out


def _plain_linear(state):
    a, b = _scaled(state["a"], state["sa"], 1), _scaled(state["b"], state["sb"], 128)
    return _finish(a @ b.t().contiguous(), state["case"], state)


def _plain_backward(state):
    c, dy, z, dt = state["case"], state["dy"].float(), state["z"].float(), DTYPE[state["case"]["dtype"]]
    out = {}
    if c["gate"]:
        out["dgate"] = (dy * _activate(z, c["activation"])).to(dt)
        dy = dy * state["gate"].float()
    dz = dy * _slope(z, c["activation"])
    out["dz"] = dz.to(dt)
    if c["bias"]:
        out["dbias"] = dz.sum(dim=0)
    return out


def _plain(state):
    return {"quantise": _plain_quantise, "grouped": _plain_grouped, "weight_gradient": _plain_weight_gradient,
            "linear": _plain_linear, "backward": _plain_backward}[state["case"]["op"]](state)


def _own(state):
    import block_scaled_precision_e4m3_amd as lib

    c = state["case"]
    op = c["op"]
    if op == "quantise":
        fmt = lib.MXG_FMT_E4M3 if c["fmt"] == "e4m3" else lib.MXG_FMT_E5M2
        q, s, qt, st = lib.block128_quantize(state["x"], fmt=fmt, rows=c["rows"], cols=True, offsets=state["offsets"])
        return {k: v for k, v in (("q", q), ("s", s), ("qt", qt), ("st", st)) if v is not None}
    if op == "grouped":
        return lib.block128_grouped_gemm(state["a"], state["sa"], state["b"], state["sb"], state["offsets"],
                                         activation=c["activation"], gate=state["gate"], preact=c["preact"],
                                         c_dtype=DTYPE[c["c_dtype"]])
    if op == "weight_gradient":
        return lib.block128_grouped_weight_gradient(state["a"], state["sa"], state["b"], state["sb"], state["offsets"])
    if op == "linear":
        return lib.block128_linear(state["a"], state["sa"], state["b"], state["sb"], bias=state["bias"],
                                   activation=c["activation"], gate=state["gate"], residual=state["residual"],
                                   preact=c["preact"], c_dtype=DTYPE[c["c_dtype"]])
    dz, dgate, dbias = lib.activation_backward(state["dy"], state["z"], activation=c["activation"], gate=state["gate"],
                                               bias=c["bias"])
    return {k: v for k, v in (("dgate", dgate), ("dz", dz), ("dbias", dbias)) if v is not None}


def run(state):
    return _own(state) if own else _plain(state)


# --- the work of one pass -------------------------------------------------------------------------------------------

def work(case):
    c, op = case, case["op"]
    if op == "backward":
        values = c["M"] * c["N"]
        moved = values * SIZE[c["dtype"]] * (5 if c["gate"] else 3) + (4 * c["N"] if c["bias"] else 0)
        return {"bytes": moved, "flops": 20 * values}
    if op == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        kb, e = -(-K // 128), SIZE[c["c_dtype"]]
        moved = M * K + N * K + 4 * kb * (M + -(-N // 128)) + (N * e if c["bias"] else 0)
        moved += M * N * e * (1 + int(c["gate"]) + int(c["residual"]) + int(c["preact"]))
        return {"bytes": moved, "flops": 2 * M * N * K}
    T, E, used = c["T"], c["E"], c["T"] - c["behind"]
    index = (E + 1) * (4 if c["index"] == "int32" else 8)
    blocks = _group_blocks(T, E)
    if op == "quantise":
        K, e = c["K"], SIZE[c["dtype"]]
        moved = T * K * e + 128 * blocks * K + 4 * blocks * K + index
        if c["rows"]:
            moved += T * K + 4 * T * -(-K // 128)
        return {"bytes": moved, "flops": 2 * T * K * (2 if c["rows"] else 1)}
    if op == "grouped":
        N, K, e = c["N"], c["K"], SIZE[c["c_dtype"]]
        met = E * (1 - (1 - 1 / E) ** used)     # experts that are expected to have a row
        kb = -(-K // 128)
        moved = used * (K + 4 * kb) + met * (N * K + 4 * kb * -(-N // 128)) + index
        moved += N * e * (T * (1 + int(c["preact"])) + used * int(c["gate"]))
        return {"bytes": int(moved), "flops": 2 * used * N * K}
    M, N = c["M"], c["N"]
    return {"bytes": (M + N) * (used + 4 * (-(-used // 128))) + 4 * E * M * N + index, "flops": 2 * used * M * N}


# --- exact values ---------------------------------------------------------------------------------------------------

def _nearest(v, fmt):
    """v (float64) rounded to the nearest value of the 8-bit format, ties to even."""
    bits, lowest = (3, -6) if fmt == "e4m3" else (2, -14)
    exponent = torch.frexp(v)[1].double() - 1
    step = torch.exp2(exponent.clamp(min=lowest) - bits)
    return ((v / step).round() * step).clamp(-FMAX[fmt], FMAX[fmt])


def _exact_quantise(c, state):
    x, fmt = state["x"].double(), c["fmt"]
    T, K = x.shape
    out = {}
    if c["rows"]:
        wide = x.new_zeros(T, -(-K // 128) * 128)
        wide[:, :K] = x
        tiles = wide.unflatten(1, (-1, 128))
        top = tiles.abs().amax(dim=2, keepdim=True).clamp(min=TINY)
        out["q"] = _nearest(tiles * FMAX[fmt] / top, fmt).flatten(1)[:, :-(-K // 16) * 16].contiguous()
        out["s"] = (top[..., 0] / FMAX[fmt]).mT.contiguous()
    at = _regroup(state["sizes"], _group_blocks(T, c["E"]))
    gathered = torch.where((at >= 0)[:, None], x[at.clamp(min=0)], 0.0).unflatten(0, (-1, 128))
    top = gathered.abs().amax(dim=1, keepdim=True).clamp(min=TINY)
    out["qt"] = _nearest(gathered * FMAX[fmt] / top, fmt).flatten(0, 1).mT.contiguous()
    used = (at.view(-1, 128) >= 0).any(dim=1)
    out["st"] = torch.where(used[:, None], top[:, 0] / FMAX[fmt], 0.0)
    return out


def _values(q, s, block):
    """float64 values of codes (R, K): scales (K blocks, R) or (R blocks, K blocks)."""
    r, k = torch.arange(q.shape[0], device="cuda"), torch.arange(q.shape[1], device="cuda") // 128
    return q.double() * (s.double()[k][:, r].t() if block == 1 else s.double()[r // block][:, k])


def _exact_activation(z, kind):
    """(value, slope) in float64."""
    if kind is None:
        return z, torch.ones_like(z)
    if kind == "relu":
        return z.clamp(min=0), (z > 0).double()
    if kind == "gelu":
        phi = torch.special.ndtr(z)
        return z * phi, phi + z * torch.exp(-z * z / 2) / (2 * math.pi) ** 0.5
    if kind == "silu":
        s = torch.special.expit(z)
        return z * s, s + z * s * torch.special.expit(-z)
    a = (2 / math.pi) ** 0.5
    u, du = a * (z + 0.044715 * z ** 3), a * (1 + 0.134145 * z ** 2)
    # (1 + tanh u) / 2, without its cancellation
    s = torch.special.expit(2 * u)
    return z * s, s + 2 * z * s * torch.special.expit(-2 * u) * du


def _exact_ends(c, z, bias, gate, residual):
    if bias is not None:
        z = z + bias.double()
    y = _exact_activation(z, c["activation"])[0]
    y = y if gate is None else y * gate.double()
    y = y if residual is None else y + residual.double()
    return (y, z) if c["preact"] else (y,)


def exact(case, seed):
    state = prepare(case, seed)
    c, op = case, case["op"]
    if op == "quantise":
        return _exact_quantise(c, state)
    if op == "linear":
        out = []
        b = _values(state["b"], state["sb"], 128).t().contiguous()
        for m in range(0, c["M"], 1024):
            at = slice(m, m + 1024)
            z = _values(state["a"][at], state["sa"][:, at], 1) @ b
            out.append(_exact_ends(c, z, *(state[k] if k == "bias" or state[k] is None else state[k][at]
                                           for k in ("bias", "gate", "residual"))))
        out = tuple(torch.cat(parts) for parts in zip(*out))
        return out if c["preact"] else out[0]
    if op == "backward":
        dy, (value, slope) = state["dy"].double(), _exact_activation(state["z"].double(), c["activation"])
        out = {}
        if c["gate"]:
            out["dgate"] = dy * value
            slope = slope * state["gate"].double()
        out["dz"] = dy * slope
        if c["bias"]:
            out["dbias"] = out["dz"].sum(dim=0)
        return out
    ends = torch.tensor(state["sizes"]).cumsum(0).tolist()
    if op == "grouped":
        outs = [torch.zeros(c["T"], c["N"], dtype=torch.float64, device="cuda") for _ in range(1 + int(c["preact"]))]
        for e, end in enumerate(ends):
            at = slice(end - state["sizes"][e], end)
            if at.start == at.stop:
                continue
            z = _values(state["a"][at], state["sa"][:, at], 1) @ _values(state["b"][e], state["sb"][e], 128).t().contiguous()
            gate = None if state["gate"] is None else state["gate"][at]
            for o, v in zip(outs, _exact_ends(c, z, None, gate, None)):
                o[at] = v
        return tuple(outs) if c["preact"] else outs[0]
    a, b = _values(state["a"], state["sa"], 1), _values(state["b"], state["sb"], 1)
    total = torch.zeros(c["E"], c["M"], c["N"], dtype=torch.float64, device="cuda")
    first = 0
    for e, n in enumerate(state["sizes"]):
        last = first + -(-n // 128) * 128
        if n:
            total[e] = a[:, first:last].contiguous() @ b[:, first:last].t().contiguous()
        first = last
    return total
