"""The operators of a routed feed-forward block as they are measured: their cases, their inputs, and for each a
plain form.

T tokens choose k of E experts each: n = T k choices.  On the library's formats (E4M3 codes with FP32 scales,
1 x 128 for activations and 128 x 128 for weights):

* expert_sort              the stable sort of the choices by expert: offsets [E + 1], rows [T, k], choices [n];
                           choices of no expert (a number outside 0 .. E - 1) come last and have rows ~r
* expert_dispatch          y[rows[t, j]] = x[t]; rows of choices of no expert are zero
* expert_dispatch_quant    the same, quantized: s = max(amax, 1e-4) / 448 per 1 x 128 (ue8m0: the next power of
                           two), codes E4M3(x / s)
* expert_combine           out[t] = sum_j w[t, j] y[rows[t, j]]; without weights the gradient of expert_dispatch
* expert_combine_backward  dy[rows[t, j]] = w[t, j] dout[t],  dw[t, j] = <dout[t], y[rows[t, j]]>
* expert_gemm              c[r] = a[r] W[e]^T for the rows offsets[e] <= r < offsets[e + 1] of expert e
* expert_gated_ffn         h[r] = silu(a[r] Wg[e]^T) * (a[r] Wu[e]^T)

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits; with ``own`` true it makes
the calls a user makes.
"""

import math

import torch

own = False

BLOCK = 128  # activation and weight block of the E4M3 formats
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

MOST_CHOICES = 8192 * 8
MOST_MOVED = 8192 * 8 * 7168       # elements of the sorted rows
MOST_WEIGHTS = 32 * 2048 * 7168    # weights of all experts, of one projection
MOST_PRODUCT = 4096 * 4 * 2048 * 7168


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token's choices: the decode step, launch latency is what counts
        {"name": "sort_one_token", "op": "sort", "t": 1, "k": 8, "e": 256, "drop": 0.0},
        # a prefill batch's choices, some of them padding
        {"name": "sort_prefill", "op": "sort", "t": 8192, "k": 8, "e": 256, "drop": 0.05},
        # a few requests decoded together
        {"name": "dispatch_quant_decode", "op": "dispatch_quant", "t": 16, "k": 8, "e": 256, "drop": 0.0, "h": 7168, "x": "bf16", "fmt": "ue8m0"},
        # a prefill batch: every token's row eight times over, bound by the writes
        {"name": "dispatch_quant_prefill", "op": "dispatch_quant", "t": 8192, "k": 8, "e": 256, "drop": 0.0, "h": 7168, "x": "bf16", "fmt": ""},
        # a training batch of a small model in fp32, rows of odd length
        {"name": "dispatch_odd_f32", "op": "dispatch", "t": 1333, "k": 3, "e": 24, "drop": 0.0, "h": 1001, "x": "f32"},
        # the gradient of sorting a training batch's rows, half of its choices at experts of another rank
        {"name": "dispatch_backward_half", "op": "dispatch_backward", "t": 4096, "k": 8, "e": 64, "drop": 0.5, "h": 2048, "x": "bf16"},
        # one token's experts put together: the decode step
        {"name": "combine_one_token", "op": "combine", "t": 1, "k": 8, "e": 256, "drop": 0.0, "h": 7168, "x": "bf16", "w": "f32"},
        # gradients of a training batch
        {"name": "combine_backward_train", "op": "combine_backward", "t": 4096, "k": 8, "e": 64, "drop": 0.02, "h": 4096, "x": "bf16", "w": "f32"},
        # one token at its eight experts, gate and up: the decode step, bound by the weights' bytes
        {"name": "gated_one_token", "op": "gated", "t": 1, "k": 8, "e": 32, "drop": 0.0, "n": 2048, "kk": 7168, "out": "bf16"},
        # a prefill batch at the experts' gate and up
        {"name": "gated_prefill", "op": "gated", "t": 4096, "k": 4, "e": 32, "drop": 0.0, "n": 2048, "kk": 7168, "out": "bf16"},
        # a ragged batch, some sixty rows an expert, width not a multiple of 128: bound by the weights' bytes
        {"name": "gemm_ragged", "op": "gemm", "t": 700, "k": 6, "e": 64, "drop": 0.03, "n": 2300, "kk": 1408, "out": "bf16"},
        # a prefill batch at the experts' down projection
        {"name": "gemm_prefill", "op": "gemm", "t": 4096, "k": 4, "e": 32, "drop": 0.0, "n": 7168, "kk": 2048, "out": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))


def draw(rng):
    op = rng.choice(["sort", "dispatch_quant", "dispatch_quant", "dispatch", "dispatch_backward", "combine", "combine",
                     "combine_backward", "gated", "gated", "gemm", "gemm"])
    k, drop = rng.choice([1, 2, 3, 4, 6, 8, 8]), rng.choice([0.0, 0.0, 0.04, 0.5])
    if op in ("gated", "gemm"):
        kk = BLOCK * _log_int(rng, 1, 56)
        n = _log_int(rng, 16, 7168)
        e = _log_int(rng, k, min(64, max(k, MOST_WEIGHTS // (n * kk))))
        t = _log_int(rng, 1, min(8192 // 2, MOST_PRODUCT // (n * kk * k)))
        return {"op": op, "t": t, "k": k, "e": e, "drop": drop, "n": n, "kk": kk, "out": "bf16"}
    case = {"op": op, "t": _log_int(rng, 1, MOST_CHOICES // k), "k": k, "e": _log_int(rng, k, 512), "drop": drop}
    if op == "sort":
        return case
    most = min(7168, MOST_MOVED // (2 * case["t"] * k))
    case["h"] = BLOCK * _log_int(rng, 1, max(1, most // BLOCK)) if op == "dispatch_quant" else _log_int(rng, 16, max(16, most))
    case["x"] = rng.choice(["bf16", "bf16", "f32"])
    if op == "dispatch_quant":
        case["fmt"] = rng.choice(["", "ue8m0"])
    if op in ("combine", "combine_backward"):
        case["w"] = rng.choice(["f32", "f32", "bf16"])
    return case


def _taking_part(case):
    """Choices that have an expert, and experts that have any, as expected of an even spread."""
    rows = case["t"] * case["k"] * (1 - case["drop"])
    return round(rows), max(1, round(case["e"] * (1 - (1 - 1 / case["e"]) ** rows)))


def work(case):
    op, t, n = case["op"], case["t"], case["t"] * case["k"]
    if op == "sort":
        return {"bytes": 8 * n + 8 * n + 4 * (case["e"] + 1), "flops": n}
    rows, experts = _taking_part(case)
    if op in ("gated", "gemm"):
        width, kk = case["n"] * (2 if op == "gated" else 1), case["kk"]
        weights = experts * (width * kk + -(-width // BLOCK) * (kk // BLOCK) * 4)
        return {"bytes": weights + rows * (kk + kk // BLOCK * 4) + n * case["n"] * 2, "flops": 2 * rows * width * kk}
    h, size = case["h"], TYPES[case["x"]].itemsize
    if op == "dispatch_quant":
        return {"bytes": 4 * n + t * h * size + n * (h + h // BLOCK * 4), "flops": 3 * t * h}
    if op == "dispatch":
        return {"bytes": 4 * n + t * h * size + n * h * size, "flops": 0}
    if op == "dispatch_backward":
        return {"bytes": 4 * n + rows * h * size + t * h * size, "flops": rows * h}
    weights = n * TYPES[case["w"]].itemsize
    if op == "combine":
        return {"bytes": 4 * n + weights + rows * h * size + t * h * size, "flops": 2 * rows * h}
    return {"bytes": 4 * n + 2 * weights + (rows + t) * h * size + n * h * size, "flops": 3 * rows * h}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _uniform(gen, *shape):
    return torch.rand(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _activations(gen, m, k):
    """Hidden states: N(0, 1) with a few features twenty times as large."""
    return _normal(gen, m, k) * torch.where(_uniform(gen, k) < 0.002, 20.0, 1.0)


def _weight(gen, e, n, k):
    """E4M3 weights of spread 0.02, their 128 x 128 blocks' magnitudes within a factor of four."""
    codes = torch.empty(e, n, k, dtype=torch.float8_e4m3fn, device="cuda")
    for i in range(e):
        codes[i] = (_normal(gen, n, k) * 100.0).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes, torch.exp2(_uniform(gen, e, -(-n // BLOCK), -(-k // BLOCK)) * 2 - 1) * (0.02 / 100.0)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, t, k, e = case["op"], case["t"], case["k"], case["e"]
    # a router's choices: experts differ in how often they are chosen, a token's k experts are different ones
    ids = (_normal(gen, t, e) + 0.5 * _normal(gen, e)).topk(k, dim=1).indices
    ids = torch.where(_uniform(gen, t, k) < case["drop"], -1, ids)
    state = {"case": case, "ids": ids}
    if op == "sort":
        return state
    state["offsets"], state["rows"], state["choices"] = _sort_plain(ids, e)
    if op in ("gated", "gemm"):
        x = _activations(gen, t, case["kk"])[torch.div(state["choices"], k, rounding_mode="floor").long()]
        state["a"], state["a_s"] = _quantized(x.bfloat16().float(), "")
        state["w0"], state["w0_s"] = _weight(gen, e, case["n"], case["kk"])
        if op == "gated":
            state["w1"], state["w1_s"] = _weight(gen, e, case["n"], case["kk"])
        return state
    h, kind = case["h"], TYPES[case["x"]]
    if op in ("dispatch", "dispatch_quant"):
        state["x"] = _activations(gen, t, h).to(kind)
        return state
    if op == "dispatch_backward":
        state["y"] = (_normal(gen, t * k, h) * 1e-3).to(kind)
        return state
    state["y"] = _normal(gen, t * k, h).to(kind)
    state["w"] = torch.softmax(_normal(gen, t, k), 1).to(TYPES[case["w"]])
    if op == "combine_backward":
        state["dout"] = (_normal(gen, t, h) * torch.exp2(_uniform(gen, t, 1) * 4 - 10)).to(kind)
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    import fp8_block_scaled_quant_amd as fb

    case, op = state["case"], state["case"]["op"]
    if op == "sort":
        return tuple(fb.expert_sort(state["ids"], case["e"]))
    if op == "dispatch_quant":
        return fb.expert_dispatch_quant(state["x"], state["rows"], scale_fmt=case["fmt"] or None)
    if op == "dispatch":
        return fb.expert_dispatch(state["x"], state["rows"])
    if op == "dispatch_backward":
        return fb.expert_combine(state["y"], state["rows"])
    if op == "combine":
        return fb.expert_combine(state["y"], state["rows"], state["w"])
    if op == "combine_backward":
        return fb.expert_combine_backward(state["dout"], state["y"], state["rows"], state["w"])
    if op == "gated":
        return fb.expert_gated_ffn(state["a"], state["a_s"], state["offsets"], state["w0"], state["w0_s"], state["w1"],
                                   state["w1_s"], out_dtype=TYPES[case["out"]])
    return fb.expert_gemm(state["a"], state["a_s"], state["offsets"], state["w0"], state["w0_s"], out_dtype=TYPES[case["out"]])


def _run_plain(state):
    case, op = state["case"], state["case"]["op"]
    if op == "sort":
        return _sort_plain(state["ids"], case["e"])
    rows = state["rows"].long()
    if op in ("gated", "gemm"):
        ends = state["offsets"].tolist()
        products = [_product_plain(state, i, begin, end) for i, (begin, end) in enumerate(zip(ends, ends[1:])) if end > begin]
        behind = state["a"].new_zeros((len(state["a"]) - ends[-1], case["n"]), dtype=torch.float32)
        return torch.cat(products + [behind]).to(TYPES[case["out"]])
    live = (rows >= 0)[..., None]
    if op in ("dispatch", "dispatch_quant"):
        # each sorted row's token, and whether the row is an expert's
        token = torch.div(state["choices"], case["k"], rounding_mode="floor").long()
        behind = torch.arange(len(token), device="cuda")[:, None] >= state["offsets"][-1]
        x = state["x"].float()
        y = torch.where(behind, 0.0, x[token])
        return _quantized(y, case["fmt"]) if op == "dispatch_quant" else y.to(state["x"].dtype)
    y = state["y"].float()
    if op == "dispatch_backward":
        return torch.where(live, y[rows.clamp(min=0)], 0.0).sum(1).to(state["y"].dtype)
    w = state["w"].float()[..., None]
    if op == "combine":
        return torch.where(live, w * y[rows.clamp(min=0)], 0.0).sum(1).to(state["y"].dtype)
    dout = state["dout"].float()[:, None, :]
    dy = torch.empty_like(y)
    dy[torch.where(rows < 0, -1 - rows, rows)] = torch.where(live, w * dout, 0.0)
    dw = torch.where(live, y[rows.clamp(min=0)] * dout, 0.0).sum(-1)
    return dy.to(state["y"].dtype), dw.to(state["w"].dtype)


def _sort_plain(ids, e):
    shape, ids = ids.shape, ids.flatten()
    key = torch.where((ids >= 0) & (ids < e), ids, e)
    choices = torch.sort(key, stable=True).indices
    at = torch.empty_like(choices)
    at[choices] = torch.arange(len(ids), device="cuda")
    counts = torch.zeros(e + 1, dtype=torch.long, device="cuda").index_add_(0, key, torch.ones_like(key))
    offsets = counts.cumsum(0) - counts
    rows = torch.where(key < e, at, -1 - at)
    return offsets.int(), rows.int().view(shape), choices.int()


def _product_plain(state, i, begin, end):
    """The rows of expert i."""
    a = state["a"][begin:end].float() * state["a_s"][begin:end].repeat_interleave(BLOCK, 1)
    g = a @ _dequantized(state["w0"][i], state["w0_s"][i]).T
    if "w1" not in state:
        return g
    return g * torch.sigmoid(g) * (a @ _dequantized(state["w1"][i], state["w1_s"][i]).T)


def _power32(e):
    """2^e from its bits (exponents of normal values): torch's own powers are not exact everywhere."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantized(x, fmt):
    """1 x 128 E4M3 quantization: (codes, scales)."""
    b = x.view(x.shape[0], -1, BLOCK)
    # by a tensor: by a Python number torch multiplies with the rounded inverse
    s = b.abs().amax(-1, keepdim=True).clamp_min(1e-4) / b.new_tensor(448.0)
    if fmt == "ue8m0":
        part, e = torch.frexp(s)
        s = _power32(torch.where(part == 0.5, e - 1, e))
    return (b / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view_as(x), s[..., 0]


def _dequantized(codes, scale):
    n, k = codes.shape
    return codes.float() * scale.repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    op, state = case["op"], prepare(case, seed)
    if op == "sort":
        return None  # whole numbers only
    rows, k = state["rows"].long(), case["k"]
    if op in ("gated", "gemm"):
        out = torch.zeros(len(state["a"]), case["n"], dtype=torch.float64, device="cuda")
        ends = state["offsets"].tolist()
        for i in range(case["e"]):
            part = slice(ends[i], ends[i + 1])
            a = state["a"][part].double().unflatten(1, (-1, BLOCK)) * state["a_s"][part].double()[..., None]
            a = a.flatten(1)
            g = torch.matmul(a, _weight64(state["w0"][i], state["w0_s"][i]).t())
            if op == "gated":
                g = g / (1 + torch.exp(-g)) * torch.matmul(a, _weight64(state["w1"][i], state["w1_s"][i]).t())
            out[part] = g
        return out
    if op in ("dispatch", "dispatch_quant"):
        x = state["x"].double()
        y = torch.zeros(rows.numel(), x.shape[1], dtype=torch.float64, device="cuda")
        for j in range(k):
            there = rows[:, j] >= 0
            y[rows[there, j]] = x[there]
        if op == "dispatch":
            return y
        b = y.unflatten(1, (-1, BLOCK))
        # 1e-4 and the quotients are the format's FP32 numbers
        s = (b.abs().amax(-1).clamp(min=torch.tensor(1e-4).double().item()) / 448).float().double()
        if case["fmt"] == "ue8m0":
            part, e = torch.frexp(s)
            s = ((e.long() - (part == 0.5).long() + 1023) << 52).view(torch.float64)
        codes = _nearest_e4m3((b / s[..., None]).float().double()).flatten(1)
        return codes, s
    y = state["y"].double()
    if op in ("combine", "dispatch_backward"):
        out = torch.zeros(case["t"], case["h"], dtype=torch.float64, device="cuda")
        for j in range(k):
            there = rows[:, j] >= 0
            w = state["w"][there, j].double()[:, None] if op == "combine" else 1.0
            out[there] += w * y[rows[there, j]]
        return out
    dout = state["dout"].double()
    dy, dw = torch.zeros_like(y), torch.zeros(rows.shape, dtype=torch.float64, device="cuda")
    for j in range(k):
        there = rows[:, j] >= 0
        at = rows[there, j]
        dy[at] = state["w"][there, j].double()[:, None] * dout[there]
        dw[there, j] = torch.linalg.vecdot(dout[there], y[at])
    return dy, dw


def _nearest_e4m3(v):
    """Nearest E4M3 value, ties to even, saturating: 2^-9 apart up to 2^-6, then eight steps a binade."""
    v = v.clamp(-448, 448)
    # frexp's exponent counts from 0.5, one above the binade's
    e = torch.frexp(v.abs().clamp(min=2.0 ** -6))[1]
    quantum = ((e.long() - 4 + 1023) << 52).view(torch.float64)
    return torch.round(v / quantum) * quantum


def _weight64(codes, scale):
    rows = torch.arange(codes.shape[0], device="cuda") // BLOCK
    cols = torch.arange(codes.shape[1], device="cuda") // BLOCK
    return codes.double() * scale.double()[rows][:, cols]
