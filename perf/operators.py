"""The feed-forward operators as they are measured: their cases, their inputs, and for each a plain form.

The operators, on the library's own formats (E4M3 codes with FP32 scales, 1 x 128 for activations and
128 x 128 for weights; E2M1 codes with one power-of-two scale per 32 for 4-bit weights):

* gated_ffn           h = silu(g) * u,  g = Q(x) Wg^T,  u = Q(x) Wu^T  (Q: 1 x 128 E4M3 quantization)
* gated_ffn_backward  dg = dh u silu'(g),  du = dh silu(g);
                      dx = Q(dg) Wg + Q(du) Wu  (Q along the hidden features),
                      dWg = Q(dg)^T Q(x),  dWu = Q(du)^T Q(x)  (Q along the tokens)
* fp4_weight_quant    per 32 weights of a row: s = smallest power of two with amax <= 6 s, code = E2M1(w / s)
* fp4_gemv            y = x W^T (+ bias) with such a weight
* clip_grad_norm      norm = sqrt(sum of squares over all tensors); every tensor times
                      min(1, max_norm / (norm + 1e-6))

With ``own`` false, ``run`` computes them with elementary torch operations in 32 bits; with ``own`` true it
makes the calls a user makes.
"""

import math

import torch

own = False

BLOCK = 128          # activation and weight block of the E4M3 formats
GROUP = 32           # weights that share one scale in the 4-bit format
FLOOR = 2.0 ** -100  # smallest amax a power-of-two scale is made from
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

MOST_FFN = 8192 * 18432 * 7168
MOST_BACKWARD = 4096 * 18432 * 7168
MOST_WEIGHT = 18432 * 7168
MOST_GRADS = 400_000_000


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token through the dense block's two up-projections: the decode step, bound by the weights' bytes
        {"name": "ffn_one_token", "op": "ffn", "m": 1, "f": 18432, "k": 7168, "x": "bf16", "fmt": "", "save": False},
        # a small layer on fp32 activations: launch latency is what counts
        {"name": "ffn_tiny_f32", "op": "ffn", "m": 16, "f": 256, "k": 512, "x": "f32", "fmt": "", "save": False},
        # a ragged batch of tokens at one narrow expert, hidden width not a multiple of 128
        {"name": "ffn_expert_ragged", "op": "ffn", "m": 211, "f": 2300, "k": 7168, "x": "bf16", "fmt": "ue8m0", "save": False},
        # a training step's forward pass: the gate and up values are kept for the backward pass
        {"name": "ffn_train_forward", "op": "ffn", "m": 8192, "f": 18432, "k": 7168, "x": "bf16", "fmt": "ue8m0", "save": True},
        # backward pass of a narrow layer, an odd number of tokens
        {"name": "ffn_backward_odd", "op": "ffn_backward", "m": 333, "f": 1024, "k": 896},
        # backward pass of the dense block
        {"name": "ffn_backward_dense", "op": "ffn_backward", "m": 4096, "f": 18432, "k": 7168},
        # packing a small fp32 weight, last tile of rows not full
        {"name": "fp4_quant_small_f32", "op": "fp4_quant", "n": 300, "k": 1056, "x": "f32"},
        # packing one of the dense block's weights
        {"name": "fp4_quant_dense", "op": "fp4_quant", "n": 18432, "k": 7168, "x": "bf16"},
        # one token through a 4-bit weight: the decode step
        {"name": "fp4_one_token", "op": "fp4_gemv", "m": 1, "n": 18432, "k": 7168, "x": "bf16", "out": "bf16", "bias": False},
        # a few requests decoded together, fp32 in and out, odd sizes, with a bias
        {"name": "fp4_batch_odd_f32", "op": "fp4_gemv", "m": 13, "n": 2311, "k": 4128, "x": "f32", "out": "f32", "bias": True},
        # gradients of many small tensors (norm weights, biases, narrow layers), in two types
        {"name": "clip_many_small", "op": "clip", "tensors": 240, "mean": 3000, "type": "mixed", "over": 2.0},
        # gradients of a block's three large weights and its vectors
        {"name": "clip_dense_block", "op": "clip", "tensors": 3, "mean": 18432 * 7168, "type": "bf16", "over": 3.0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "ffn_backward", "ffn_backward", "fp4_quant", "fp4_gemv", "fp4_gemv", "clip"])
    if op == "ffn":
        f, k = _log_int(rng, 64, 18432), BLOCK * _log_int(rng, 1, 56)
        m = _log_int(rng, 1, min(8192, MOST_FFN // (f * k)))
        return {"op": op, "m": m, "f": f, "k": k, "x": rng.choice(["bf16", "bf16", "f32"]),
                "fmt": rng.choice(["", "ue8m0"]), "save": rng.random() < 0.4}
    if op == "ffn_backward":
        f, k = BLOCK * _log_int(rng, 1, 144), BLOCK * _log_int(rng, 1, 56)
        return {"op": op, "m": _log_int(rng, 1, min(4096, MOST_BACKWARD // (f * k))), "f": f, "k": k}
    if op == "fp4_quant":
        k = GROUP * _log_int(rng, 1, 576)
        return {"op": op, "n": _log_int(rng, 1, min(18432, MOST_WEIGHT // k)), "k": k, "x": rng.choice(["bf16", "f32"])}
    if op == "fp4_gemv":
        k = GROUP * _log_int(rng, 2, 576)
        return {"op": op, "m": _log_int(rng, 1, 64), "n": _log_int(rng, 16, min(32768, MOST_WEIGHT // k)), "k": k,
                "x": rng.choice(["bf16", "f32"]), "out": rng.choice(["bf16", "f32"]), "bias": rng.random() < 0.5}
    tensors = _log_int(rng, 1, 400)
    return {"op": op, "tensors": tensors, "mean": _log_int(rng, 300, MOST_GRADS // (2 * tensors)),
            "type": rng.choice(["bf16", "f32", "mixed"]), "over": round(rng.uniform(0.5, 4.0), 2)}


def _sizes(case):
    """Element counts of a clip case's gradient tensors: some vectors, most odd, around the mean size."""
    mean = case["mean"]
    if case["tensors"] == 3:
        return [mean, mean, mean, 7168, 18432]
    return [max(1, mean * (1 + (7 * i) % 13) // 7 - (5 * i) % 3) for i in range(case["tensors"])]


def _grad_types(case):
    kinds = {"bf16": [torch.bfloat16], "f32": [torch.float32], "mixed": [torch.bfloat16, torch.float32]}[case["type"]]
    return [kinds[i % len(kinds)] for i in range(len(_sizes(case)))]


def work(case):
    op = case["op"]
    if op == "ffn":
        m, f, k = case["m"], case["f"], case["k"]
        outs = m * f * 2 * (3 if case["save"] else 1)
        scales = 2 * -(-f // BLOCK) * (k // BLOCK) * 4
        return {"bytes": m * k * TYPES[case["x"]].itemsize + 2 * f * k + scales + outs, "flops": 4 * m * f * k}
    if op == "ffn_backward":
        m, f, k = case["m"], case["f"], case["k"]
        scales = 2 * (f // BLOCK) * (k // BLOCK) * 4
        return {"bytes": 3 * m * f * 2 + m * k * 2 + 2 * f * k + scales + m * k * 2 + 2 * f * k * 2, "flops": 8 * m * f * k}
    if op == "fp4_quant":
        n, k = case["n"], case["k"]
        return {"bytes": n * k * TYPES[case["x"]].itemsize + n * k // 2 + n * k // GROUP, "flops": 3 * n * k}
    if op == "fp4_gemv":
        m, n, k = case["m"], case["n"], case["k"]
        out = (m + (1 if case["bias"] else 0)) * n * TYPES[case["out"]].itemsize
        return {"bytes": n * k // 2 + n * k // GROUP + m * k * TYPES[case["x"]].itemsize + out, "flops": 2 * m * n * k}
    sizes, types = _sizes(case), _grad_types(case)
    return {"bytes": 2 * sum(n * t.itemsize for n, t in zip(sizes, types)), "flops": 3 * sum(sizes)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _uniform(gen, *shape):
    return torch.rand(*shape, generator=gen, device="cuda", dtype=torch.float32)


def _activations(gen, m, k):
    """Hidden states: N(0, 1) with a few features twenty times as large."""
    x = _normal(gen, m, k)
    return x * torch.where(_uniform(gen, k) < 0.002, 20.0, 1.0)


def _e4m3_weight(gen, n, k):
    """An E4M3 weight of spread 0.02, its 128 x 128 blocks' magnitudes within a factor of four."""
    codes = (_normal(gen, n, k) * 100.0).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    scale = torch.exp2(_uniform(gen, -(-n // BLOCK), -(-k // BLOCK)) * 2 - 1) * (0.02 / 100.0)
    return codes, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    state = {"case": case}
    if op == "ffn":
        state["x"] = _activations(gen, case["m"], case["k"]).to(TYPES[case["x"]])
        state["wg"], state["wg_s"] = _e4m3_weight(gen, case["f"], case["k"])
        state["wu"], state["wu_s"] = _e4m3_weight(gen, case["f"], case["k"])
    elif op == "ffn_backward":
        m, f, k = case["m"], case["f"], case["k"]
        # gradients of a mean loss: small, rows of different weight, one token in sixteen masked out
        rows = torch.exp2(_uniform(gen, m, 1) * 4 - 14) * (_uniform(gen, m, 1) >= 1 / 16)
        state["dh"] = (_normal(gen, m, f) * rows).to(torch.bfloat16)
        state["x"] = _activations(gen, m, k).to(torch.bfloat16)
        state["g"] = (_normal(gen, m, f) * 1.7).to(torch.bfloat16)
        state["u"] = (_normal(gen, m, f) * 1.7).to(torch.bfloat16)
        state["wg"], state["wg_s"] = _e4m3_weight(gen, f, k)
        state["wu"], state["wu_s"] = _e4m3_weight(gen, f, k)
    elif op == "fp4_quant":
        n, k = case["n"], case["k"]
        w = _normal(gen, n, k) * (torch.exp2(_uniform(gen, n, 1) * 4 - 2) * 0.02)
        w[n // 2, : GROUP] = 0.0  # a group of pruned weights
        state["w"] = w.to(TYPES[case["x"]])
    elif op == "fp4_gemv":
        m, n, k = case["m"], case["n"], case["k"]
        state["x"] = _activations(gen, m, k).to(TYPES[case["x"]])
        state["q"] = torch.randint(0, 256, (n, k // 2), generator=gen, device="cuda", dtype=torch.uint8)
        state["s"] = torch.randint(116, 124, (n, k // GROUP), generator=gen, device="cuda", dtype=torch.uint8)
        state["bias"] = _normal(gen, n).to(TYPES[case["out"]]) if case["bias"] else None
    else:
        sizes, types = _sizes(case), _grad_types(case)
        # the tensors are views of one buffer per type, as gradient buckets are
        state["grads"], state["out"], state["flat_out"] = [], [], {}
        total = {t: sum(n for n, u in zip(sizes, types) if u == t) for t in types}
        flat = {t: (_normal(gen, n) * 1e-3).to(t) for t, n in total.items()}
        state["flat_out"] = {str(t): torch.empty_like(v) for t, v in flat.items()}
        at = dict.fromkeys(total, 0)
        for n, t in zip(sizes, types):
            state["grads"].append(flat[t][at[t]:at[t] + n])
            state["out"].append(state["flat_out"][str(t)][at[t]:at[t] + n])
            at[t] += n
        state["max_norm"] = 1e-3 * math.sqrt(sum(sizes)) / case["over"]
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    import fp8_block_scaled_quant_amd as fb

    case, op = state["case"], state["case"]["op"]
    if op == "ffn":
        return fb.gated_ffn(state["x"], state["wg"], state["wg_s"], state["wu"], state["wu_s"],
                            scale_fmt=case["fmt"] or None, save=case["save"])
    if op == "ffn_backward":
        return fb.gated_ffn_backward(state["dh"], state["x"], state["g"], state["u"], state["wg"], state["wg_s"],
                                     state["wu"], state["wu_s"])
    if op == "fp4_quant":
        return fb.fp4_weight_quant(state["w"])
    if op == "fp4_gemv":
        return fb.fp4_gemv(state["x"], state["q"], state["s"], out_dtype=TYPES[case["out"]], bias=state["bias"])
    norm = fb.clip_grad_norm(state["grads"], state["max_norm"], out=state["out"])
    return norm, state["flat_out"]


def _run_plain(state):
    case, op = state["case"], state["case"]["op"]
    if op == "ffn":
        xq = _quantized(state["x"].float(), case["fmt"])
        g = xq @ _dequantized(state["wg"], state["wg_s"]).T
        u = xq @ _dequantized(state["wu"], state["wu_s"]).T
        h = (g * torch.sigmoid(g) * u).to(torch.bfloat16)
        return (h, g.to(torch.bfloat16), u.to(torch.bfloat16)) if case["save"] else h
    if op == "ffn_backward":
        dh, g, u, x = (state[name].float() for name in ("dh", "g", "u", "x"))
        sig = torch.sigmoid(g)
        dg = dh * u * (sig * (1 + g * (1 - sig)))
        du = dh * (g * sig)
        dx = _quantized_pow2(dg) @ _dequantized(state["wg"], state["wg_s"])
        dx += _quantized_pow2(du) @ _dequantized(state["wu"], state["wu_s"])
        xq = _quantized_pow2_tokens(x)
        dwg = _quantized_pow2_tokens(dg).T @ xq
        dwu = _quantized_pow2_tokens(du).T @ xq
        return dx.to(torch.bfloat16), dwg.to(torch.bfloat16), dwu.to(torch.bfloat16)
    if op == "fp4_quant":
        return _fp4_codes(state["w"].float())
    if op == "fp4_gemv":
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
        q = state["q"].long()
        w = torch.stack([table[q & 15], table[q >> 4]], dim=-1).reshape(q.shape[0], -1, GROUP)
        w = (w * _power32(state["s"].int() - 127)[..., None]).reshape(q.shape[0], -1)
        y = state["x"].float() @ w.T
        if state["bias"] is not None:
            y = y + state["bias"].float()
        return y.to(TYPES[case["out"]])
    squares = [g.float().square().sum() for g in state["grads"]]
    norm = torch.stack(squares).sum().sqrt()
    factor = (state["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    [o.copy_(g.float() * factor) for g, o in zip(state["grads"], state["out"])]
    return norm, state["flat_out"]


def _power32(e):
    """2^e from its bits (exponents of normal values): torch's own powers are not exact everywhere."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _to_e4m3(v):
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()


def _quantized(x, fmt):
    """x after 1 x 128 E4M3 quantization: the values the codes and scales stand for."""
    b = x.view(x.shape[0], -1, BLOCK)
    # by a tensor: by a Python number torch multiplies with the rounded inverse
    s = b.abs().amax(-1, keepdim=True).clamp_min(1e-4) / b.new_tensor(448.0)
    if fmt == "ue8m0":
        part, e = torch.frexp(s)
        s = _power32(torch.where(part == 0.5, e - 1, e))
    return (_to_e4m3(b / s) * s).view_as(x)


def _quantized_pow2(x):
    """The same with s the smallest power of two such that amax <= 448 s."""
    b = x.view(x.shape[0], -1, BLOCK)
    part, e = torch.frexp(b.abs().amax(-1, keepdim=True).clamp_min(FLOOR))
    s = _power32(torch.where(part <= 0.875, e - 9, e - 8))
    return (_to_e4m3(b / s) * s).view_as(x)


def _quantized_pow2_tokens(x):
    """_quantized_pow2 with the blocks along the tokens, the last one filled up with zeros."""
    m = x.shape[0]
    x = torch.nn.functional.pad(x, (0, 0, 0, -m % BLOCK))
    return _quantized_pow2(x.T.contiguous()).T[:m]


def _dequantized(codes, scale):
    n, k = codes.shape
    wide = scale.repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]
    return codes.float() * wide


def _fp4_codes(w):
    """(two codes a byte, the even weight in the low half; E8M0 scales)."""
    b = w.view(w.shape[0], -1, GROUP)
    part, e = torch.frexp(b.abs().amax(-1, keepdim=True).clamp_min(FLOOR))
    e = torch.where(part <= 0.75, e - 3, e - 2)
    v = b / _power32(e)
    a = v.abs()
    # the number of rounding boundaries below; on a boundary, the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * torch.signbit(v)).to(torch.uint8).view(w.shape[0], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), (e[..., 0] + 127).to(torch.uint8)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    op, state = case["op"], prepare(case, seed)
    if op == "ffn":
        x = state["x"].double()
        top = x.unflatten(1, (-1, BLOCK)).abs().amax(2).clamp(min=1e-4)
        step = (top / 448).float().double()  # the format's scale, and the quotient it encodes, are FP32
        if case["fmt"] == "ue8m0":
            step = _power_above(step)
        step = step.repeat_interleave(BLOCK, 1)
        xq = _nearest_e4m3((x / step).float().double()) * step
        g = torch.matmul(xq, _weight64(state["wg"], state["wg_s"]).t())
        u = torch.matmul(xq, _weight64(state["wu"], state["wu_s"]).t())
        h = g / (1 + torch.exp(-g)) * u
        return (h, g, u) if case["save"] else h
    if op == "ffn_backward":
        dh, g, u = state["dh"].double(), state["g"].double(), state["u"].double()
        s = 1 / (1 + torch.exp(-g))
        dgu = torch.cat([dh * u * s * (1 + g - g * s), dh * g * s], 1)
        w = torch.cat([_weight64(state["wg"], state["wg_s"]), _weight64(state["wu"], state["wu_s"])])
        dx = torch.matmul(_blocks64(dgu), w)
        del w
        m, x = dh.shape[0], state["x"].double()
        fill = -(-m // BLOCK) * BLOCK - m
        tokens = lambda v: _blocks64(torch.cat([v, v.new_zeros(fill, v.shape[1])]).t().contiguous())  # noqa: E731
        dw = torch.matmul(tokens(dgu), tokens(x).t())
        f = dh.shape[1]
        return dx, dw[:f], dw[f:]
    if op == "fp4_quant":
        return None  # whole numbers only
    if op == "fp4_gemv":
        q, s = state["q"], state["s"]
        codes = torch.empty(q.shape[0], 2 * q.shape[1], dtype=torch.float64, device="cuda")
        codes[:, 0::2], codes[:, 1::2] = q.remainder(16), q.div(16, rounding_mode="floor")
        sign = torch.where(codes >= 8, -1.0, 1.0)
        mag = codes.remainder(8)
        mag = torch.where(mag < 2, mag / 2, (1 + mag.remainder(2) / 2) * _power64(torch.floor(mag / 2) - 1))
        w = sign * mag * _power64(s.long().repeat_interleave(GROUP, 1) - 127)
        y = torch.matmul(state["x"].double(), w.t())
        return y if state["bias"] is None else y + state["bias"].double()
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for g in state["grads"]:
        total += torch.linalg.vector_norm(g, dtype=torch.float64) ** 2
    norm = torch.sqrt(total)
    factor = torch.clamp(state["max_norm"] / (norm + 1e-6), max=1.0)
    flat = {name: torch.empty(v.shape, dtype=torch.float64, device="cuda") for name, v in state["flat_out"].items()}
    at = dict.fromkeys(flat, 0)
    for g in state["grads"]:
        name, n = str(g.dtype), g.numel()
        flat[name][at[name]:at[name] + n] = g.double() * factor
        at[name] += n
    return norm, flat


def _nearest_e4m3(v):
    """Nearest E4M3 value, ties to even, saturating: 2^-9 apart up to 2^-6, then eight steps a binade."""
    v = v.clamp(-448, 448)
    # frexp's exponent counts from 0.5, one above the binade's
    quantum = _power64(torch.frexp(v.abs().clamp(min=2.0 ** -6))[1] - 4)
    return torch.round(v / quantum) * quantum


def _power64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _power_above(v):
    """The smallest power of two that is not below v."""
    part, e = torch.frexp(v)
    return _power64(e - (part == 0.5).int())


def _blocks64(v):
    """1 x 128 blocks of v rounded to E4M3 under the smallest power-of-two scale that holds them."""
    top = v.unflatten(1, (-1, BLOCK)).abs().amax(2).clamp(min=FLOOR)
    step = _power_above(top / 448).repeat_interleave(BLOCK, 1)
    return _nearest_e4m3(v / step) * step


def _weight64(codes, scale):
    rows = torch.arange(codes.shape[0], device="cuda") // BLOCK
    cols = torch.arange(codes.shape[1], device="cuda") // BLOCK
    return codes.double() * scale.double()[rows][:, cols]
