"""The expert operators at the ends of their ranges: 2^31 choices less a few, the
products' most rows with the most experts, and what choices that take no part may
bring along."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from tests import expert_util as E
from tests import ffn_util as U
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


def _parts(n, part=1 << 27):
    return [slice(i, min(i + part, n)) for i in range(0, n, part)]


def test_most_choices():
    tokens, top_k, experts = (1 << 28) - 8, 8, 1000
    n = tokens * top_k   # 2^31 - 64
    G.announce(f"expert rows, {n} choices")
    gen = torch.Generator(G.device()).manual_seed(0)
    ids = torch.empty(n, dtype=torch.int32, device=G.device())
    for p in _parts(n):
        ids[p] = torch.randint(-1, experts, (p.stop - p.start,), generator=gen, device=G.device(), dtype=torch.int32)
    s = fb.expert_sort(ids.view(tokens, top_k), experts)
    torch.cuda.synchronize()
    G.announce("sorted")
    counts = sum(torch.bincount(ids[p] + 1, minlength=experts + 1) for p in _parts(n))
    assert torch.equal(s.offsets.long(), torch.cat([counts.new_zeros(1), counts[1:].cumsum(0)]))
    behind, rows, before = int(s.offsets[-1]), s.rows.view(-1), None
    for p in _parts(n):
        # the inverse of each other
        choice = torch.arange(p.start, p.stop, device=G.device(), dtype=torch.int32)
        at = torch.where(rows[p] < 0, ~rows[p], rows[p])
        assert torch.equal(s.choices[at], choice) and torch.equal(rows[p] < 0, at >= behind)
        # experts in order, and an expert's choices
        expert = ids[s.choices[p]]
        key = torch.where(expert < 0, experts, expert).long() << 32 | s.choices[p]
        if before is not None:
            assert before < key[0]
        assert bool((key[1:] > key[:-1]).all())
        before = key[-1].clone()
    del choice, at, expert, key
    x = torch.randn(tokens, 1, generator=gen, device=G.device()).bfloat16()
    y = fb.expert_dispatch(x, s.rows)
    torch.cuda.synchronize()
    G.announce("dispatched")
    for p in _parts(n):
        expert = s.choices[p] // top_k
        got, want = y[p, 0], x[expert, 0]
        last = max(0, min(behind - p.start, len(got)))
        assert torch.equal(got[:last], want[:last]) and not got[last:].any()
    # as many equal terms as take part: exact in FP32
    out = fb.expert_combine(y, s.rows)
    live = (s.rows >= 0).sum(1, keepdim=True)
    assert torch.equal(out, (x.float() * live).bfloat16())
    dy, dw = fb.expert_combine_backward(x, y, s.rows)
    torch.cuda.synchronize()
    G.announce("gradients")
    assert torch.equal(dy, y)   # ones for weights
    for p in _parts(tokens, 1 << 24):
        assert torch.equal(dw[p], torch.where(s.rows[p] >= 0, x[p].float() ** 2, 0.0))
    del ids, s, rows, x, y, out, dy, dw, live
    torch.cuda.empty_cache()


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("n", [24, 300])
def test_most_rows_of_most_experts(n, gated):
    """One K block: each product is exact in FP32 but for the instruction's own sums."""
    rows, experts, k = 65535 * 16, 1024, 128
    G.announce(f"expert products, {rows} rows of {experts} experts, n={n} gated={gated}")
    gen = torch.Generator(G.device()).manual_seed(n)
    cuts = torch.randint(0, rows - 100, (experts - 1,), generator=gen, device=G.device()).sort().values
    offsets = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), rows - 100)]).int()

    def codes(*shape):
        c = torch.randint(0, 0x60, shape, dtype=torch.uint8, generator=gen, device=G.device())
        return c | torch.randint(0, 2, shape, dtype=torch.uint8, generator=gen, device=G.device()) << 7

    a, a_s = codes(rows, k), torch.rand(rows, 1, generator=gen, device=G.device()) * 0.01
    ws = [(codes(experts, n, k), torch.rand(experts, -(-n // 128), 1, generator=gen, device=G.device()) * 0.01) for _ in range(2 if gated else 1)]
    got = (fb.expert_gated_ffn if gated else fb.expert_gemm)(a, a_s, offsets, *[t for w in ws for t in w], out_dtype=torch.float32)
    assert not got[rows - 100:].any()
    at, value = offsets.tolist(), lambda c: c.view(torch.float8_e4m3fn).float().double()  # noqa: E731
    for e in range(experts):
        p = slice(at[e], at[e + 1])
        if p.start == p.stop:
            continue
        left, products = value(a[p]) * a_s[p].double(), []
        for w, w_s in ws:
            right = value(w[e]) * w_s[e].double().repeat_interleave(128, 0)[:n]
            products.append((left @ right.t(), 1e-3 * (left.abs() @ right.abs().t())))
        (g, dg), want, off = products[0], products[0][0], products[0][1]
        if gated:
            u, du = products[1]
            silu = g * torch.sigmoid(g)
            want, off = silu * u, 1.1 * dg * u.abs() + silu.abs() * du + 1.1 * dg * du + (silu * u).abs() * 2.0 ** -20
        assert bool(((got[p].double() - want).abs() <= off + want.abs() * 2.0 ** -24 + 1e-30).all()), e
    del a, got
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_choices_that_take_no_part_bring_nothing(kind):
    """Their weights, and what their tokens hold, may be anything."""
    tokens, top_k, h = 12, 3, 256
    ids = E.choices(3, tokens, top_k, 5, 0.4)
    ids[4] = -1   # a token with no expert at all
    rows = U.gpu(E.sort(ids, 5)[1])
    out_of = rows < 0
    x, w = E.normal(1, (tokens, h), kind).to(G.device()), E.normal(2, (tokens, top_k), "f32").to(G.device())
    y = fb.expert_dispatch(x, rows)
    clean = [fb.expert_combine(y, rows, w), *fb.expert_combine_backward(x, y, rows, w)]
    assert not clean[0][4].any() and not clean[2][out_of].any()
    for bad in (float("nan"), float("inf")):
        dirty = torch.where(out_of, bad, w)
        assert all(torch.equal(p, q) for p, q in zip([fb.expert_combine(y, rows, dirty), *fb.expert_combine_backward(x, y, rows, dirty)], clean))
        # the token with no expert: its row reaches no output
        lost = x.clone()
        lost[4] = bad
        assert torch.equal(fb.expert_dispatch(lost, rows), y)
        assert all(torch.equal(p, q) for p, q in zip(fb.expert_combine_backward(lost, y, rows, w), clean[1:]))
        for fmt in (None, "ue8m0"):
            assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8))
                       for p, q in zip(fb.expert_dispatch_quant(lost, rows, fmt), fb.expert_dispatch_quant(x, rows, fmt)))
