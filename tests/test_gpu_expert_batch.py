"""What a token's output owes to the tokens that come with it: nothing up to K = 512, bit
for bit; from K = 640 on its last bits can change with their number, since few tiles are
added up by another kernel in another order, and both results meet the bound."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from tests import expert_util as E
from tests import ffn_util as U
from tests import gpu_util as G
from tests.test_gpu_expert_products import _tolerance
from tests.test_gpu_expert_shapes import CASES, SIZES, _device, _host
from tests.test_gpu_experts_module import _layer, _reference

pytestmark = pytest.mark.gpu


def _alone(case, args, e, rows):
    """The call with these of expert e's rows alone, and no other expert."""
    a, a_s, offsets, *w = args
    only = torch.tensor([0, len(rows)], dtype=torch.int32, device=G.device())
    at = torch.from_numpy(rows).to(G.device())
    w = [v[e:e + 1] for v in w]
    return (fb.expert_gated_ffn if case[0] else fb.expert_gemm)(a[at], a_s[at], only, *w, out_dtype=torch.float32)


@pytest.mark.parametrize("case", [c for c in CASES if c[4] <= 512 and SIZES[c] != "few"], ids=lambda c: f"{SIZES[c]}-{c[0]}-{c[3]}x{c[4]}")
def test_rows_are_independent_up_to_four_blocks(case):
    """From the kernel for many rows to that for one, the same bits."""
    G.announce(f"experts' rows alone {SIZES[case]} {case[0]} {case[3]} x {case[4]}")
    args, offsets = _device(case), _host(case)[0]
    got = (fb.expert_gated_ffn if case[0] else fb.expert_gemm)(*args, out_dtype=torch.float32)
    for e in np.flatnonzero(np.diff(offsets))[:6]:
        for rows in (np.array([offsets[e]]), np.array([offsets[e + 1] - 1]), np.arange(offsets[e], offsets[e + 1])[:40]):
            assert torch.equal(_alone(case, args, int(e), rows), got[torch.from_numpy(rows).to(got.device)])


@pytest.mark.parametrize("case", [c for c in CASES if SIZES[c] == "many" and c[4] >= 640 and not c[0]], ids=lambda c: f"{c[3]}x{c[4]}")
def test_rows_alone_meet_the_bound_beyond(case):
    G.announce(f"experts' rows alone, {case[3]} x {case[4]}")
    args, (offsets, a, a_s, w, _) = _device(case), _host(case)
    got = fb.expert_gemm(*args, out_dtype=torch.float32)
    for e in np.flatnonzero(np.diff(offsets))[:6]:
        rows = np.arange(offsets[e], offsets[e + 1])[:5]
        off = _tolerance(a[rows], a_s[rows], np.array([0, len(rows)]), w[0][e:e + 1], w[1][e:e + 1])
        E.within(_alone(case, args, int(e), rows), U.values(got[torch.from_numpy(rows).to(got.device)]), 2 * off)


@pytest.mark.parametrize("k,f", [(512, 384), (768, 640)])
def test_layer(k, f):
    """The token alone and among others: one output, to the bits or within both bounds."""
    G.announce(f"Experts, a token alone and among others, {k} x {f}")
    tokens, top_k, experts = 40, 2, 5
    layer = _layer(9, experts, k, f, "f32", None)
    ids, x = E.choices(3, tokens, top_k, experts, 0.1), E.normal(4, (tokens, k), "f32").to(G.device())
    w = torch.softmax(E.normal(5, (tokens, top_k), "f32"), 1).to(G.device())
    together = layer(x, U.gpu(ids), w)
    # others in their place, and as many: the same bits, whatever K
    for t in (0, 17, tokens - 1):
        others = np.random.default_rng(t).permutation(np.delete(np.arange(tokens), t))
        others = np.insert(others, t, t)
        at = torch.from_numpy(others).to(G.device())
        assert torch.equal(layer(x[at], U.gpu(ids[others]), w[at])[t], together[t])
    alone = torch.cat([layer(x[t:t + 1], U.gpu(ids[t:t + 1]), w[t:t + 1]) for t in range(tokens)])
    if k <= 512 and f <= 512:
        assert torch.equal(alone, together)
    out, off = _reference(layer, U.values(x), ids, U.values(w))
    E.within(together, out, off)
    E.within(alone, out, off)
