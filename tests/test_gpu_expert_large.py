"""The expert operators where offsets pass 32 bits: sorted rows, weights and outputs
of 4 GiB and more, on sampled rows."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_quant_amd as fb
import oracle
from oracle import experts as want
from tests import expert_util as E
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


def _codes(gen, *shape):
    """Finite E4M3 codes: all but the NaNs 0x7F and 0xFF."""
    out = torch.randint(0, 256, shape, dtype=torch.uint8, generator=gen, device=G.device())
    for part in out.view(-1).split(1 << 28):   # bounded scratch
        part.sub_(((part & 0x7F) == 0x7F).to(torch.uint8))
    return out


def _scales(gen, *shape):
    return torch.rand(shape, generator=gen, device=G.device()) * 0.01 + 1e-3


# tiles of 256 rows over a > 4 GiB; of 64 over a > 4 GiB; weights > 4 GiB, few rows; outputs > 2^32 elements
@pytest.mark.parametrize("experts,each,n,k", [(4, 150100, 40, 7168), (1024, 40, 24, 131072), (40, 3, 16000, 7168), (3, 100100, 14336, 128)])
def test_products(experts, each, n, k):
    G.announce(f"expert_gemm large {experts} x {each} n={n} k={k}")
    gen = torch.Generator(G.device()).manual_seed(n)
    rows = experts * each
    a, a_s, w, w_s = _codes(gen, rows, k), _scales(gen, rows, k // 128), _codes(gen, experts, n, k), _scales(gen, experts, -(-n // 128), k // 128)
    offsets = torch.arange(0, rows + 1, each, dtype=torch.int32, device=G.device())
    got = fb.expert_gemm(a, a_s, offsets, w, w_s)
    for e in sorted({0, experts // 2, experts - 1}):
        picked = [e * each + r for r in sorted({0, each // 2, each - 1})]
        cols = np.unique(np.r_[0, n - 1, np.random.default_rng(e).integers(0, n, 30)]) if n > 128 else np.arange(n)
        ah, sh = a[picked].cpu().numpy(), a_s[picked].cpu().numpy()
        for col in cols:   # a weight row at a time, with its block's scales
            b, b_s = w[e, col:col + 1].cpu().numpy(), w_s[e, col // 128:col // 128 + 1].cpu().numpy()
            c = oracle.fp8_gemm(ah, sh, b, b_s)
            E.within(got[picked, col:col + 1], c, oracle.gemm_tolerance(ah, sh, b, b_s) * (1 + 2.0 ** -8) + np.abs(c) * 2.0 ** -8)
    del a, w, got
    torch.cuda.empty_cache()


def test_rows():
    tokens, top_k, h, experts = 66000, 8, 8320, 64   # 4.39e9 elements in sorted order
    G.announce(f"expert rows large {tokens} x {top_k} x {h}")
    ids = np.random.default_rng(0).integers(-1, experts, (tokens, top_k))
    s = fb.expert_sort(torch.from_numpy(ids).to(G.device()), experts)
    rows = s.rows.cpu().numpy()
    assert np.array_equal(rows, E.sort(ids, experts)[1])
    gen = torch.Generator(G.device()).manual_seed(1)
    x = torch.randn(tokens, h, generator=gen, device=G.device(), dtype=torch.bfloat16)
    w = torch.rand(tokens, top_k, generator=gen, device=G.device())
    y = fb.expert_dispatch(x, s.rows)
    at = np.where(rows < 0, ~rows, rows)
    last = np.unravel_index(np.argsort(at, axis=None)[-3:], at.shape)[0]   # the tokens of the last rows
    some = np.unique(np.r_[0, tokens - 1, last, np.random.default_rng(1).integers(0, tokens, 20)])
    for t in some:
        live = torch.from_numpy(rows[t] >= 0).to(G.device())[:, None]
        assert torch.equal(y[at[t]], torch.where(live, x[t], torch.zeros_like(x[t])))
    codes, scales = fb.expert_dispatch_quant(x, s.rows)
    ref_codes, ref_scales = fb.act_quant(x[some].contiguous())
    for i, t in enumerate(some):
        for r in rows[t][rows[t] >= 0]:
            assert torch.equal(codes[r].view(torch.uint8), ref_codes[i].view(torch.uint8)) and torch.equal(scales[r], ref_scales[i])
    del codes, scales
    out = fb.expert_combine(y, s.rows, w)
    dy, dw = fb.expert_combine_backward(x, y, s.rows, w)
    for t in some:
        mine = np.arange(top_k)[None]
        sub = np.where(rows[t] >= 0, mine, ~mine).reshape(1, top_k)
        yv, xv, wv = (v.float().double().cpu().numpy() for v in (y[at[t]], x[t:t + 1], w[t:t + 1]))
        c, size = want.combine(yv, sub, wv)
        E.within(out[t:t + 1], c, size * (top_k * 2.0 ** -24 + 2.0 ** -8 * (1 + 2.0 ** -20)) + E.LEAST["bf16"])
        gy, gw, gsize = want.combine_backward(xv, yv, sub, wv)
        E.within(dy[at[t]], gy, np.abs(gy) * (2.0 ** -24 + 2.0 ** -8 * (1 + 2.0 ** -20)) + E.LEAST["bf16"])
        E.within(dw[t:t + 1], gw, gsize * h * 2.0 ** -24 + E.LEAST["f32"])
    del y, dy, x
    torch.cuda.empty_cache()
