"""4-bit weights at what one launch can take in threads and beyond: the quantizer on
2^35 weights and some, sampled on both sides of where one launch ends and the next
begins, and the product with as many weight rows as it takes."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from oracle import fp4
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()


def test_quantizer_past_2_to_the_35():
    n, k = (1 << 20) + 5, 1 << 15
    G.announce(f"fp4_weight_quant {n} x {k} bf16 ({n * k / 2 ** 30:.1f} Gi weights)")
    w = torch.empty(n, k, dtype=torch.bfloat16, device=G.device())
    # every row a shift of the same values, so that neighbours differ
    row = torch.randn(2 * k, generator=torch.Generator().manual_seed(0)).bfloat16().to(G.device())
    for at in range(0, n, 1 << 16):
        w[at:at + (1 << 16)] = row[:k]
    rows = np.unique([0, 1, n // 2 - 1, n // 2, (1 << 19) - 1, 1 << 19, (1 << 19) + 1, (1 << 20) - 1, 1 << 20, (1 << 20) + 1, n - 1])
    for i, r in enumerate(rows):
        w[r] = row[17 * i + 1:17 * i + 1 + k]
    q, s = fb.fp4_weight_quant(w)
    for r in rows:
        codes, scales = fp4.weight_quant(w[r:r + 1].float().cpu().numpy())
        assert np.array_equal(q[r:r + 1].cpu().numpy(), codes) and np.array_equal(s[r:r + 1].cpu().numpy(), scales), r
    # all others hold the same row: none was left out
    codes, scales = fb.fp4_weight_quant(row[:k].view(1, k))
    marked = torch.zeros(n, dtype=torch.bool, device=w.device)
    marked[torch.from_numpy(rows).to(w.device)] = True
    for at in range(0, n, 1 << 16):
        same = (s[at:at + (1 << 16)] == scales).all(1) & (q[at:at + (1 << 16)] == codes).all(1)
        assert bool((same | marked[at:at + (1 << 16)]).all()), at


def test_gemv_with_the_most_rows():
    n, k = 144 * ((1 << 22) - 1), 32
    G.announce(f"fp4_gemv 1 x {n} x {k}")
    gen = torch.Generator(G.device()).manual_seed(1)
    x = torch.randn(1, k, generator=gen, device=G.device()).bfloat16()
    q = torch.zeros(n, k // 2, dtype=torch.uint8, device=G.device())
    first = torch.randint(256, (1 << 20,), generator=gen, device=G.device(), dtype=torch.uint8)
    for at in range(0, n, 1 << 20):
        q[at:at + (1 << 20), 3] = first[:min(1 << 20, n - at)]
    s = torch.full((n, 1), 127, dtype=torch.uint8, device=G.device())
    y = fb.fp4_gemv(x, q, s, torch.float32)
    byte = torch.arange(256)
    values = torch.from_numpy(fp4.DECODE).float()
    table = (values[byte & 15] * x[0, 6].float().cpu() + values[byte >> 4] * x[0, 7].float().cpu()).to(x.device)
    for at in range(0, n, 1 << 20):   # two exact products: one rounding
        want = table[first[:min(1 << 20, n - at)].long()]
        got = y[0, at:at + (1 << 20)]
        assert bool(((got - want).abs() <= 2.0 ** -23 * want.abs()).all()), at
