"""fp4_gemv at the ends of its values' ranges.

A row of one nonzero weight and one nonzero x makes one product: exact, and the
sums with zeros exact too.  Below |x| = 2^-110 an fp32 x keeps its bits down to
bf16's smallest value, 2^-133.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from oracle import fp4
from tests import ffn_util as U
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


def _one_product(x, codes, scale_bytes):
    """x times every code of a column, one row each, under the row's scale."""
    q = np.zeros((len(codes), 16), np.uint8)
    q[:, 2] = np.asarray(codes) << 4                       # weight 5
    s = np.asarray(scale_bytes, np.uint8).reshape(-1, 1)
    xs = torch.zeros(1, 32, dtype=x.dtype)
    xs[0, 5] = x
    got = U.values(fb.fp4_gemv(xs.to(G.device()), U.gpu(q), U.gpu(s), torch.float32))[0]
    return got, fp4.dequant(q, s)[:, 5]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_every_scale(dtype):
    """All codes under all scale bytes whose products with 6 are finite: weights
    down to 2^-128, subnormal in bf16."""
    codes, scales = (v.ravel() for v in np.meshgrid(np.arange(16), np.arange(253)))
    got, w = _one_product(torch.ones((), dtype=dtype), codes, scales)
    assert np.array_equal(got, w) and np.isfinite(got).all()


def test_quantized_weights_at_the_top():
    """Weights up to 6 * 2^125 survive quantizer and product; x brings them back into range."""
    rng = np.random.default_rng(0)
    w = (rng.uniform(-1, 1, (40, 64)) * 6 * 2.0 ** 125).astype(np.float32)
    w[:, 0] = np.float32(6 * 2.0 ** 125)
    q, s = fb.fp4_weight_quant(U.gpu(w))
    assert int(s.max()) == 252
    x = (rng.standard_normal((3, 64)) * 2.0 ** -100).astype(np.float32)
    deq = fp4.dequant(q.cpu().numpy(), s.cpu().numpy())
    want, terms = x.astype(np.float64) @ deq.T, np.abs(x).astype(np.float64) @ np.abs(deq).T
    assert np.all(np.abs(U.values(fb.fp4_gemv(U.gpu(x), q, s, torch.float32)) - want) <= 64 * 2.0 ** -24 * terms + np.abs(want) * 2.0 ** -23)


@pytest.mark.parametrize("exponent", [-110, -109, -60, 0, 100])
def test_fp32_x_is_whole(exponent):
    for significand in (0xFFFFFF, 0x800001, 0xAAAAAB, 0x923456):
        for code in range(1, 5):                           # 0.5, 1, 1.5, 2
            x = torch.tensor(significand * 2.0 ** (exponent - 23), dtype=torch.float64).float()
            if code == 3:                                  # 1.5: whole if x has a bit to spare
                x = (x.view(torch.int32) & -2).view(torch.float32)
            got, w = _one_product(x, [code], [128])
            exact = float(x) * w
            assert abs(got[0] - exact[0]) <= abs(exact[0]) * 2.0 ** -24 * (code == 3)


@pytest.mark.parametrize("exponent", [-111, -118, -126, -130, -140, -149])
def test_tiny_fp32_x_keeps_what_bf16_reaches(exponent):
    for significand in (1.0, 1 + 2.0 ** -10, 2 - 2.0 ** -23):
        x = torch.tensor(significand * 2.0 ** exponent, dtype=torch.float64).float()
        got, w = _one_product(x, [2], [200])
        assert abs(got[0] - float(x) * w[0]) <= 2.0 ** -133 * w[0]


def test_tiny_bf16_x_is_whole():
    for exponent in range(-133, -100):
        x = torch.tensor(2.0 ** exponent, dtype=torch.float64).to(torch.bfloat16)
        got, w = _one_product(x, [2], [200])
        assert got[0] == 2.0 ** exponent * w[0] != 0
