"""Gradients at the ends of the value range: finite inputs whose gradients have
finite values do not pass through infinities on the way."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from oracle import ffn
from tests import ffn_util as U
from tests import gpu_util as G
from tests.test_gpu_gated_ffn_backward import _check, _inputs, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m", [40, 4200])
def test_large_gradients_behind_closed_gates(m):
    """dh u above fp32's range where the gate's slope is zero to fp32's precision:
    the gradient is 0 there, in a block whose other values are ordinary."""
    f, k = (128, 128) if m == 40 else (1024, 128)
    acts, wg, wu = _inputs(m, f, k, "f32", 1.0)
    dh, _, g, u = acts
    g[:, 3], g[::2, 70] = -200.0, -1e4
    dh[:, 3], dh[::2, 70] = 2.0 ** 90, 2.0 ** 10
    u[:, 3], u[::2, 70] = -2.0 ** 60, 2.0 ** 120
    got = _run(acts, wg, wu, out_dtype=torch.float32)
    assert all(torch.isfinite(t).all() for t in got)
    _check(acts, wg, wu, got, "f32")


def test_long_sums_of_one_sign():
    """dW over 131,072 tokens whose terms all have one sign: a sum that lost its low
    bits on the way would drift, block by block.  Each of the 1024 blocks rounds
    twice (its own sum, and the running one): 2^-14 at most, and the E4M3 values of
    the two operands are the oracle's."""
    m, f, k = 1 << 17, 128, 256
    gen = torch.Generator(G.device()).manual_seed(0)
    rand = lambda n: (torch.rand(m, n, generator=gen, device=G.device()) + 0.25).bfloat16()  # noqa: E731
    dh, x, g, u = rand(f), rand(k), rand(f), rand(f)
    weights = [U.gpu(v) for seed in (1, 2) for v in U.weight(seed, f, k)]
    _, *dw = fb.gated_ffn_backward(dh, x, g, u, *weights, out_dtype=torch.float32, input_grad=False)
    feats = np.array([0, 5, f - 1])
    xq = ffn.quantize_tokens(U.values(x))
    for have, v in zip(dw, ffn.activation_grads(*[U.values(t[:, feats]) for t in (dh, g, u)])):
        want = ffn.quantize_tokens(v).T @ xq
        # an E4M3 rounding taken to the other side costs an eighth of one of the terms: 1e-4 of the sum for a hundred
        assert np.all(np.abs(U.values(have[feats]) - want) <= (2.0 ** -13 + 1e-4) * want)
