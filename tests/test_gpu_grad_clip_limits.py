"""clip_grad_norm where the factor's quotient has no value: nothing is above the
bound there, so nothing is scaled."""

import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_infinite_bound_leaves_infinite_gradients(dtype):
    g = torch.tensor([1.0, -INF, 3.0], device=G.device(), dtype=dtype)
    before, out = g.clone(), torch.zeros_like(g)
    assert float(fb.clip_grad_norm([g], INF, out=[out])) == INF and torch.equal(out, before)
    assert float(fb.clip_grad_norm([g], INF)) == INF and torch.equal(g, before)


def test_infinite_norm_of_finite_gradients():
    """A norm above fp32's range: infinite, and below an infinite bound."""
    g = torch.full((4,), 3e38, device=G.device())
    before = g.clone()
    assert float(fb.clip_grad_norm([g], INF)) == INF and torch.equal(g, before)
    assert float(fb.clip_grad_norm([g], 1.0)) == INF and not g.any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_zeros_under_a_zero_bound(dtype):
    g = torch.zeros(70, device=G.device(), dtype=dtype)
    out = torch.ones_like(g)
    assert float(fb.clip_grad_norm([g], 0.0, out=[out], eps=0.0)) == 0.0 and not out.any()
    assert float(fb.clip_grad_norm([g], 0.0, eps=0.0)) == 0.0 and not g.any()


def test_nan_is_kept_under_any_bound():
    for bound in (0.0, 1.0, INF):
        g = torch.tensor([1.0, float("nan")], device=G.device())
        assert torch.isnan(fb.clip_grad_norm([g], bound)) and torch.isnan(g).all()
