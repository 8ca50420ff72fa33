"""Clipping writes tensors that autograd may have saved: like torch's own in-place
operations it marks them changed, so that a later backward pass refuses them."""

import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


def _saved():
    """A tensor and a product that saved it for its backward pass."""
    w = torch.ones(8, device=G.device(), requires_grad=True)
    g = torch.full((8,), 2.0, device=G.device())
    return g, (w * g).sum()


def test_clipped_in_place_is_marked_changed():
    g, loss = _saved()
    before = g._version
    fb.clip_grad_norm([g], 0.5)
    assert g._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_outputs_are_marked_changed_and_inputs_are_not():
    (src, src_loss), (out, out_loss) = _saved(), _saved()
    fb.clip_grad_norm([src], 0.5, out=[out])
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out_loss.backward()
    src_loss.backward()


def test_norm_changes_nothing():
    g, loss = _saved()
    before = g._version
    assert float(fb.grad_norm([g])) > 0 and g._version == before
    loss.backward()


def test_inference_tensors_have_no_version():
    with torch.inference_mode():
        g = torch.full((8,), 2.0, device=G.device())
        fb.clip_grad_norm([g], 0.5)
        assert abs(float(g.norm()) - 0.5) < 1e-5
