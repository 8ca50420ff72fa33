"""``GatedFFN``'s place in autograd, on the CPU: the three native calls under it
are replaced by float64 arithmetic on the same arguments, so that what is tested
is which gradients the module hands on, and what it refuses.
"""

import pytest
import torch
from torch.autograd import forward_ad

from fp8_block_scaled_quant_amd import ffn


@torch.no_grad()
def _forward(x, wg, wg_s, wu, wu_s, scale_fmt=None, out_dtype=torch.bfloat16, save=False):
    assert x.is_contiguous() and x.data_ptr() % 16 == 0
    g, u = x.double() @ wg.T, x.double() @ wu.T
    out = [t.to(out_dtype) for t in (g * torch.sigmoid(g) * u, g, u)]
    return tuple(out) if save else out[0]


@torch.no_grad()
def _backward(dh, x, g, u, wg, wg_s, wu, wu_s, out_dtype=torch.bfloat16, input_grad=True, weight_grad=True):
    assert all(t.is_contiguous() and t.data_ptr() % 16 == 0 for t in (dh, x, g, u))
    dh, x, g, u = (t.double() for t in (dh, x, g, u))
    s = torch.sigmoid(g)
    dg, du = dh * u * s * (1 + g * (1 - s)), dh * g * s
    dx = (dg @ wg + du @ wu).to(out_dtype) if input_grad else None
    return dx, *((t.T @ x).to(out_dtype) if weight_grad else None for t in (dg, du))


@pytest.fixture
def module(monkeypatch):
    monkeypatch.setattr(ffn, "weight_quant", lambda w: (w.detach().double(), torch.ones(1, 1)))
    monkeypatch.setattr(ffn, "gated_ffn", _forward)
    monkeypatch.setattr(ffn, "gated_ffn_backward", _backward)
    torch.manual_seed(0)
    return ffn.GatedFFN(128, 128, torch.float32)


def _x(requires_grad=True):
    return torch.randn(5, 128, generator=torch.Generator().manual_seed(1)).requires_grad_(requires_grad)


def _reference(module, x):
    w = [p.detach().clone().requires_grad_() for p in (module.w_gate, module.w_up)]
    x = x.detach().clone().requires_grad_()
    return torch.nn.functional.silu(x @ w[0].T) * (x @ w[1].T), [x, *w]


@pytest.mark.parametrize("create_graph", [False, True])
def test_first_order_gradients(module, create_graph):
    x = _x()
    got = torch.autograd.grad(module(x).square().sum(), [x, module.w_gate, module.w_up], create_graph=create_graph)
    h, leaves = _reference(module, x)
    for have, want in zip(got, torch.autograd.grad(h.square().sum(), leaves)):
        torch.testing.assert_close(have.detach(), want, rtol=1e-4, atol=1e-4)


# a loss linear in h hands the backward pass a constant dh
@pytest.mark.parametrize("loss", [torch.sum, lambda h: h.square().sum()])
def test_second_order_gradients_raise(module, loss):
    x = _x()
    h = module(x)
    dx, = torch.autograd.grad(loss(h), x, create_graph=True)
    with pytest.raises(RuntimeError, match="second-order"):
        (h.sum() + dx.square().sum()).backward()
    dw, = torch.autograd.grad(loss(module(x.detach())), module.w_up, create_graph=True)
    with pytest.raises(RuntimeError, match="second-order"):
        dw.sum().backward()


@pytest.mark.parametrize("grad_mode", [True, False])
def test_forward_mode_raises(module, grad_mode):
    with forward_ad.dual_level(), torch.set_grad_enabled(grad_mode):
        x = forward_ad.make_dual(_x(False), torch.ones(5, 128))
        with pytest.raises(NotImplementedError):
            module(x)


def test_without_gradients(module):
    x = _x()
    with torch.no_grad():
        h = module(x)
    assert not h.requires_grad and torch.equal(h, module(x).detach())
    with torch.inference_mode():
        assert torch.equal(module(x), h)


def test_only_the_gradients_asked_for(module):
    module.w_gate.requires_grad_(False)
    module(_x(False)).sum().backward()
    assert module.w_gate.grad is None and module.w_up.grad is not None
    module.w_up.requires_grad_(False)
    x = _x()
    module(x).sum().backward()
    assert x.grad is not None


def test_views_that_start_anywhere(module):
    """x one element into a buffer; h joined behind one element, whose gradient is
    then a contiguous view one element into another."""
    x = _x(False)
    shifted = torch.cat([torch.zeros(1), x.flatten()])[1:].view(5, 128).requires_grad_()
    assert shifted.is_contiguous() and shifted.data_ptr() % 16
    weights = torch.randn(5 * 128, generator=torch.Generator().manual_seed(2))
    joined = torch.cat([torch.zeros(1), module(shifted).flatten()])
    (joined * torch.cat([torch.zeros(1), weights])).sum().backward()
    h, leaves = _reference(module, x)
    (h.flatten() * weights).sum().backward()
    for have, want in zip((shifted, module.w_gate, module.w_up), leaves):
        torch.testing.assert_close(have.grad, want.grad, rtol=1e-4, atol=1e-4)
    with torch.no_grad():
        assert torch.equal(module(shifted), module(x))


def test_views_that_are_not_contiguous(module):
    x = torch.randn(128, 5).t().requires_grad_()
    h = module(x)
    h.t().contiguous().square().sum().backward()
    ref, leaves = _reference(module, x)
    ref.square().sum().backward()
    torch.testing.assert_close(x.grad, leaves[0].grad, rtol=1e-4, atol=1e-4)
