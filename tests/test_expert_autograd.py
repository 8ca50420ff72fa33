"""``expert_dispatch``'s and ``expert_combine``'s place in autograd, on the CPU: the
native calls under them are replaced by float64 arithmetic on the same arguments, so
that what is tested is which gradients are handed on, and what is refused."""

import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from fp8_block_scaled_quant_amd import _ffn_lib
from tests import expert_util as E

TOKENS, TOP_K, EXPERTS, H = 7, 3, 4, 5


class _Native:
    """The binding's functions, in torch; None where autograd has to see the call."""

    @staticmethod
    def _tracked(*tensors):
        return torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors)

    def expert_dispatch(self, x, rows, ask):
        if ask and self._tracked(x):
            return None
        assert x.is_contiguous()
        with torch.no_grad():
            y = x.new_zeros(rows.numel(), x.shape[1])
            for j in range(rows.shape[1]):
                live = rows[:, j] >= 0
                y[rows[live, j].long()] = x[live]
            return y

    def expert_combine(self, y, rows, weights, ask):
        if ask and self._tracked(y, weights):
            return None
        assert y.is_contiguous()
        with torch.no_grad():
            live = (rows >= 0)[..., None]
            terms = torch.where(live, y[rows.clamp(min=0).long()], 0.0)
            return (terms if weights is None else terms * weights[..., None]).sum(1)

    def expert_combine_backward(self, dout, y, rows, weights, row_grad, weight_grad):
        assert dout.is_contiguous() and not (weights is None and weight_grad)
        with torch.no_grad():
            live, at = rows >= 0, rows.clamp(min=0).long()
            dy = torch.zeros_like(y) if row_grad else None
            if row_grad:
                for t, j in live.nonzero().tolist():
                    dy[rows[t, j]] = weights[t, j] * dout[t]
            dw = torch.where(live, (dout[:, None] * y[at]).sum(-1), 0.0) if weight_grad else None
            return dy, dw


@pytest.fixture
def rows(monkeypatch):
    native = _Native()
    monkeypatch.setattr(_ffn_lib, "ext", lambda: native)
    torch.manual_seed(0)
    return torch.from_numpy(E.sort(E.choices(1, TOKENS, TOP_K, EXPERTS, 0.3), EXPERTS)[1])


def _leaf(*shape):
    return torch.randn(*shape, dtype=torch.float64, requires_grad=True)


def test_first_order(rows):
    x, y, w = _leaf(TOKENS, H), _leaf(TOKENS * TOP_K, H), _leaf(TOKENS, TOP_K)
    assert torch.autograd.gradcheck(lambda x: fb.expert_dispatch(x, rows), x)
    assert torch.autograd.gradcheck(lambda y: fb.expert_combine(y, rows), y)
    assert torch.autograd.gradcheck(lambda y, w: fb.expert_combine(y, rows, w), (y, w))
    assert torch.autograd.gradcheck(lambda y: fb.expert_combine(y, rows, w.detach()), y)
    assert torch.autograd.gradcheck(lambda w: fb.expert_combine(y.detach(), rows, w), w)


def test_second_order_exists_without_weights_alone(rows):
    x, y, w = _leaf(TOKENS, H), _leaf(TOKENS * TOP_K, H), _leaf(TOKENS, TOP_K)
    assert torch.autograd.gradgradcheck(lambda x: fb.expert_dispatch(x, rows), x)
    assert torch.autograd.gradgradcheck(lambda y: fb.expert_combine(y, rows), y)
    for inputs in ((y, w), (y, w.detach()), (y.detach(), w)):
        wanted = [t for t in inputs if t.requires_grad]
        grads = torch.autograd.grad(fb.expert_combine(inputs[0], rows, inputs[1]).sum(), wanted, create_graph=True)
        for g in grads:
            with pytest.raises(RuntimeError, match="second-order"):
                g.sum().backward(retain_graph=True)


def test_gradients_reach_what_comes_before_and_no_more(rows):
    x, scale = _leaf(TOKENS, H), _leaf(TOKENS, TOP_K)
    out = fb.expert_combine(torch.tanh(fb.expert_dispatch(x, rows)), rows, torch.softmax(scale, 1))
    gx, gs = torch.autograd.grad(out.square().sum(), (x, scale))
    live = (rows >= 0)[..., None]
    dense = (torch.where(live, torch.tanh(x)[:, None].expand(-1, TOP_K, -1), 0.0) * torch.softmax(scale, 1)[..., None]).sum(1)
    for got, want in zip((gx, gs), torch.autograd.grad(dense.square().sum(), (x, scale))):
        assert torch.allclose(got, want, rtol=1e-12, atol=1e-12)
    with torch.no_grad():
        assert fb.expert_combine(fb.expert_dispatch(x, rows), rows, scale).grad_fn is None
    assert fb.expert_dispatch(x.detach(), rows).grad_fn is None
