"""expert_dispatch's and expert_combine's place in autograd: gradients equal the
operators' own and the differences of these (bi)linear functions, to the order that
exists; what does not exist raises."""

import pytest
import torch
from torch.autograd import forward_ad

import fp8_block_scaled_quant_amd as fb
from tests import expert_util as E
from tests import ffn_util as U
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

TOKENS, TOP_K, EXPERTS, H = 21, 3, 5, 72


def _case(kind="f32", drop=0.25):
    _, rows, _ = E.sort(E.choices(1, TOKENS, TOP_K, EXPERTS, drop), EXPERTS)
    make = lambda seed, *shape: E.normal(seed, shape, kind).to(G.device()).requires_grad_()  # noqa: E731
    return U.gpu(rows), make(2, TOKENS, H), make(3, TOKENS * TOP_K, H), E.normal(4, (TOKENS, TOP_K), "f32").to(G.device()).requires_grad_()


def _dot(a, b):
    return float((a.double() * b.double()).sum())


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_gradients_are_the_operators_own(kind):
    rows, x, y, w = _case(kind)
    gy, gout = torch.randn_like(y), torch.randn_like(x)
    assert torch.equal(torch.autograd.grad(fb.expert_dispatch(x, rows), x, gy)[0], fb.expert_combine(gy, rows))
    dy, dw = torch.autograd.grad(fb.expert_combine(y, rows, w), (y, w), gout)
    want = fb.expert_combine_backward(gout, y.detach(), rows, w.detach())
    assert torch.equal(dy, want[0]) and torch.equal(dw, want[1]) and dw.dtype == w.dtype
    assert torch.equal(torch.autograd.grad(fb.expert_combine(y, rows), y, gout)[0], fb.expert_dispatch(gout, rows))
    # one of the two alone, and a gradient that is not contiguous
    assert torch.equal(torch.autograd.grad(fb.expert_combine(y.detach(), rows, w), w, gout)[0], dw)
    assert torch.equal(torch.autograd.grad(fb.expert_combine(y, rows, w.detach()), y, gout)[0], dy)
    turned = gout.t().contiguous().t()
    assert not turned.is_contiguous() and torch.equal(torch.autograd.grad(fb.expert_combine(y, rows, w), y, turned)[0], dy)
    one = torch.ones((), device=x.device, dtype=x.dtype).expand(TOKENS, H)   # a sum's gradient
    assert torch.equal(torch.autograd.grad(fb.expert_combine(y, rows, w).sum(), y)[0], fb.expert_combine_backward(one.contiguous(), y.detach(), rows, w.detach())[0])


def test_gradients_against_differences():
    """A loss that is linear in each argument: its difference along a direction is the
    gradient's product with it, up to FP32 sums of some thousand terms on either side."""
    rows, x, y, w = _case()
    gout, gy = torch.randn_like(x), torch.randn_like(y)
    cases = [(lambda v: _dot(fb.expert_dispatch(v, rows), gy), x, torch.autograd.grad(fb.expert_dispatch(x, rows), x, gy)[0]),
             (lambda v: _dot(fb.expert_combine(v, rows, w.detach()), gout), y, torch.autograd.grad(fb.expert_combine(y, rows, w), y, gout)[0]),
             (lambda v: _dot(fb.expert_combine(y.detach(), rows, v), gout), w, torch.autograd.grad(fb.expert_combine(y, rows, w), w, gout)[0])]
    for loss, at, grad in cases:
        direction = torch.randn_like(at)
        want, plus, minus = _dot(grad, direction), loss((at + direction).detach()), loss((at - direction).detach())
        # each FP32 value is within top_k + 1 roundings of the true one, each gradient within H
        size = 4 * float(gout.abs().double().sum() + gy.abs().double().sum()) * float(at.detach().abs().max() + direction.abs().max()) * max(1.0, float(y.detach().abs().max()))
        assert abs((plus - minus) / 2 - want) <= size * (TOP_K + H) * 2.0 ** -24


def test_second_order():
    rows, x, y, w = _case()
    # without weights the functions are linear, and gradients of gradients exist
    gy = torch.randn_like(y).requires_grad_()
    dx, = torch.autograd.grad(fb.expert_dispatch(x, rows), x, gy, create_graph=True)
    v = torch.randn_like(x)
    assert torch.equal(torch.autograd.grad(dx, gy, v)[0], fb.expert_dispatch(v, rows))
    gout = torch.randn_like(x).requires_grad_()
    dy, = torch.autograd.grad(fb.expert_combine(y, rows), y, gout, create_graph=True)
    u = torch.randn_like(y)
    assert torch.equal(torch.autograd.grad(dy, gout, u)[0], fb.expert_combine(u, rows))
    # with weights they do not
    dy, dw = torch.autograd.grad(fb.expert_combine(y, rows, w), (y, w), torch.randn_like(x), create_graph=True)
    for g in (dy, dw):
        with pytest.raises(RuntimeError, match="second-order"):
            g.sum().backward(retain_graph=True)
    dw, = torch.autograd.grad(fb.expert_combine(y.detach(), rows, w), w, torch.randn_like(x), create_graph=True)
    with pytest.raises(RuntimeError, match="second-order"):
        dw.sum().backward()


def test_forward_mode_raises():
    rows, x, y, w = (t.detach() for t in _case())
    with forward_ad.dual_level():
        for call in (lambda: fb.expert_dispatch(forward_ad.make_dual(x, x), rows), lambda: fb.expert_combine(forward_ad.make_dual(y, y), rows),
                     lambda: fb.expert_combine(y, rows, forward_ad.make_dual(w, w))):
            with pytest.raises((RuntimeError, NotImplementedError)):
                call()


def test_no_graph_where_none_is_asked_for():
    rows, x, y, w = _case()
    with torch.no_grad():
        assert fb.expert_dispatch(x, rows).grad_fn is None and fb.expert_combine(y, rows, w).grad_fn is None
    assert fb.expert_dispatch(x.detach(), rows).grad_fn is None and fb.expert_combine(y.detach(), rows).grad_fn is None
    assert fb.expert_combine(y, rows, w).grad_fn is not None


def test_saved_tensors_that_changed_are_noticed():
    rows, x, y, w = _case()
    out = fb.expert_combine(y, rows, w)
    with torch.no_grad():
        w.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.sum().backward()


def test_training_step_through_experts_of_the_callers_own():
    """Routed matrices in torch, sorted and combined by the operators: gradients of all
    weights, the router's among them, against the same step written densely in 64 bits.
    Three products of sums of up to H terms follow each other, forward and back: some
    3 H FP32 roundings of 2^-24, 1.3e-5 of the terms' magnitudes were all of one sign."""
    x = E.normal(1, (TOKENS, H), "f32").to(G.device())
    router = E.normal(2, (H, EXPERTS), "f32", 0.1).to(G.device()).requires_grad_()
    experts = E.normal(3, (EXPERTS, H, H), "f32", 0.1).to(G.device()).requires_grad_()
    target = E.normal(4, (TOKENS, H), "f32").to(G.device())
    p = torch.softmax(x @ router, 1)
    w, ids = p.topk(TOP_K, dim=1)
    s = fb.expert_sort(ids, EXPERTS)
    rows = fb.expert_dispatch(x, s.rows)
    at = s.offsets.tolist()
    y = torch.cat([rows[at[e]:at[e + 1]] @ experts[e] for e in range(EXPERTS)])
    out = fb.expert_combine(y, s.rows, w)
    grads = torch.autograd.grad(((out - target) ** 2).sum(), (router, experts))
    router64, experts64 = router.detach().double().requires_grad_(), experts.detach().double().requires_grad_()
    p = torch.softmax(x.double() @ router64, 1)
    mask = torch.zeros_like(p).scatter(1, ids, 1.0)
    dense = torch.stack([x.double() @ experts64[e] for e in range(EXPERTS)], 1)
    want = torch.autograd.grad(((((p * mask)[..., None] * dense).sum(1) - target.double()) ** 2).sum(), (router64, experts64))
    for g, v in zip(grads, want):
        assert float((g.double() - v).norm()) <= 3 * H * 2.0 ** -24 * float(v.norm())


def test_captured_backward_replays():
    """Forward and backward captured together, on leaves that no eager graph holds."""
    G.announce("expert autograd graph")
    rows, x, y, w = _case()
    gout = torch.randn_like(x)
    want = torch.autograd.grad(fb.expert_combine(y, rows, w), (y, w), gout)
    static = [t.detach().clone().requires_grad_() for t in (y, w)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(fb.expert_combine(static[0], rows, static[1]), static, gout)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = torch.autograd.grad(fb.expert_combine(static[0], rows, static[1]), static, gout)
    for factor in (1.0, 0.5, 2.0):
        with torch.no_grad():
            static[0].copy_(y * factor)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured[0], want[0]) and torch.equal(captured[1], want[1] * factor)   # powers of two: exact
