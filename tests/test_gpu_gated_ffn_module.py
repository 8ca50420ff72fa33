"""``GatedFFN`` over the kernels: its outputs and gradients are those of the calls it
is made of, bit for bit, in both types and scale formats, for decode and training
sizes, for inputs that lie anywhere; and what it refuses.
"""

import pytest
import torch
from torch.autograd import forward_ad

import fp8_block_scaled_quant_amd as fb
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _module(k, f, dtype=BF, fmt=None):
    torch.manual_seed(k + f)
    return fb.GatedFFN(k, f, dtype, fmt, G.device())


def _randn(*shape, dtype, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(G.device())


def _calls(mod, x, dh):
    """(h, dx, dw_gate, dw_up) by the operators themselves."""
    wg, wu = fb.weight_quant(mod.w_gate.detach()), fb.weight_quant(mod.w_up.detach())
    h, g, u = fb.gated_ffn(x, *wg, *wu, mod.scale_fmt, x.dtype, save=True)
    return h, *fb.gated_ffn_backward(dh, x, g, u, *wg, *wu, out_dtype=x.dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("fmt", [None, "ue8m0"])
@pytest.mark.parametrize("shape,f", [((1, 128), 128), ((2, 7, 256), 384), ((130, 512), 256), ((3, 100, 384), 1152), ((1100, 256), 1024)])
def test_matches_the_calls(shape, f, dtype, fmt):
    G.announce(f"GatedFFN {shape} -> {f} {dtype} {fmt}")
    mod = _module(shape[-1], f, dtype, fmt)
    x, dh = _randn(*shape, dtype=dtype), _randn(*shape[:-1], f, dtype=dtype, seed=1) * 1e-3
    want = _calls(mod, x, dh)
    x.requires_grad_()
    h = mod(x)
    h.backward(dh)
    assert h.dtype == dtype and h.shape == (*shape[:-1], f)
    for have, ref in zip((h, x.grad, mod.w_gate.grad, mod.w_up.grad), want):
        assert have.dtype == dtype and torch.equal(have, ref)
    with torch.no_grad():
        assert torch.equal(mod(x), h)
    with torch.inference_mode():
        assert torch.equal(mod(x), h)


def test_no_tokens():
    mod = _module(128, 256)
    x = torch.zeros(0, 128, dtype=BF, device=G.device(), requires_grad=True)
    mod(x).sum().backward()
    assert x.grad.shape == (0, 128) and not mod.w_gate.grad.any() and not mod.w_up.grad.any()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_inputs_and_gradients_that_lie_anywhere(dtype):
    mod, one = _module(256, 128, dtype), torch.zeros(1, dtype=dtype, device=G.device())
    x, dh = _randn(9, 256, dtype=dtype), _randn(9, 128, dtype=dtype, seed=1)
    want = _calls(mod, x, dh)
    shifted = torch.cat([one, x.flatten()])[1:].view(9, 256)
    assert shifted.is_contiguous() and shifted.data_ptr() % 16
    strided = torch.stack([x, x], -1)[..., 0]
    for source in (shifted, strided):
        leaf = source.detach().requires_grad_()
        mod.zero_grad()
        h = mod(leaf)
        # the gradient that reaches h is a contiguous view one element into a buffer
        (torch.cat([one, h.flatten()]) * torch.cat([one, dh.flatten()])).sum().backward()
        for have, ref in zip((h, leaf.grad, mod.w_gate.grad, mod.w_up.grad), want):
            assert torch.equal(have, ref)
        with torch.no_grad():
            assert torch.equal(mod(leaf), want[0])


def test_gradients_on_other_streams():
    mod = _module(256, 384)
    x, dh = _randn(300, 256, dtype=BF), _randn(300, 384, dtype=BF, seed=1)
    want = _calls(mod, x, dh)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        leaf = x.clone().requires_grad_()
        mod(leaf).backward(dh)
    side.synchronize()
    for have, ref in zip((leaf.grad, mod.w_gate.grad, mod.w_up.grad), want[1:]):
        assert torch.equal(have, ref)


def test_second_order_and_forward_mode_raise():
    mod = _module(128, 128, F32)
    x = _randn(5, 128, dtype=F32).requires_grad_()
    for loss in (torch.sum, lambda h: h.square().sum()):
        dx, = torch.autograd.grad(loss(mod(x)), x, create_graph=True)
        first, = torch.autograd.grad(loss(mod(x)), x)
        assert torch.equal(dx.detach(), first)
        with pytest.raises(RuntimeError, match="second-order"):
            (mod(x).sum() + dx.square().sum()).backward()
    for grad_mode in (True, False):
        with forward_ad.dual_level(), torch.set_grad_enabled(grad_mode):
            with pytest.raises(NotImplementedError):
                mod(forward_ad.make_dual(x.detach(), torch.ones_like(x)))


def test_refusals():
    mod = _module(128, 128)
    with pytest.raises(ValueError):
        mod(torch.zeros(2, 256, dtype=BF, device=G.device()))
    with pytest.raises(ValueError):
        fb.GatedFFN(128, 128)(torch.zeros(2, 128, dtype=BF))          # on the CPU
