"""GPU tests of the global gradient norm and clipping against float64.

The norm is the FP64 sum's root rounded to FP32 (2^-24, and the partials' sums a
thousand times finer).  The factor adds two FP32 roundings and the product one,
so an FP32 result is within 4 * 2^-24 of the exact one, a bf16 result within half
an ulp more.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from oracle.fp8_gemm import bf16_ulp
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


def _grads(sizes, types, seed=0, scale=1e-3):
    gen = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=gen) * scale).to(t) for n, t in zip(sizes, types)]


def _norm(grads):
    return np.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))


def _check(grads, outs, norm, max_norm, eps=1e-6):
    want = _norm(grads)
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
    factor = min(1.0, max_norm / (want + eps))
    for g, o in zip(grads, outs):
        ref = g.double().numpy() * factor
        tol = np.abs(ref) * 4 * 2.0 ** -24 + 2.0 ** -149
        if g.dtype == torch.bfloat16:
            tol = tol + bf16_ulp(ref) / 2
        assert o.dtype == g.dtype and np.all(np.abs(o.double().cpu().numpy() - ref) <= tol)


BF, F32 = torch.bfloat16, torch.float32
# one value; less than a vector; the ends of a chunk of 16384; a table of 256
# tensors exactly, one more, and three tables
CASES = [([1], [F32]), ([3], [BF]), ([7, 0, 9], [BF, F32, F32]), ([16384, 16383, 16385], [BF, F32, BF]),
         ([40001, 5], [F32, BF]), ([10] * 96, [BF] * 96), ([11] * 97, [F32, BF] * 49), ([300 + i for i in range(200)], [BF, F32] * 100),
         ([13] * 256, [F32, BF] * 128), ([20 + i % 7 for i in range(257)], [BF] * 256 + [F32]), ([i % 40 for i in range(600)], [BF, F32] * 300),
         ([3_000_001, 17], [BF, F32])]


@pytest.mark.parametrize("sizes,types", CASES)
@pytest.mark.parametrize("over", [0.5, 4.0])
def test_clip_into_out_and_in_place(sizes, types, over):
    G.announce(f"clip {len(sizes)} tensors, {sum(sizes)} values, over {over}")
    grads = _grads(sizes, types)
    dev = [g.to(G.device()) for g in grads]
    max_norm = _norm(grads) / over
    outs = [torch.full_like(g, 7.0) for g in dev]
    norm = fb.clip_grad_norm(dev, max_norm, out=outs)
    _check(grads, outs, norm, max_norm)
    assert all(torch.equal(d.cpu(), g) for d, g in zip(dev, grads))     # sources untouched
    again = [torch.empty_like(g) for g in dev]
    assert torch.equal(fb.clip_grad_norm(dev, max_norm, out=again), norm) and torch.equal(fb.grad_norm(dev), norm)
    assert all(torch.equal(p, q) for p, q in zip(outs, again))
    in_place = fb.clip_grad_norm(dev, max_norm)
    assert torch.equal(in_place, norm) and all(torch.equal(p, q) for p, q in zip(dev, outs))
    if over < 1:
        assert all(torch.equal(d.cpu(), g) for d, g in zip(dev, grads))  # factor 1: the same bits


@pytest.mark.parametrize("dtype", [BF, F32])
def test_views_at_every_offset(dtype):
    """Tensors that start anywhere in a buffer, in and out at different offsets."""
    gen = torch.Generator().manual_seed(1)
    flat = torch.randn(5000, generator=gen).to(dtype)
    src, dst = flat.to(G.device()), torch.full((5000,), 3.0, dtype=dtype, device=G.device())
    grads = [src[600 * i + i:600 * i + i + 500 + i] for i in range(8)]
    outs = [dst[600 * i + (7 * i) % 16:600 * i + (7 * i) % 16 + 500 + i] for i in range(8)]
    norm = fb.clip_grad_norm(grads, 1.0, out=outs)
    _check([g.cpu() for g in grads], outs, norm, 1.0)
    written = torch.zeros(5000, dtype=torch.bool)
    for i in range(8):
        written[600 * i + (7 * i) % 16:600 * i + (7 * i) % 16 + 500 + i] = True
    assert torch.all(dst.cpu()[~written] == 3.0) and torch.equal(src.cpu(), flat)


@pytest.mark.parametrize("scale", [1e-30, 1e30])
def test_no_overflow_or_underflow(scale):
    grads = _grads([1000, 2000], [F32, BF], scale=scale)
    dev = [g.to(G.device()) for g in grads]
    norm = fb.clip_grad_norm(dev, float(np.float32(_norm(grads) / 2)), eps=0.0)
    _check(grads, dev, norm, float(np.float32(_norm(grads) / 2)), eps=0.0)


def test_zero_nan_and_inf():
    zero = [torch.zeros(100, device=G.device())]
    assert fb.clip_grad_norm(zero, 1.0) == 0 and not zero[0].any()
    bad = [torch.ones(5, device=G.device()), torch.ones(5, device=G.device(), dtype=BF)]
    bad[1][3] = float("nan")
    assert torch.isnan(fb.clip_grad_norm(bad, 1.0)) and all(torch.isnan(t).all() for t in bad)
    inf = [torch.ones(5, device=G.device())]
    inf[0][2] = float("inf")
    assert torch.isinf(fb.clip_grad_norm(inf, 1.0))
    assert torch.isnan(inf[0][2]) and torch.equal(inf[0][:2], torch.zeros(2, device=G.device()))
    assert fb.clip_grad_norm([torch.ones(4, device=G.device())], 0.0) == 2.0


def test_more_than_one_pass_of_the_grid():
    """More chunks than workgroups: 1024 x 16384 values and some."""
    n = 1024 * 16384 + 12345
    g = torch.full((n,), 0.5, dtype=BF, device=G.device())
    norm = fb.clip_grad_norm([g], 1.0)
    assert abs(float(norm) - 0.5 * np.sqrt(n)) <= 2.0 ** -23 * float(norm)
    assert torch.all(g == g[0]) and abs(float(g[0]) * float(norm) - 0.5) <= 2.0 ** -9


def test_other_stream_graph_and_refusals():
    grads = [g.to(G.device()) for g in _grads([1000, 70000], [BF, F32])]
    outs = [torch.empty_like(g) for g in grads]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        norm = fb.clip_grad_norm(grads, 0.1, out=outs)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    assert torch.equal(norm, fb.grad_norm(grads))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = fb.clip_grad_norm(grads, 0.1, out=outs)
    for _ in range(3):
        [o.zero_() for o in outs]
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured, norm) and all(torch.equal(p, q) for p, q in zip(outs, want))
    with pytest.raises(TypeError):
        fb.clip_grad_norm([grads[0].half()], 1.0)
    for bad in (lambda: fb.clip_grad_norm([torch.ones(4, 4, device=G.device()).t()], 1.0),
                lambda: fb.clip_grad_norm(grads, 1.0, out=outs[:1]), lambda: fb.clip_grad_norm(grads, 1.0, out=outs[::-1]),
                lambda: fb.clip_grad_norm([grads[0], grads[1].cpu()], 1.0), lambda: fb.clip_grad_norm(grads, 1.0, eps=-1.0)):
        with pytest.raises(ValueError):
            bad()
