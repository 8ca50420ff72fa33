"""``Experts``, and the operators together as it calls them: bit for bit the calls it
stands for, and within a bound of the block's definition in 64 bits.

The bound, element by element: a product moves by 1e-3 sum |a b|; h = silu(g) u by
1.1 dg |u| + |silu(g)| du + 1.1 dg du, and 2^-20 of it; each rounding to bf16 by 2^-8
of the value (or 2^-24 in FP32); E4M3 by 2^-4 of the value or, below the normal codes,
by 2^-10 of the block's scale.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_quant_amd as fb
import oracle
from tests import expert_util as E
from tests import ffn_util as U
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


def _layer(seed, experts, k, f, kind, fmt):
    gen = torch.Generator(G.device()).manual_seed(seed)
    w = [torch.randn(experts, *shape, generator=gen, device=G.device()) * shape[1] ** -0.5 for shape in ((f, k), (f, k), (k, f))]
    return fb.Experts.from_weights(*w, dtype=E.TYPES[kind], scale_fmt=fmt)


def _dense(codes, scales):
    wide = np.repeat(np.repeat(scales.astype(np.float64), 128, 1), 128, 2)
    return oracle.e4m3.decode(codes.reshape(-1, codes.shape[2])).reshape(codes.shape) * wide[:, :codes.shape[1], :codes.shape[2]]


def _reference(layer, x, ids, w):
    """(out, how far the layer's may be from it), x [T, K] and w [T, top_k] in 64 bits."""
    step = E.STEP["bf16" if layer.dtype == torch.bfloat16 else "f32"]
    weights = {}
    for name in ("w_gate", "w_up", "w_down"):
        weights[name] = _dense(getattr(layer, name).view(torch.uint8).cpu().numpy(), getattr(layer, name + "_scale").cpu().numpy())
    codes, scales = oracle.act_quant(x.astype(np.float32), 128, layer.scale_fmt)
    a = oracle.e4m3.decode(codes) * np.repeat(scales.astype(np.float64), 128, 1)
    out, off, size = np.zeros((3, *x.shape))
    for t in range(x.shape[0]):
        for j, e in enumerate(ids[t]):
            if not 0 <= e < layer.num_experts:
                continue
            wg, wu, wd = (weights[n][e] for n in ("w_gate", "w_up", "w_down"))
            g, u = wg @ a[t], wu @ a[t]
            dg, du = 1e-3 * (np.abs(wg) @ np.abs(a[t])), 1e-3 * (np.abs(wu) @ np.abs(a[t]))
            h = g * oracle.ffn.sigmoid(g) * u
            dh = 1.1 * dg * np.abs(u) + np.abs(g * oracle.ffn.sigmoid(g)) * du + 1.1 * dg * du + np.abs(h) * 2.0 ** -20
            dh = dh * (1 + step) + np.abs(h) * step
            top = (np.abs(h) + dh).reshape(-1, 128).max(1)
            scale = np.repeat(np.maximum(top, 1e-4) / 448 * (2 if layer.scale_fmt else 1), 128)
            dh = dh + np.maximum((np.abs(h) + dh) * 2.0 ** -4, scale * 2.0 ** -10)
            y, dy = wd @ h, np.abs(wd) @ dh
            dy = dy + 1e-3 * (np.abs(wd) @ (np.abs(h) + dh))
            dy = dy * (1 + step) + np.abs(y) * step
            out[t] += w[t, j] * y
            off[t] += abs(w[t, j]) * dy
            size[t] += abs(w[t, j]) * (np.abs(y) + dy)
    return out, off + size * ids.shape[1] * 2.0 ** -23 + (np.abs(out) + off) * step


@pytest.mark.parametrize("tokens,top_k,experts,drop", [(1, 4, 6, 0.0), (19, 2, 5, 0.3), (150, 3, 4, 0.0), (9, 2, 3, 1.0)])
@pytest.mark.parametrize("kind,fmt", [("bf16", None), ("bf16", "ue8m0"), ("f32", None)])
def test_layer(tokens, top_k, experts, drop, kind, fmt):
    k, f = 256, 384
    G.announce(f"Experts {tokens} x {top_k} of {experts} {kind} {fmt}")
    layer = _layer(tokens, experts, k, f, kind, fmt)
    ids = E.choices(1, tokens, top_k, experts, drop)
    x, w = E.normal(2, (tokens, k), kind).to(G.device()), torch.softmax(E.normal(3, (tokens, top_k), "f32"), 1).to(G.device())
    got = layer(x, U.gpu(ids), w)
    assert got.dtype == layer.dtype and got.shape == x.shape
    out, off = _reference(layer, U.values(x), ids, U.values(w))
    E.within(got, out, off)
    # the calls it stands for, one by one
    s = fb.expert_sort(U.gpu(ids), experts)
    a = fb.act_quant(fb.expert_dispatch(x, s.rows), 128, fmt)
    h = fb.expert_gated_ffn(*a, s.offsets, layer.w_gate, layer.w_gate_scale, layer.w_up, layer.w_up_scale, layer.dtype)
    y = fb.expert_gemm(*fb.act_quant(h, 128, fmt), s.offsets, layer.w_down, layer.w_down_scale, layer.dtype)
    assert torch.equal(got, fb.expert_combine(y, s.rows, w))
    # leading dimensions, strides and index types of other kinds
    assert torch.equal(layer(x[None], U.gpu(ids.astype(np.int32))[None], w[None]), got[None])
    twice = torch.cat([x, x], 1)
    assert torch.equal(layer(twice[:, :k], torch.cat([U.gpu(ids)] * 2, 1)[:, :top_k], torch.cat([w, w], 1)[:, :top_k]), got)


def test_tokens_are_independent():
    """A token's output does not depend on which others come with it."""
    layer = _layer(5, 8, 256, 256, "bf16", None)
    ids, x, w = E.choices(6, 33, 2, 8), E.normal(7, (33, 256), "bf16").to(G.device()), torch.rand(33, 2, device=G.device())
    all_together = layer(x, U.gpu(ids), w)
    alone = torch.cat([layer(x[t:t + 1], U.gpu(ids[t:t + 1]), w[t:t + 1]) for t in range(33)])
    assert torch.equal(all_together, alone)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_rows_that_start_anywhere(kind):
    """A contiguous view that is not 16-byte aligned: the same output."""
    layer = _layer(3, 4, 128, 256, kind, None)
    x, w = E.normal(1, (7, 128), kind).to(G.device()), torch.rand(7, 2, device=G.device())
    ids = U.gpu(E.choices(2, 7, 2, 4))
    shifted = lambda t: torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)  # noqa: E731
    assert shifted(x).data_ptr() % 16 and torch.equal(layer(shifted(x), shifted(ids), shifted(w)), layer(x, ids, w))


def test_no_tokens_and_refusals():
    layer = _layer(1, 3, 128, 128, "bf16", None)
    x, ids, w = torch.zeros(0, 128, dtype=torch.bfloat16, device=G.device()), torch.zeros(0, 2, dtype=torch.int64, device=G.device()), torch.zeros(0, 2, device=G.device())
    assert layer(x, ids, w).shape == (0, 128)
    x, ids, w = torch.zeros(4, 128, device=G.device()), torch.zeros(4, 2, dtype=torch.int64, device=G.device()), torch.zeros(4, 2, device=G.device())
    for bad in (lambda: layer(x[:3], ids, w), lambda: layer(x, ids, w[:3]), lambda: layer(x[:, :64], ids, w), lambda: layer(x.cpu(), ids, w)):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("tokens", [1, 40, 700])
def test_captured_layer_replays(tokens):
    """A captured step serves later tokens with other choices: nothing is read back to the host."""
    G.announce(f"Experts graph {tokens}")
    layer = _layer(2, 6, 256, 256, "bf16", "ue8m0")
    cases = [(E.normal(s, (tokens, 256), "bf16").to(G.device()), U.gpu(E.choices(s, tokens, 2, 6, 0.2 * s)), torch.rand(tokens, 2, device=G.device())) for s in range(3)]
    static = [t.clone() for t in cases[0]]
    layer(*static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = layer(*static)
    for case in cases + cases:
        for t, v in zip(static, case):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured, layer(*case))
