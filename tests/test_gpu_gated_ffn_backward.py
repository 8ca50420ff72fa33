"""GPU parity of the feed-forward block's backward pass.

Against the float64 oracle, which rounds as the kernels do: REL in the 2-norm,
plus what an E4M3 rounding costs that the FP32 and the float64 value of a
gradient take to different sides (a few in 10^6 values lie that near to a
boundary): a step is at most 2^-3 of the value, so one of a value three times
the root mean square, among m f values, is 3 / 8 / sqrt(m f).  Against differences of the formula
without rounding: E4M3 rounds a value by up to 2^-4 of it, 2.6% in the mean
square, for one operand of dx and both of dW.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from fp8_block_scaled_quant_amd import _ffn_lib, _lib
from inputs import gen
from oracle import ffn
from tests import ffn_util as U
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


def _inputs(m, f, k, dtype="bf16", scale=1e-4):
    rng = np.random.default_rng(m * 7919 + f * 31 + k)
    cast = (lambda v: gen.to_bf16(v)) if dtype == "bf16" else (lambda v: torch.from_numpy(v))
    dh = rng.standard_normal((m, f), dtype=np.float32) * np.float32(scale)
    dh[rng.random(m) < 0.1] = 0                         # masked tokens
    g, u = (rng.standard_normal((m, f), dtype=np.float32) * np.float32(1.7) for _ in range(2))
    x = gen.normal_f32(rng, (m, k))
    x[:, :2] *= 20
    return [cast(v) for v in (dh, x, g, u)], U.weight(rng.integers(1 << 30), f, k), U.weight(rng.integers(1 << 30), f, k)


def _run(acts, wg, wu, **kw):
    return fb.gated_ffn_backward(*[t.to(G.device()) for t in acts], *[U.gpu(v) for v in (*wg, *wu)], **kw)


def _check(acts, wg, wu, got, out):
    want = ffn.gated_ffn_backward(*[t.float().numpy() for t in acts], *wg, *wu)
    for name, have, ref in zip(("dx", "dw_gate", "dw_up"), got, want):
        assert have.dtype == U.TYPES[out]
        err = U.rel_error(U.values(have), ref)
        assert err <= U.REL[out] + 3 / 8 / np.sqrt(acts[0].numel()), (name, err)


# one token; the ends of 128-token blocks; two to five blocks of tokens (their
# exponents come four to a word); sizes that fill no 256-wide tile
@pytest.mark.parametrize("m,f,k", [(1, 128, 128), (2, 256, 128), (127, 128, 384), (128, 384, 256), (129, 256, 640),
                                   (300, 512, 384), (513, 128, 256), (640, 640, 128), (65, 1024, 896), (1100, 256, 512)])
def test_shapes(m, f, k):
    G.announce(f"gated_ffn_backward m={m} f={f} k={k}")
    acts, wg, wu = _inputs(m, f, k)
    got = _run(acts, wg, wu)
    _check(acts, wg, wu, got, "bf16")
    assert all(torch.equal(p, q) for p, q in zip(got, _run(acts, wg, wu)))


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("m,f,k", [(5, 256, 128), (200, 128, 384)])
def test_types(m, f, k, dtype, out):
    G.announce(f"gated_ffn_backward m={m} f={f} k={k} {dtype} -> {out}")
    acts, wg, wu = _inputs(m, f, k, dtype)
    _check(acts, wg, wu, _run(acts, wg, wu, out_dtype=U.TYPES[out]), out)


@pytest.mark.parametrize("scale", [1e-12, 1.0, 1e6])
def test_gradients_of_any_size(scale):
    """No floor: gradients far below act_quant's 1e-4 keep their precision."""
    acts, wg, wu = _inputs(140, 256, 128, "f32", scale)
    _check(acts, wg, wu, _run(acts, wg, wu, out_dtype=torch.float32), "f32")


# both products in 256 x 256 tiles: dx's last round short by 56 workgroups, which
# take two of dW's tiles first; and by 168 after two full rounds, dW's tiles being
# the longer ones.  A dx of 128 x 128 tiles beside three rounds of dW's, and a dW
# too large for that.
@pytest.mark.parametrize("m,f,k", [(1600, 2304, 7040), (3000, 512, 12800), (70, 1792, 3456), (3, 5120, 3968)])
def test_many_tiles(m, f, k):
    """Sampled rows of dx, and sampled features and columns of dW."""
    G.announce(f"gated_ffn_backward m={m} f={f} k={k}")
    (dh, x, g, u), wg, wu = _inputs(m, f, k)
    got = [U.values(t) for t in _run((dh, x, g, u), wg, wu)]
    dh, x, g, u = (t.float().double().numpy() for t in (dh, x, g, u))
    rng = np.random.default_rng(0)
    rows = np.unique(np.r_[0, m - 1, rng.integers(m, size=40)])
    dg, du = (ffn.quantize_rows(v) for v in ffn.activation_grads(dh[rows], g[rows], u[rows]))
    want = dg @ ffn.weight(*wg) + du @ ffn.weight(*wu)
    assert U.rel_error(got[0][rows], want) <= U.REL["bf16"] + 3 / 8 / np.sqrt(dg.size)
    feats = np.unique(np.r_[0, f - 1, rng.integers(f, size=40)])
    cols = np.unique(np.r_[0, k - 1, rng.integers(k, size=600)])
    xq = ffn.quantize_tokens(x[:, cols])
    for have, v in zip(got[1:], ffn.activation_grads(dh[:, feats], g[:, feats], u[:, feats])):
        want = ffn.quantize_tokens(v).T @ xq
        assert U.rel_error(have[np.ix_(feats, cols)], want) <= U.REL["bf16"] + 3 / 8 / np.sqrt(v.size)


def test_parts_and_zero_gradients():
    acts, wg, wu = _inputs(70, 256, 384)
    dx, dwg, dwu = _run(acts, wg, wu)
    only_x, none1, none2 = _run(acts, wg, wu, weight_grad=False)
    assert none1 is None and none2 is None and torch.equal(only_x, dx)
    none, only_g, only_u = _run(acts, wg, wu, input_grad=False)
    assert none is None and torch.equal(only_g, dwg) and torch.equal(only_u, dwu)
    acts[0] = torch.zeros_like(acts[0])
    assert not any(bool(t.any()) for t in _run(acts, wg, wu))
    empty = [t[:0] for t in acts]
    dx, dwg, dwu = _run(empty, wg, wu)
    assert dx.shape == (0, 384) and not dwg.any() and not dwu.any() and dwg.shape == (256, 384)


def test_extreme_gates_have_finite_gradients():
    acts, wg, wu = _inputs(40, 128, 128, "f32", 1.0)
    acts[2][:, :6] = torch.tensor([-1e4, -200.0, -88.5, 0.0, 200.0, 1e4])
    got = _run(acts, wg, wu, out_dtype=torch.float32)
    assert all(torch.isfinite(t).all() for t in got)
    _check(acts, wg, wu, got, "f32")


def test_writes_stay_inside():
    m, f, k = 130, 256, 384
    acts, wg, wu = _inputs(m, f, k)
    dev = [t.to(G.device()) for t in acts] + [U.gpu(v) for v in (*wg, *wu)]
    lib = _ffn_lib.lib()
    outs = [U.guarded_like(s, torch.bfloat16) for s in ((m, k), (f, k), (f, k))]
    nbytes = lib.fp8_gated_ffn_backward_workspace(m, f, k)
    ws, ws_guard = U.guarded_like((nbytes,), torch.uint8)
    p = [t.data_ptr() for t in dev]
    assert lib.fp8_gated_ffn_backward(*p[:4], 1, *p[4:], *[t.data_ptr() for t, _ in outs], 1, m, f, k, ws.data_ptr(), nbytes,
                                      G.stream()) == _lib.OK
    torch.cuda.synchronize()
    for _, guard in outs + [(ws, ws_guard)]:
        guard.check_guards()
    _check(acts, wg, wu, [t for t, _ in outs], "bf16")


def test_against_differences():
    """Directional derivatives along the computed gradients themselves."""
    m, f, k = 256, 256, 384
    acts, wg, wu = _inputs(m, f, k, "f32", 1.0)
    dh, x = (acts[i].double().numpy() for i in (0, 1))
    w1, w2 = ffn.weight(*wg), ffn.weight(*wu)

    def loss(x, w1, w2):
        g, u = x @ w1.T, x @ w2.T
        return np.sum(dh * (g * ffn.sigmoid(g) * u))

    acts[2], acts[3] = (torch.from_numpy((x @ w.T).astype(np.float32)) for w in (w1, w2))
    grads = [U.values(t) for t in _run(acts, wg, wu, out_dtype=torch.float32)]
    for i, (grad, at) in enumerate(zip(grads, (x, w1, w2))):
        d = grad / np.linalg.norm(grad)
        eps = 1e-4 * np.linalg.norm(at)
        plus, minus = [x, w1, w2], [x, w1, w2]
        plus[i], minus[i] = at + eps * d, at - eps * d
        slope = (loss(*plus) - loss(*minus)) / (2 * eps)
        # <true, got> / |got|: |got| up to the rounding's 2.6% per operand, whose
        # part along the gradient is of second order plus a 1% allowance
        assert abs(slope - np.linalg.norm(grad)) <= 0.02 * np.linalg.norm(grad), i


def test_module_trains_and_matches_the_calls():
    torch.manual_seed(0)
    mod = fb.GatedFFN(256, 384, device=G.device())
    x = torch.randn(3, 50, 256, device=G.device(), dtype=torch.bfloat16, requires_grad=True)
    h = mod(x)
    dh = torch.randn_like(h) * 1e-3
    h.backward(dh)
    wg, wu = fb.weight_quant(mod.w_gate.detach()), fb.weight_quant(mod.w_up.detach())
    h2, g, u = fb.gated_ffn(x.detach(), *wg, *wu, save=True)
    want = fb.gated_ffn_backward(dh, x.detach(), g, u, *wg, *wu)
    assert torch.equal(h, h2)
    for have, ref in zip((x.grad, mod.w_gate.grad, mod.w_up.grad), want):
        assert torch.equal(have, ref)
    mod.w_gate.grad = None
    mod.w_up.requires_grad_(False)
    mod(x.detach()).sum().backward()                     # no input gradient asked for
    assert mod.w_gate.grad is not None


def test_refusals():
    acts, wg, wu = _inputs(4, 128, 256)
    with pytest.raises(TypeError):
        _run([acts[0].float()] + acts[1:], wg, wu)
    with pytest.raises(ValueError):
        _run([acts[0][:2]] + acts[1:], wg, wu)
    with pytest.raises(ValueError):
        _run([t[:, :100].contiguous() for t in acts], wg, wu)
    with pytest.raises(ValueError):
        _run(acts, (wg[0][:64], wg[1]), wu)
    with pytest.raises(TypeError):
        _run(acts, wg, wu, out_dtype=torch.half)


def test_graph_replays():
    acts, wg, wu = _inputs(200, 256, 384)
    args = [t.to(G.device()) for t in acts] + [U.gpu(v) for v in (*wg, *wu)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fb.gated_ffn_backward(*args)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = fb.gated_ffn_backward(*args)
    for factor in (1.0, 0.5, -2.0, 1.0):
        args[0].copy_(acts[0] * factor)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(captured, fb.gated_ffn_backward(*args)))
