"""GPU parity of the gated feed-forward block against the float64 oracle.

g and u are held to the block GEMM's bound (1e-3 sum |a b|, + 1 bf16 ulp) and h
to what that bound lets through: |silu'| <= 1.1, so
|dh| <= 1.1 T_g (|u| + T_u) + |silu(g)| T_u.  All three are also held to REL in
the 2-norm, which a wrong scale, row or block breaks by orders of magnitude.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_quant_amd as fb
import oracle
from fp8_block_scaled_quant_amd import _ffn_lib, _lib
from inputs import gen
from oracle import ffn
from tests import ffn_util as U
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


def _inputs(m, f, k, x_type="bf16", seed=None):
    rng = np.random.default_rng(m * 7919 + f * 31 + k if seed is None else seed)
    x = gen.activations(rng, m, k, dtype=x_type, outliers=True)
    return x, U.weight(rng.integers(1 << 30), f, k), U.weight(rng.integers(1 << 30), f, k)


def _check(x, wg, wu, fmt, out, got, rows=None):
    xr = x.float().numpy() if rows is None else x.float().numpy()[rows]
    h, g, u = ffn.gated_ffn(xr, *wg, *wu, fmt)
    a, a_s = oracle.act_quant(xr, 128, fmt)
    tg, tu = oracle.gemm_tolerance(a, a_s, *wg), oracle.gemm_tolerance(a, a_s, *wu)
    th = 1.1 * tg * (np.abs(u) + tu) + np.abs(g * ffn.sigmoid(g)) * tu
    for name, have, want, tol in zip("hgu", got, (h, g, u), (th, tg, tu)):
        have = U.values(have) if rows is None else U.values(have)[rows]
        assert oracle.gemm_check(have, want, tol, out).all(), name
        assert U.rel_error(have, want) <= U.REL[out], (name, U.rel_error(have, want))


# one row; sixteen and seventeen; the ends of 16-, 32-, 64- and 256-row tiles;
# features that are not a multiple of 16, 64 or 128, one feature; one K block,
# odd numbers of them, and a long K
SHAPES = [(1, 128, 128), (1, 2300, 1024), (2, 1, 256), (3, 130, 384), (8, 4096, 512), (15, 333, 640), (16, 256, 512),
          (17, 129, 1152), (31, 700, 256), (33, 64, 128), (64, 1000, 768), (65, 257, 512), (127, 384, 640),
          (128, 128, 1024), (200, 1111, 384), (257, 640, 128), (300, 513, 2048), (513, 260, 896), (5, 300, 20608)]


@pytest.mark.parametrize("m,f,k", SHAPES)
def test_shapes(m, f, k):
    G.announce(f"gated_ffn m={m} f={f} k={k}")
    x, wg, wu = _inputs(m, f, k)
    args = (x.to(G.device()), U.gpu(wg[0]), U.gpu(wg[1]), U.gpu(wu[0]), U.gpu(wu[1]))
    fmt = "ue8m0" if (m + f) % 2 else None
    got = fb.gated_ffn(*args, scale_fmt=fmt, save=True)
    _check(x, wg, wu, fmt, "bf16", got)
    assert torch.equal(fb.gated_ffn(*args, scale_fmt=fmt), got[0])     # the same h without save
    again = fb.gated_ffn(*args, scale_fmt=fmt, save=True)
    assert all(torch.equal(p, q) for p, q in zip(got, again))


@pytest.mark.parametrize("m,f,k", [(1, 300, 512), (16, 256, 512), (90, 200, 384), (300, 130, 1024)])
@pytest.mark.parametrize("fmt", [None, "ue8m0"])
@pytest.mark.parametrize("x_type,out", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
def test_types(m, f, k, fmt, x_type, out):
    G.announce(f"gated_ffn m={m} f={f} k={k} {x_type} -> {out} {fmt}")
    x, wg, wu = _inputs(m, f, k, x_type)
    got = fb.gated_ffn(x.to(G.device()), U.gpu(wg[0]), U.gpu(wg[1]), U.gpu(wu[0]), U.gpu(wu[1]), scale_fmt=fmt,
                       out_dtype=U.TYPES[out], save=True)
    _check(x, wg, wu, fmt, out, got)


@pytest.mark.parametrize("m,f,k", [(1, 18432, 7168), (40, 18432, 7168), (1000, 2304, 7168)])
def test_dense_block_sampled_rows(m, f, k):
    G.announce(f"gated_ffn dense m={m} f={f} k={k}")
    x, wg, wu = _inputs(m, f, k)
    got = fb.gated_ffn(x.to(G.device()), U.gpu(wg[0]), U.gpu(wg[1]), U.gpu(wu[0]), U.gpu(wu[1]), save=True)
    rows = np.unique(np.concatenate([[0, m - 1], np.random.default_rng(0).integers(0, m, 6)]))
    _check(x, wg, wu, None, "bf16", got, rows)


# more 256 x 256 tiles than CUs; features in whole vectors, and not
@pytest.mark.parametrize("f", [2304, 2309])
@pytest.mark.parametrize("fmt,out", [(None, "bf16"), ("ue8m0", "bf16"), (None, "f32"), ("ue8m0", "f32")])
def test_many_tiles_sampled_rows(f, fmt, out):
    m, k = 4000, 512
    G.announce(f"gated_ffn m={m} f={f} k={k} {fmt} -> {out}")
    x, wg, wu = _inputs(m, f, k)
    args = (x.to(G.device()), U.gpu(wg[0]), U.gpu(wg[1]), U.gpu(wu[0]), U.gpu(wu[1]), fmt, U.TYPES[out])
    got = fb.gated_ffn(*args, save=True)
    rows = np.unique(np.r_[0, 255, 256, 3839, 3840, m - 1, np.random.default_rng(0).integers(0, m, 24)])
    _check(x, wg, wu, fmt, out, got, rows)
    assert torch.equal(fb.gated_ffn(*args), got[0])


@pytest.mark.parametrize("m,f,k", [(1, 129, 128), (16, 45, 256), (50, 77, 128), (129, 259, 256), (260, 1, 128)])
def test_writes_stay_inside(m, f, k):
    G.announce(f"gated_ffn guards m={m} f={f} k={k}")
    x, wg, wu = _inputs(m, f, k)
    dev = [x.to(G.device()), U.gpu(wg[0]), U.gpu(wg[1]), U.gpu(wu[0]), U.gpu(wu[1])]
    lib = _ffn_lib.lib()
    outs = [U.guarded_like((m, f), torch.bfloat16) for _ in range(3)]
    nbytes = lib.fp8_gated_ffn_workspace(m, f, k)
    ws, ws_guard = U.guarded_like((nbytes,), torch.uint8)
    assert lib.fp8_gated_ffn(dev[0].data_ptr(), 1, 0, *[t.data_ptr() for t in dev[1:]], *[t.data_ptr() for t, _ in outs], 1,
                             m, f, k, ws.data_ptr(), nbytes, G.stream()) == _lib.OK
    torch.cuda.synchronize()
    for _, guard in outs + [(ws, ws_guard)]:
        guard.check_guards()
    _check(x, wg, wu, None, "bf16", [t for t, _ in outs])


def test_extreme_gates():
    """g far below and above zero: silu is -0..0 and g there, with no NaN."""
    k = 128
    codes = np.zeros((4, k), np.uint8)
    codes[:, 0] = oracle.e4m3.encode(np.array([-448.0, 448.0, 0.0, -448.0]))
    ones = np.full((4, k), 0, np.uint8)
    ones[:, 0] = 0x38
    x = torch.zeros(2, k, dtype=torch.bfloat16)
    x[0, 0], x[1, 0] = 1.0, 1e30
    s = np.ones((1, 1), np.float32)
    h, g, u = fb.gated_ffn(x.to(G.device()), U.gpu(codes), U.gpu(s), U.gpu(ones), U.gpu(s), out_dtype=torch.float32, save=True)
    assert torch.isfinite(h[0]).all() and h[0, 0] == 0 and h[0, 2] == 0 and h[0, 3] == 0
    # 448 (448 s) s with the FP32 scale s = 1 / 448, twice rounded
    assert abs(float(h[0, 1]) - 448.0) <= 448.0 * 2.0 ** -22
    assert h[1, 0] == 0 and h[1, 2] == 0 and not torch.isnan(h).any()


def test_empty_and_leading_dimensions():
    x, wg, wu = _inputs(6, 96, 128)
    args = [U.gpu(wg[0]), U.gpu(wg[1]), U.gpu(wu[0]), U.gpu(wu[1])]
    x = x.to(G.device())
    h = fb.gated_ffn(x, *args)
    assert torch.equal(fb.gated_ffn(x.view(2, 3, 128), *args), h.view(2, 3, 96))
    assert fb.gated_ffn(x[:0], *args).shape == (0, 96)
    empty = [args[0][:0], args[1][:0], args[2][:0], args[3][:0]]
    assert fb.gated_ffn(x, *empty).shape == (6, 0)


def test_refusals():
    x, wg, wu = _inputs(4, 128, 256)
    x, wg, wu = x.to(G.device()), [U.gpu(v) for v in wg], [U.gpu(v) for v in wu]
    fb.gated_ffn(x, *wg, *wu)
    for bad in (lambda: fb.gated_ffn(x.t(), *wg, *wu), lambda: fb.gated_ffn(x[:, :128], *wg, *wu),
                lambda: fb.gated_ffn(x, wg[0], wg[1][:, :1].contiguous(), *wu),
                lambda: fb.gated_ffn(x, wg[0][:64], wg[1], *wu), lambda: fb.gated_ffn(x, *wg, *wu, scale_fmt="e8"),
                lambda: fb.gated_ffn(x.cpu(), *wg, *wu)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fb.gated_ffn(x.half(), *wg, *wu), lambda: fb.gated_ffn(x, wg[0].float(), wg[1], *wu),
                lambda: fb.gated_ffn(x, wg[0], wg[1].double(), *wu), lambda: fb.gated_ffn(x, *wg, *wu, out_dtype=torch.half)):
        with pytest.raises(TypeError):
            bad()
    shifted = torch.empty(4 * 256 + 1, dtype=torch.bfloat16, device=x.device)[1:].view(4, 256)
    with pytest.raises(fb.Fp8Error):
        fb.gated_ffn(shifted, *wg, *wu)                # 2-byte aligned activations


@pytest.mark.parametrize("m", [1, 12, 40, 300])
def test_graph_replays_and_other_streams(m):
    f, k = 640, 512
    G.announce(f"gated_ffn graph m={m}")
    _, wg, wu = _inputs(m, f, k)
    args = [U.gpu(v) for v in (*wg, *wu)]
    xs = [gen.activations(np.random.default_rng(s), m, k).to(G.device()) for s in range(3)]
    static = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = fb.gated_ffn(static, *args)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(other, fb.gated_ffn(static, *args))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = fb.gated_ffn(static, *args, save=True)
    for x in xs + xs:
        static.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        eager = fb.gated_ffn(x, *args, save=True)
        assert all(torch.equal(p, q) for p, q in zip(captured, eager))
