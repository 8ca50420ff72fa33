"""GPU parity of the 4-bit weights: the quantizer bit for bit against the oracle;
the matrix-vector product against float64 sums.  Its products are exact, so only
the FP32 sums round: at most k additions of 2^-24 of the running sum, which
sum |x w| bounds, and the output's half ulp.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from inputs import gen
from oracle import fp4
from oracle.fp8_gemm import bf16_ulp
from tests import ffn_util as U
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


def _quant(w):
    q, s = fb.fp4_weight_quant(w.to(G.device()))
    return q.cpu().numpy(), s.cpu().numpy()


@pytest.mark.parametrize("n,k", [(1, 32), (3, 64), (5, 1056), (300, 1024), (17, 4128), (1000, 96)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quant_matches_oracle(n, k, dtype):
    G.announce(f"fp4_weight_quant n={n} k={k} {dtype}")
    rng = np.random.default_rng(n + k)
    w = rng.standard_normal((n, k), dtype=np.float32) * np.exp2(rng.uniform(-30, 30, (n, 1))).astype(np.float32)
    w[n // 2, :32] = 0
    w[0, 0] = -0.0
    w = gen.to_bf16(w) if dtype == "bf16" else torch.from_numpy(w)
    for have, want in zip(_quant(w), fp4.weight_quant(w.float().numpy())):
        assert np.array_equal(have, want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quant_every_boundary(dtype):
    """Every rounding boundary and its neighbours, at scales over the whole range."""
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, 0.0], np.float32)
    step = np.float32(2.0 ** -7 if dtype == "bf16" else 2.0 ** -23)
    row = np.concatenate([mids, mids * (1 + step), mids * (1 - step / 2), -mids])
    row = np.minimum(row, 6).astype(np.float32)                       # 60 of them; each group gets its 6
    w = np.stack([np.concatenate([row[:31], [6.0], row[31:], [0, 0, 6.0]]) * np.float32(2.0 ** e) for e in (-120, -103, -102, -90, -3, 0, 7, 60, 124)])
    w = w.astype(np.float32)
    w = gen.to_bf16(w) if dtype == "bf16" else torch.from_numpy(w)
    for have, want in zip(_quant(w), fp4.weight_quant(w.float().numpy())):
        assert np.array_equal(have, want)


def test_quant_writes_stay_inside_and_empty():
    from fp8_block_scaled_quant_amd import _ffn_lib, _lib
    w = torch.randn(37, 96, device=G.device())
    q, qg = U.guarded_like((37, 48), torch.uint8)
    s, sg = U.guarded_like((37, 3), torch.uint8)
    assert _ffn_lib.lib().fp4_weight_quant(w.data_ptr(), 0, 37, 96, q.data_ptr(), s.data_ptr(), G.stream()) == _lib.OK
    torch.cuda.synchronize()
    qg.check_guards()
    sg.check_guards()
    assert np.array_equal(q.cpu().numpy(), fp4.weight_quant(w.cpu().numpy())[0])
    assert [tuple(t.shape) for t in fb.fp4_weight_quant(w[:0])] == [(0, 48), (0, 3)]
    assert [tuple(t.shape) for t in fb.fp4_weight_quant(w[:, :0].contiguous())] == [(37, 0), (37, 0)]


def _gemv_case(m, n, k, x_type, out, bias, seed=0):
    rng = np.random.default_rng(m * 7919 + n * 31 + k + seed)
    x = gen.activations(rng, m, k, dtype="f32", outliers=True)
    x = x.to(U.TYPES[x_type])
    q = rng.integers(0, 256, (n, k // 2)).astype(np.uint8)
    s = rng.integers(100, 140, (n, k // 32)).astype(np.uint8)
    b = torch.from_numpy(rng.standard_normal(n, dtype=np.float32)).to(U.TYPES[out]) if bias else None
    return x, q, s, b


def _gemv_check(x, q, s, b, out, got):
    w = fp4.dequant(q, s)
    xd = x.double().numpy()
    want = xd @ w.T + (0 if b is None else b.double().numpy())
    tol = x.shape[1] * 2.0 ** -24 * (np.abs(xd) @ np.abs(w).T) + np.abs(want) * 2.0 ** -23
    if out == "bf16":
        tol = tol + bf16_ulp(want) / 2 * (1 + 2.0 ** -6)
    assert np.all(np.abs(U.values(got) - want) <= tol)


# one row and one weight row; K of one group, of odd numbers of groups and of
# whole steps; the ends of the 16-row tiles on both sides; more rows than any tile
@pytest.mark.parametrize("m,n,k", [(1, 1, 32), (1, 16, 64), (1, 1000, 96), (2, 17, 160), (1, 4096, 7168), (3, 1000, 1056),
                                   (13, 311, 4128), (16, 64, 512), (17, 33, 544), (32, 100, 2048), (40, 2048, 256),
                                   (64, 129, 1024), (65, 48, 128), (200, 70, 352), (8, 18432, 512), (5, 40, 18432),
                                   (32, 500, 512), (45, 20, 4128), (3, 20, 100032)])
@pytest.mark.parametrize("x_type,out", [("bf16", "bf16"), ("f32", "f32")])
def test_gemv_shapes(m, n, k, x_type, out):
    G.announce(f"fp4_gemv m={m} n={n} k={k} {x_type} -> {out}")
    bias = (m + n) % 2 == 1
    x, q, s, b = _gemv_case(m, n, k, x_type, out, bias)
    args = (x.to(G.device()), U.gpu(q), U.gpu(s), U.TYPES[out], None if b is None else b.to(G.device()))
    got = fb.fp4_gemv(*args)
    _gemv_check(x, q, s, b, out, got)
    assert torch.equal(got, fb.fp4_gemv(*args))


@pytest.mark.parametrize("x_type,out,bias", [("f32", "bf16", True), ("bf16", "f32", True), ("bf16", "f32", False)])
def test_gemv_types(x_type, out, bias):
    x, q, s, b = _gemv_case(6, 500, 736, x_type, out, bias)
    got = fb.fp4_gemv(x.to(G.device()), U.gpu(q), U.gpu(s), U.TYPES[out], None if b is None else b.to(G.device()))
    _gemv_check(x, q, s, b, out, got)


def test_gemv_is_exact_on_small_integers():
    """Sums of halves below 2^24 have no rounding in any order: exact results,
    fp32 activations with 24 significant bits included."""
    rng = np.random.default_rng(4)
    q = rng.integers(0, 256, (70, 48)).astype(np.uint8)
    s = np.full((70, 3), 127, np.uint8)
    for hi in (4, 1 << 12):
        x = rng.integers(-hi, hi, (9, 96)).astype(np.float32)
        got = fb.fp4_gemv(U.gpu(x), U.gpu(q), U.gpu(s), torch.float32)
        assert np.array_equal(U.values(got), x.astype(np.float64) @ fp4.dequant(q, s).T)
    x = np.zeros((1, 96), np.float32)
    x[0, 40] = np.float32(1 + 2.0 ** -23)                  # exact times the powers of two among the weights
    got = fb.fp4_gemv(U.gpu(x), U.gpu(q), U.gpu(s), torch.float32)
    w = fp4.dequant(q, s)[:, 40]
    powers = (w == 0) | (np.frexp(np.abs(w))[0] == 0.5)
    assert powers.sum() > 20 and np.array_equal(U.values(got)[0, powers], (float(x[0, 40]) * w)[powers])


@pytest.mark.parametrize("m,n,k", [(1, 17, 96), (16, 33, 160), (33, 31, 64)])
def test_gemv_writes_stay_inside(m, n, k):
    from fp8_block_scaled_quant_amd import _ffn_lib, _lib
    for out, code in (("bf16", 1), ("f32", 0)):
        x, q, s, _ = _gemv_case(m, n, k, "bf16", out, False)
        y, guard = U.guarded_like((m, n), U.TYPES[out])
        xd, qd, sd = x.to(G.device()), U.gpu(q), U.gpu(s)
        assert _ffn_lib.lib().fp4_gemv(xd.data_ptr(), 1, qd.data_ptr(), sd.data_ptr(), None, y.data_ptr(), code, m, n, k,
                                       G.stream()) == _lib.OK
        torch.cuda.synchronize()
        guard.check_guards()
        _gemv_check(x, q, s, None, out, y)


def test_gemv_leading_dimensions_empty_and_refusals():
    x, q, s, _ = _gemv_case(6, 40, 64, "bf16", "bf16", False)
    x, q, s = x.to(G.device()), U.gpu(q), U.gpu(s)
    y = fb.fp4_gemv(x, q, s)
    assert torch.equal(fb.fp4_gemv(x.view(3, 2, 64), q, s), y.view(3, 2, 40))
    assert fb.fp4_gemv(x[:0], q, s).shape == (0, 40) and fb.fp4_gemv(x, q[:0], s[:0]).shape == (6, 0)
    bias = torch.zeros(40, device=x.device)
    for bad in (lambda: fb.fp4_gemv(x, q, s[:, :1].contiguous()), lambda: fb.fp4_gemv(x, q[:, :16].contiguous(), s),
                lambda: fb.fp4_gemv(x[:, :48].contiguous(), q, s), lambda: fb.fp4_gemv(x, q, s, bias=bias),
                lambda: fb.fp4_gemv(x.t(), q, s), lambda: fb.fp4_gemv(x, q.cpu(), s), lambda: fb.fp4_weight_quant(x[0]),
                lambda: fb.fp4_weight_quant(x[:, :48].contiguous())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fb.fp4_gemv(x.half(), q, s), lambda: fb.fp4_gemv(x, q.int(), s), lambda: fb.fp4_gemv(x, q, s, torch.half),
                lambda: fb.fp4_weight_quant(x.half())):
        with pytest.raises(TypeError):
            bad()


def test_gemv_graph_replays():
    x, q, s, _ = _gemv_case(3, 700, 1024, "bf16", "bf16", False)
    static, q, s = x.to(G.device()), U.gpu(q), U.gpu(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fb.fp4_gemv(static, q, s)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = fb.fp4_gemv(static, q, s)
    for factor in (1.0, -3.0, 0.5, 1.0):
        static.copy_(x * factor)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured, fb.fp4_gemv(static, q, s))
