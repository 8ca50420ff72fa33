"""The feed-forward operators on operands whose offsets pass 32 bits: sampled
outputs on both sides of 2^31 and 2^32, against float64.

Products: within 1e-3 sum |a b| per element (the block GEMM's bound), and half an
ulp of bf16, 2^-8, of the result; that covers the few E4M3 roundings that FP32
and float64 values take to different sides (an eighth of one term of the sum).
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_quant_amd as fb
import oracle
from oracle import ffn, fp4
from tests import ffn_util as U
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

M, F, K = 131077, 32896, 128   # M F = 4.3e9


@pytest.fixture(autouse=True)
def _release():
    yield
    torch.cuda.empty_cache()


def _rows():
    return np.unique([0, 1, 2 ** 31 // F, 2 ** 31 // F + 1, 2 ** 32 // F, 2 ** 32 // F + 1, M - 2, M - 1])


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device=G.device(), dtype=torch.bfloat16)


def test_gated_ffn():
    G.announce(f"gated_ffn {M} x {F} x {K}")
    gen = torch.Generator(G.device()).manual_seed(0)
    x = _normal(gen, M, K)
    wg, wu = U.weight(1, F, K), U.weight(2, F, K)
    got = fb.gated_ffn(x, *[U.gpu(v) for v in (*wg, *wu)], "ue8m0", save=True)
    rows = _rows()
    xr = x[rows].float().cpu().numpy()
    h, g, u = ffn.gated_ffn(xr, *wg, *wu, "ue8m0")
    a, a_s = oracle.act_quant(xr, 128, "ue8m0")
    tg, tu = oracle.gemm_tolerance(a, a_s, *wg), oracle.gemm_tolerance(a, a_s, *wu)
    th = 1.1 * tg * (np.abs(u) + tu) + np.abs(g * ffn.sigmoid(g)) * tu
    for have, want, tol in zip(got, (h, g, u), (th, tg, tu)):
        assert oracle.gemm_check(U.values(have[rows]), want, tol, "bf16").all()


def test_gated_ffn_backward():
    G.announce(f"gated_ffn_backward {M} x {F} x {K}")
    gen = torch.Generator(G.device()).manual_seed(1)
    dh, g, u, x = _normal(gen, M, F), _normal(gen, M, F), _normal(gen, M, F), _normal(gen, M, K)
    wg, wu = U.weight(3, F, K), U.weight(4, F, K)
    dx, dwg, dwu = fb.gated_ffn_backward(dh, x, g, u, *[U.gpu(v) for v in (*wg, *wu)])
    rows = _rows()
    dg, du = (ffn.quantize_rows(v) for v in ffn.activation_grads(*[U.values(t[rows]) for t in (dh, g, u)]))
    w, v = ffn.weight(*wg), ffn.weight(*wu)
    want = dg @ w + du @ v
    tol = 1e-3 * (np.abs(dg) @ np.abs(w) + np.abs(du) @ np.abs(v)) + 2.0 ** -8 * np.abs(want)
    assert np.all(np.abs(U.values(dx[rows]) - want) <= tol)
    feats = np.array([0, 1, 127, 128, 16400, F - 1])
    xq = ffn.quantize_tokens(U.values(x))
    for have, grad in zip((dwg, dwu), ffn.activation_grads(*[U.values(t[:, feats]) for t in (dh, g, u)])):
        grad = ffn.quantize_tokens(grad)
        want = grad.T @ xq
        tol = 1e-3 * (np.abs(grad).T @ np.abs(xq)) + 2.0 ** -8 * np.abs(want)
        assert np.all(np.abs(U.values(have[feats]) - want) <= tol)


def test_fp4_quantizer_and_product():
    n, k = 640007, 13440   # 4.3e9 bytes of codes
    G.announce(f"fp4_weight_quant and fp4_gemv {n} x {k}")
    gen = torch.Generator(G.device()).manual_seed(2)
    w, x = _normal(gen, n, k), _normal(gen, 3, k)
    q, s = fb.fp4_weight_quant(w)
    rows = np.unique([0, 1, 2 ** 31 // k, 2 ** 32 // k, 2 ** 31 // (k // 2), 2 ** 32 // (k // 2), 2 ** 32 // (k // 2) + 1, n - 2, n - 1])
    codes, scales = fp4.weight_quant(w[rows].float().cpu().numpy())
    assert np.array_equal(q[rows].cpu().numpy(), codes) and np.array_equal(s[rows].cpu().numpy(), scales)
    y = U.values(fb.fp4_gemv(x, q, s, torch.float32)[:, rows])
    deq, xv = fp4.dequant(codes, scales), U.values(x)
    assert np.all(np.abs(y - xv @ deq.T) <= k * 2.0 ** -24 * (np.abs(xv) @ np.abs(deq).T))


def test_clip():
    n = 2 ** 32 + 12345
    G.announce(f"clip_grad_norm {n}")
    g = torch.full((n,), 0.5, dtype=torch.bfloat16, device=G.device())
    norm = fb.clip_grad_norm([g], 0.25 * np.sqrt(n), eps=0.0)
    assert abs(float(norm) - 0.5 * np.sqrt(n)) <= 2.0 ** -23 * float(norm)
    assert float(g.max()) == float(g.min()) and abs(float(g[-1]) - 0.25) <= 2.0 ** -10
