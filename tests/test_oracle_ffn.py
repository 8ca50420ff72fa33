"""Pins of the feed-forward oracles: closed forms, brute force, and gradients
against differences, all on the CPU."""

import numpy as np
import pytest

import oracle
from oracle import ffn, fp4


def test_pow2_scale_is_the_smallest_that_holds():
    rng = np.random.default_rng(0)
    amax = np.concatenate([2.0 ** rng.uniform(-60, 60, 2000), [448.0, 447.0, 449.0, 1.75, 0.875, 6.0, 3.0, 2.0 ** -20]])
    for top in (448.0, 6.0):
        s = ffn.pow2_scale(amax, top)
        assert np.all(np.frexp(s)[0] == 0.5)
        assert np.all(amax <= top * s) and np.all(amax > top * s / 2)
        assert ffn.pow2_scale(top, top) == 1.0 and ffn.pow2_scale(np.nextafter(top, 1e9), top) == 2.0
    assert np.log2(ffn.pow2_scale(0.0, 448.0)) == -108 and np.log2(ffn.pow2_scale(0.0, 6.0)) == -102


def test_e2m1_table_and_ties():
    assert list(fp4.DECODE[:8]) == [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    assert np.array_equal(fp4.DECODE[8:], -fp4.DECODE[:8])
    # halfway cases go to the even code; their neighbours to the nearer one
    for mid, code in [(0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6)]:
        assert fp4.encode(mid) == code and fp4.encode(-mid) == code + 8
        below, above = fp4.encode(np.nextafter(mid, 0)), fp4.encode(np.nextafter(mid, 9))
        assert above == below + 1
    assert fp4.encode(0.0) == 0 and fp4.encode(-0.0) == 8 and fp4.encode(-1e-9) == 8


def test_fp4_weight_round_trip():
    rng = np.random.default_rng(1)
    w = (rng.standard_normal((5, 96)) * 2.0 ** rng.uniform(-30, 30, (5, 1))).astype(np.float32)
    w[2, 32:64] = 0
    q, s = fp4.weight_quant(w)
    assert q.shape == (5, 48) and s.shape == (5, 3) and s[2, 1] == 25
    err = np.abs(fp4.dequant(q, s) - w)
    step = np.repeat(np.ldexp(1.0, s.astype(int) - 127), 32, axis=1)
    assert np.all(err <= step)                       # half of the widest spacing, 2
    assert np.array_equal(fp4.dequant(*fp4.weight_quant(fp4.dequant(q, s).astype(np.float32))), fp4.dequant(q, s))


def test_activation_grads_against_differences():
    rng = np.random.default_rng(2)
    g, u, dh = rng.standard_normal((3, 50)) * 3
    g[:4] = [-300.0, 300.0, 0.0, -30.0]
    f = lambda g, u: g * ffn.sigmoid(g) * u  # noqa: E731
    dg, du = ffn.activation_grads(dh, g, u)
    eps = 1e-6
    assert np.allclose(dg, dh * (f(g + eps, u) - f(g - eps, u)) / (2 * eps), rtol=1e-7, atol=1e-7)
    assert np.allclose(du, dh * (f(g, u + eps) - f(g, u - eps)) / (2 * eps), rtol=1e-7, atol=1e-7)


def test_backward_without_rounding_is_the_chain_rule():
    """Values that E4M3 holds pass Q unchanged: dx and dW are then plain products."""
    rng = np.random.default_rng(3)
    m, f, k = 130, 128, 256
    wg, wu = (rng.integers(0, 0x7F, (f, k)).astype(np.uint8) for _ in range(2))
    s = np.exp2(rng.integers(-6, 0, (1, 2))).astype(np.float32)
    g, u = np.full((m, f), 400.0), np.zeros((m, f))    # silu(g) = g, so du = 400 dh, dg = 0
    dh = oracle.e4m3.DECODE[rng.integers(0x30, 0x40, (m, f))]
    x = oracle.e4m3.DECODE[rng.integers(0x30, 0x40, (m, k))]
    dx, dwg, dwu = ffn.gated_ffn_backward(dh / 400.0, x, g, u, wg, s, wu, s)
    assert not dwg.any()
    assert np.allclose(dwu, dh.T @ x, rtol=1e-12) and np.allclose(dx, dh @ ffn.weight(wu, s), rtol=1e-12)


@pytest.mark.parametrize("m", [1, 127, 128, 129])
def test_token_blocks_are_filled_with_zeros(m):
    rng = np.random.default_rng(m)
    v = rng.standard_normal((m, 3))
    q = ffn.quantize_tokens(v)
    assert q.shape == v.shape
    one = ffn.quantize_rows(np.concatenate([v[:min(m, 128)].T, np.zeros((3, 128 - min(m, 128)))], 1))
    assert np.array_equal(q[:128], one.T[:m])
    assert np.all(np.abs(q - v) <= np.abs(v) * 2.0 ** -4 + 2.0 ** -9 * np.abs(v).max() / 200)
