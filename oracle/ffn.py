"""The gated feed-forward block and its backward pass (oracle; test infrastructure only).

Definitions, in float64:

    (a, a_s) = act_quant(x),  g = a . Wg^T,  u = a . Wu^T,  h = g sigmoid(g) u
    dg = dh u s (1 + g (1 - s)),  du = dh g s,  s = sigmoid(g)
    dx = Q(dg) Wg + Q(du) Wu       Q over 128 features
    dWg = Q(dg)^T Q(x), dWu = Q(du)^T Q(x)   Q over 128 tokens, the last block filled up with zeros

Q rounds v / s to the nearest E4M3 value, s the smallest power of two with
max |v| <= 448 s, max |v| taken as at least 2^-100.
"""

import numpy as np

from . import e4m3
from .act_quant import act_quant
from .fp8_gemm import fp8_gemm

BLOCK = 128


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def gated_ffn(x, wg, wg_s, wu, wu_s, scale_fmt=None, rows=None):
    """(h, g, u) in float64; x float32 values, weights uint8 codes."""
    x = x if rows is None else x[rows]
    a, a_s = act_quant(x, BLOCK, scale_fmt)
    g, u = fp8_gemm(a, a_s, wg, wg_s), fp8_gemm(a, a_s, wu, wu_s)
    return g * sigmoid(g) * u, g, u


def pow2_scale(amax, top):
    """Smallest power of two s with amax <= top * s (amax at least 2^-100)."""
    amax = np.maximum(np.asarray(amax, dtype=np.float64), 2.0 ** -100)
    s = 2.0 ** np.floor(np.log2(amax / top) - 1)   # at or below the answer
    for _ in range(3):
        s = np.where(amax > top * s, 2.0 * s, s)   # exact comparisons
    return s


def quantize_rows(v):
    """The values that v [rows, n] stands for after Q over 128 columns (n a multiple of 128)."""
    b = np.asarray(v, dtype=np.float64).reshape(v.shape[0], -1, BLOCK)
    s = pow2_scale(np.abs(b).max(-1, keepdims=True), e4m3.MAX_FINITE)
    return (e4m3.decode(e4m3.encode(b / s)) * s).reshape(v.shape)


def quantize_tokens(v):
    m = v.shape[0]
    padded = np.zeros((-(-m // BLOCK) * BLOCK, v.shape[1]))
    padded[:m] = v
    return np.ascontiguousarray(quantize_rows(np.ascontiguousarray(padded.T)).T)[:m]


def weight(codes, scales):
    """The weight that codes and block scales stand for, exactly."""
    n, k = codes.shape
    wide = np.repeat(np.repeat(scales.astype(np.float64), BLOCK, 0)[:n], BLOCK, 1)[:, :k]
    return e4m3.decode(codes) * wide


def activation_grads(dh, g, u):
    s = sigmoid(g)
    return dh * u * s * (1 + g * (1 - s)), dh * g * s


def gated_ffn_backward(dh, x, g, u, wg, wg_s, wu, wu_s):
    """(dx, dwg, dwu) in float64 from float64 (or float32) dh, x, g, u."""
    dh, x, g, u = (np.asarray(v, dtype=np.float64) for v in (dh, x, g, u))
    dg, du = activation_grads(dh, g, u)
    dx = quantize_rows(dg) @ weight(wg, wg_s) + quantize_rows(du) @ weight(wu, wu_s)
    xq = quantize_tokens(x)
    return dx, quantize_tokens(dg).T @ xq, quantize_tokens(du).T @ xq
