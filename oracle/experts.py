"""The expert operators (oracle; test infrastructure only).

Choice c = t * top_k + j is token t's j-th.  Sorting is by expert, stable; choices
whose number is no expert's come last, and have ``rows`` ~r for their row r.  In
float64:

    dispatch          y[rows[t, j]] = x[t]; rows behind the experts' are zero
    combine           out[t] = sum_j w[t, j] y[rows[t, j]], over the choices that have an expert
    combine_backward  dy[rows[t, j]] = w[t, j] dout[t], dw[t, j] = <dout[t], y[rows[t, j]]>
    product           c[r] = a[r] W[e]^T for offsets[e] <= r < offsets[e + 1], rows behind zero
    gated             silu(a Wg^T) (a Wu^T) of these
"""

import numpy as np

from .ffn import sigmoid
from .fp8_gemm import fp8_gemm


def sort(experts, num_experts):
    """(offsets, rows, choices) by looking for every expert's choices in turn."""
    flat = np.asarray(experts).reshape(-1)
    order, offsets = [], [0]
    for e in range(num_experts):
        order += [c for c in range(flat.size) if flat[c] == e]
        offsets.append(len(order))
    behind = set(range(flat.size)) - set(order)
    order += sorted(behind)
    rows = np.empty(flat.size, dtype=np.int32)
    for r, c in enumerate(order):
        rows[c] = r if r < offsets[-1] else ~r
    return np.array(offsets, np.int32), rows.reshape(np.shape(experts)), np.array(order, np.int32)


def dispatch(x, rows):
    """x [T, H], rows [T, top_k] -> [T * top_k, H], x's own values and type."""
    y = np.zeros((rows.size, x.shape[1]), x.dtype)
    for t in range(rows.shape[0]):
        for r in rows[t]:
            if r >= 0:
                y[r] = x[t]
    return y


def combine(y, rows, weights=None):
    """(out, sum of the terms' magnitudes)."""
    y = np.asarray(y, np.float64)
    out, size = np.zeros((2, rows.shape[0], y.shape[1]))
    for t in range(rows.shape[0]):
        for j, r in enumerate(rows[t]):
            if r >= 0:
                term = (1.0 if weights is None else float(weights[t, j])) * y[r]
                out[t] += term
                size[t] += np.abs(term)
    return out, size


def combine_backward(dout, y, rows, weights=None):
    """(dy, dweights, sum of dweights' terms' magnitudes)."""
    dout, y = np.asarray(dout, np.float64), np.asarray(y, np.float64)
    dy, (dw, size) = np.zeros_like(y), np.zeros((2, *rows.shape))
    for t in range(rows.shape[0]):
        for j, r in enumerate(rows[t]):
            if r >= 0:
                dy[r] = (1.0 if weights is None else float(weights[t, j])) * dout[t]
                dw[t, j] = (dout[t] * y[r]).sum()
                size[t, j] = np.abs(dout[t] * y[r]).sum()
    return dy, dw, size


def product(a, a_s, offsets, w, w_s):
    """a [R, K] codes, w [E, N, K] codes -> [R, N]."""
    c = np.zeros((a.shape[0], w.shape[1]))
    for e in range(w.shape[0]):
        part = slice(offsets[e], offsets[e + 1])
        if offsets[e + 1] > offsets[e]:
            c[part] = fp8_gemm(a[part], a_s[part], w[e], w_s[e])
    return c


def gated(a, a_s, offsets, wg, wg_s, wu, wu_s):
    """(h, g, u)"""
    g, u = product(a, a_s, offsets, wg, wg_s), product(a, a_s, offsets, wu, wu_s)
    return g * sigmoid(g) * u, g, u
