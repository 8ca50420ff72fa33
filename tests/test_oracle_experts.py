"""The expert operators' oracle against independent statements of the same."""

import numpy as np
import pytest

import oracle
from oracle import experts
from tests import expert_util as E


@pytest.mark.parametrize("tokens,top_k,num,drop", [(0, 2, 3, 0.0), (1, 1, 1, 0.0), (7, 3, 5, 0.3), (40, 8, 9, 0.5), (9, 4, 2, 0.0), (5, 2, 4, 1.0)])
def test_sort(tokens, top_k, num, drop):
    ids = E.choices(tokens, tokens, top_k, num, drop)
    offsets, rows, choices = experts.sort(ids, num)
    for got, want in zip((offsets, rows, choices), E.sort(ids, num)):
        assert np.array_equal(got, want) and got.dtype == np.int32
    flat, place = ids.reshape(-1), np.where(rows < 0, ~rows, rows).reshape(-1)
    assert np.array_equal(np.sort(place), np.arange(flat.size)) and np.array_equal(choices[place], np.arange(flat.size))
    for e in range(num):
        assert np.array_equal(flat[choices[offsets[e]:offsets[e + 1]]], np.full(offsets[e + 1] - offsets[e], e))
        assert np.all(np.diff(choices[offsets[e]:offsets[e + 1]]) > 0)


def test_combine_undoes_dispatch_and_gradients_are_adjoint():
    rng = np.random.default_rng(0)
    ids = E.choices(3, 20, 4, 6, 0.25)
    _, rows, _ = experts.sort(ids, 6)
    x, y, dout, w = rng.standard_normal((20, 8)), rng.standard_normal((80, 8)), rng.standard_normal((20, 8)), rng.standard_normal((20, 4))
    assert np.allclose(experts.combine(experts.dispatch(x, rows), rows)[0], x * (rows >= 0).sum(1, keepdims=True))
    # <dispatch(x), y> = <x, combine(y)>
    assert np.isclose((experts.dispatch(x, rows) * y).sum(), (x * experts.combine(y, rows)[0]).sum())
    # the gradients against differences of a bilinear function, exact but for rounding
    dy, dw, _ = experts.combine_backward(dout, y, rows, w)
    loss = lambda y, w: (experts.combine(y, rows, w)[0] * dout).sum()  # noqa: E731
    dir_y, dir_w = rng.standard_normal(y.shape), rng.standard_normal(w.shape)
    assert np.isclose(loss(y + dir_y, w) - loss(y, w), (dy * dir_y).sum())
    assert np.isclose(loss(y, w + dir_w) - loss(y, w), (dw * dir_w).sum())
    behind = np.setdiff1d(np.arange(80), rows[rows >= 0])
    assert not dy[behind].any() and not dw[rows < 0].any()


def test_products_row_by_row():
    num, n, k = 3, 140, 256
    ids = E.choices(5, 9, 2, num, 0.2)
    offsets, _, choices = experts.sort(ids, num)
    rng = np.random.default_rng(1)
    a = oracle.e4m3.encode(rng.standard_normal((18, k)) * 50)
    a_s = rng.random((18, 2)).astype(np.float32)
    (wg, wg_s), (wu, wu_s) = E.weights(1, num, n, k), E.weights(2, num, n, k)
    h, g, u = experts.gated(a, a_s, offsets, wg, wg_s, wu, wu_s)
    for r in range(18):
        e = ids.reshape(-1)[choices[r]]
        if not 0 <= e < num:
            assert not h[r].any() and not g[r].any()
            continue
        av, bv = oracle.dequantized_operands(a[r:r + 1], a_s[r:r + 1], wg[e], wg_s[e])
        assert np.allclose(g[r], (av @ bv.T)[0], rtol=1e-12, atol=1e-12)
        assert np.allclose(h[r], g[r] / (1 + np.exp(-g[r])) * u[r], rtol=1e-12)
