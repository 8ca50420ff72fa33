"""expert_dispatch, its quantized form, expert_combine and its backward pass against
the oracle: rows of every kind of length, both types, choices that take no part.

Bounds.  dispatch copies bits.  dispatch_quant is act_quant, bit for bit.  combine
adds top_k terms by fused multiply-adds in FP32: top_k roundings, each at most
2^-24 of a partial sum that does not exceed the terms' magnitudes by more than the
roundings before it (1 + top_k 2^-24 covers these), then one to the output's type.
dweights is such a sum of h terms, added up in some order; dy is one product,
rounded to FP32 and then to its type.  Below the normal values a rounding is half
the least step.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from fp8_block_scaled_quant_amd import _ffn_lib, _lib
from oracle import experts as oracle
from tests import expert_util as E
from tests import ffn_util as U
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

# tokens, top_k, experts, drop: one token; more choices than are read together; none that takes part; many tokens
ROUTES = [(1, 8, 16, 0.0), (1, 1, 1, 0.0), (37, 3, 5, 0.2), (20, 11, 13, 0.3), (6, 4, 3, 1.0), (300, 8, 64, 0.5)]
# whole 16-byte pieces or not, one element, less and more than a workgroup's
LENGTHS = [1, 7, 8, 120, 1001, 2048, 2056]


def _rows(route, seed=0):
    tokens, top_k, experts, drop = route
    offsets, rows, _ = E.sort(E.choices(seed, tokens, top_k, experts, drop), experts)
    return rows, U.gpu(rows), int(offsets[-1])


def _poison(y, rows):
    """NaN in the rows behind the experts', whose contents must not matter."""
    y = y.clone()
    y[np.setdiff1d(np.arange(len(y)), rows[rows >= 0])] = float("nan")
    return y


def _sum_bound(terms, count, size, kind):
    return size * (count * 2.0 ** -24 * (1 + count * 2.0 ** -24) + E.STEP[kind] * (1 + count * 2.0 ** -23)) + E.LEAST[kind] + count * E.LEAST["f32"]


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("h", LENGTHS)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_dispatch(route, h, kind):
    G.announce(f"expert_dispatch {route} {h} {kind}")
    rows, dev, _ = _rows(route)
    x = E.normal(1, (rows.shape[0], h), kind)
    if h > 2:
        x[0, :3] = torch.tensor([float("nan"), float("-inf"), -0.0])
    got = fb.expert_dispatch(x.to(G.device()), dev)
    bits = torch.int16 if kind == "bf16" else torch.int32
    assert got.dtype == x.dtype and np.array_equal(got.view(bits).cpu().numpy(), oracle.dispatch(x.view(bits).numpy(), rows))


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("h", [128, 384, 2048, 2176, 7168])
@pytest.mark.parametrize("kind,fmt", [("bf16", None), ("bf16", "ue8m0"), ("f32", None), ("f32", "ue8m0")])
def test_dispatch_quant(route, h, kind, fmt):
    G.announce(f"expert_dispatch_quant {route} {h} {kind} {fmt}")
    rows, dev, _ = _rows(route)
    x = E.normal(2, (rows.shape[0], h), kind, 3.0).to(G.device())
    x[0, :128] = 0
    y, s = fb.expert_dispatch_quant(x, dev, fmt)
    want_y, want_s = fb.act_quant(fb.expert_dispatch(x, dev), 128, fmt)
    assert y.dtype == torch.float8_e4m3fn and torch.equal(y.view(torch.uint8), want_y.view(torch.uint8)) and torch.equal(s, want_s)


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("h", LENGTHS)
@pytest.mark.parametrize("kind,w_kind", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", None), ("f32", None)])
def test_combine(route, h, kind, w_kind):
    G.announce(f"expert_combine {route} {h} {kind} {w_kind}")
    rows, dev, _ = _rows(route)
    y = E.normal(3, (rows.size, h), kind)
    w = None if w_kind is None else E.normal(4, rows.shape, w_kind)
    got = fb.expert_combine(_poison(y, rows).to(G.device()), dev, None if w is None else w.to(G.device()))
    assert got.dtype == y.dtype
    want, size = oracle.combine(U.values(y), rows, None if w is None else U.values(w))
    E.within(got, want, _sum_bound(want, rows.shape[1], size, kind))


@pytest.mark.parametrize("route", ROUTES)
@pytest.mark.parametrize("h", LENGTHS)
@pytest.mark.parametrize("kind,w_kind", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", None)])
def test_combine_backward(route, h, kind, w_kind):
    G.announce(f"expert_combine_backward {route} {h} {kind} {w_kind}")
    rows, dev, _ = _rows(route)
    y, dout = E.normal(5, (rows.size, h), kind), E.normal(6, (rows.shape[0], h), kind, 1e-3)
    w = None if w_kind is None else E.normal(7, rows.shape, w_kind)
    on = [t.to(G.device()) for t in (dout, _poison(y, rows))]
    wd = None if w is None else w.to(G.device())
    dy, dw = fb.expert_combine_backward(*on, dev, wd)
    want_dy, want_dw, size = oracle.combine_backward(U.values(dout), U.values(y), rows, None if w is None else U.values(w))
    assert dy.dtype == y.dtype and dw.dtype == (torch.float32 if w is None else w.dtype)
    E.within(dy, want_dy, np.abs(want_dy) * (2.0 ** -24 + E.STEP[kind] * (1 + 2.0 ** -23)) + E.LEAST[kind])
    E.within(dw, want_dw, _sum_bound(want_dw, h, size, w_kind or "f32"))
    # one alone: the same bits
    only_dy, none = fb.expert_combine_backward(*on, dev, wd, weight_grad=False)
    assert none is None and torch.equal(only_dy, dy)
    none, only_dw = fb.expert_combine_backward(*on, dev, wd, row_grad=False)
    assert none is None and torch.equal(only_dw, dw)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_unaligned_views(kind):
    """Contiguous tensors that start anywhere: the same results."""
    rows, dev, _ = _rows((29, 4, 6, 0.2))
    shifted = lambda t: torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)  # noqa: E731
    x, y = E.normal(1, (29, 264), kind).to(G.device()), E.normal(2, (116, 264), kind).to(G.device())
    w = E.normal(3, rows.shape, "f32").to(G.device())
    assert torch.equal(fb.expert_dispatch(shifted(x), dev), fb.expert_dispatch(x, dev))
    assert torch.equal(fb.expert_combine(shifted(y), dev, w), fb.expert_combine(y, dev, w))
    got, want = fb.expert_combine_backward(shifted(x), y, dev, w), fb.expert_combine_backward(x, y, dev, w)
    assert torch.equal(got[0], want[0])
    # sums of other threads' elements: within the bound of two such sums
    _, _, size = oracle.combine_backward(U.values(x), U.values(y), rows)
    E.within(got[1], U.values(want[1]), 2 * _sum_bound(None, 264, size, "f32"))


@pytest.mark.parametrize("route", [(1, 1, 1, 0.0), (33, 5, 7, 0.3)])
@pytest.mark.parametrize("h", [1, 33, 256])
def test_writes_stay_inside(route, h):
    G.announce(f"expert rows guards {route} {h}")
    tokens, top_k = route[:2]
    rows, dev, _ = _rows(route)
    n, lib = rows.size, _ffn_lib.lib()
    x, y = E.normal(1, (tokens, h), "bf16").to(G.device()), E.normal(2, (n, h), "bf16").to(G.device())
    w = E.normal(3, rows.shape, "bf16").to(G.device())
    outs = [U.guarded_like(shape, torch.bfloat16) for shape in ((n, h), (tokens, h), (n, h), rows.shape)]
    ptr = [t.data_ptr() for t, _ in outs]
    assert lib.fp8bsq_expert_dispatch(x.data_ptr(), 1, dev.data_ptr(), tokens, top_k, h, ptr[0], G.stream()) == _lib.OK
    assert lib.fp8bsq_expert_combine(y.data_ptr(), 1, dev.data_ptr(), w.data_ptr(), 1, tokens, top_k, h, ptr[1], G.stream()) == _lib.OK
    assert lib.fp8bsq_expert_combine_backward(x.data_ptr(), y.data_ptr(), 1, dev.data_ptr(), w.data_ptr(), 1, tokens, top_k, h, ptr[2], ptr[3],
                                              G.stream()) == _lib.OK
    torch.cuda.synchronize()
    for _, guard in outs:
        guard.check_guards()
    assert torch.equal(outs[0][0], fb.expert_dispatch(x, dev)) and torch.equal(outs[1][0], fb.expert_combine(y, dev, w))
    assert all(torch.equal(t, want) for (t, _), want in zip(outs[2:], fb.expert_combine_backward(x, y, dev, w)))


def test_empty_and_leading_dimensions():
    rows, dev, _ = _rows((6, 2, 3, 0.2))
    x, y, w = E.normal(1, (6, 128), "f32").to(G.device()), E.normal(2, (12, 128), "f32").to(G.device()), E.normal(3, rows.shape, "f32").to(G.device())
    wide = dev.view(2, 3, 2)
    assert torch.equal(fb.expert_dispatch(x.view(2, 3, 128), wide), fb.expert_dispatch(x, dev))
    out = fb.expert_combine(y, dev, w)
    assert torch.equal(fb.expert_combine(y, wide, w.view(2, 3, 2)), out.view(2, 3, 128))
    dy, dw = fb.expert_combine_backward(x.view(2, 3, 128), y, wide, w.view(2, 3, 2))
    assert dw.shape == (2, 3, 2) and torch.equal(dy, fb.expert_combine_backward(x, y, dev, w)[0])
    # no tokens
    none = dev[:0]
    assert fb.expert_dispatch(x[:0], none).shape == (0, 128) and fb.expert_combine(y[:0], none, w[:0]).shape == (0, 128)
    assert [t.shape for t in fb.expert_dispatch_quant(x[:0], none)] == [(0, 128), (0, 1)]
    assert [t.shape for t in fb.expert_combine_backward(x[:0], y[:0], none, w[:0])] == [(0, 128), (0, 2)]
    # rows of no length: the sums over nothing
    assert fb.expert_dispatch(x[:, :0].contiguous(), dev).shape == (12, 0)
    dy, dw = fb.expert_combine_backward(x[:, :0].contiguous(), y[:, :0].contiguous(), dev, w)
    assert dy.shape == (12, 0) and not dw.any()


def test_values_of_infinite_magnitude_stay_with_their_tokens():
    """An infinity or NaN in one token's rows, or weights, reaches that token alone."""
    rows, dev, _ = _rows((10, 3, 4, 0.2))
    y, w = E.normal(1, (30, 64), "f32").to(G.device()), E.normal(2, rows.shape, "f32").to(G.device())
    clean = fb.expert_combine(y, dev, w)
    token, j = np.argwhere(rows >= 0)[0]
    for bad in (float("inf"), float("nan")):
        dirty = y.clone()
        dirty[rows[token, j]] = bad
        got = fb.expert_combine(dirty, dev, w)
        assert not torch.isfinite(got[token]).any()
        assert torch.equal(got[np.arange(10) != token], clean[np.arange(10) != token])


def test_rows_of_other_contents_touch_nothing_outside():
    """Numbers that expert_sort does not write: unspecified values, and no access outside."""
    n, h = 24, 40
    for bad in (10 ** 9, -10 ** 9, n, ~n, 2 ** 31 - 1, -2 ** 31):
        rows = torch.full((8, 3), bad, dtype=torch.int32, device=G.device())
        rows[0, 0] = 5
        x, y = E.normal(1, (8, h), "f32").to(G.device()), E.normal(2, (n, h), "f32").to(G.device())
        out, guard = U.guarded_like((n, h), torch.float32)
        assert _ffn_lib.lib().fp8bsq_expert_dispatch(x.data_ptr(), 0, rows.data_ptr(), 8, 3, h, out.data_ptr(), G.stream()) == _lib.OK
        torch.cuda.synchronize()
        guard.check_guards()
        assert torch.equal(out[5], x[0])
        assert torch.equal(fb.expert_combine(y, rows)[0], y[5]) and not fb.expert_combine(y, rows)[1:].any()


def test_refusals():
    rows, dev, _ = _rows((6, 2, 3, 0.0))
    x, y, w = E.normal(1, (6, 128), "f32").to(G.device()), E.normal(2, (12, 128), "f32").to(G.device()), torch.ones(6, 2, device=G.device())
    for bad in (lambda: fb.expert_dispatch(x[:5], dev), lambda: fb.expert_dispatch(x.t(), dev), lambda: fb.expert_dispatch(x.cpu(), dev),
                lambda: fb.expert_dispatch(x, dev.t()), lambda: fb.expert_dispatch_quant(x[:, :100].contiguous(), dev),
                lambda: fb.expert_dispatch_quant(x, dev, "e8"), lambda: fb.expert_combine(y[:11], dev, w), lambda: fb.expert_combine(y, dev, w[:5]),
                lambda: fb.expert_combine(y, dev, w.cpu()), lambda: fb.expert_combine_backward(x[:, :64].contiguous(), y, dev, w),
                lambda: fb.expert_combine_backward(x, y[:3], dev, w), lambda: fb.expert_combine(y, dev[:, :0].contiguous())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fb.expert_dispatch(x.half(), dev), lambda: fb.expert_dispatch(x, dev.long()), lambda: fb.expert_combine(y, dev, w.half()),
                lambda: fb.expert_combine_backward(x.bfloat16(), y, dev, w)):
        with pytest.raises(TypeError):
            bad()
    shifted = torch.cat([x.new_zeros(1), x.flatten()])[1:].view(x.shape)
    with pytest.raises(fb.Fp8Error):
        fb.expert_dispatch_quant(shifted, dev)   # 4-byte aligned


def test_graph_replays():
    G.announce("expert rows graph")
    cases = []
    for s in range(3):
        rows, dev, _ = _rows((50, 4, 8, 0.2), s)
        cases.append((dev, E.normal(s, (50, 256), "bf16").to(G.device()), E.normal(s + 9, (50, 4), "f32").to(G.device())))
    static = [t.clone() for t in cases[0]]

    def step(rows, x, w):
        y = fb.expert_dispatch(x, rows)
        out = fb.expert_combine(y, rows, w)
        return y, out, *fb.expert_combine_backward(out, y, rows, w), *fb.expert_dispatch_quant(x, rows)

    step(*static)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(*static)
    for case in cases + cases:
        for t, v in zip(static, case):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(captured, step(*case)))
