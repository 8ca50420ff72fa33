"""expert_gemm and expert_gated_ffn against the oracle: any number of rows an expert,
experts without any, rows behind the last, ragged widths, both output types.

Bounds.  A product is within 1e-3 sum |a b| of the exact one (the block GEMM's), and
rounded once.  h = silu(g) u moves by at most |silu'| dg |u| + |silu(g)| du plus the
product of both, |silu'| <= 1.1; the exponential, the reciprocal and the products by
2^-20 of it.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_quant_amd as fb
import oracle
from fp8_block_scaled_quant_amd import _ffn_lib, _lib
from oracle import experts as want
from tests import expert_util as E
from tests import ffn_util as U
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


def _counts(counts, behind=0):
    """(offsets, rows): experts with these numbers of rows, and rows behind."""
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return offsets, int(offsets[-1]) + behind


def _inputs(seed, counts, behind, n, k):
    offsets, rows = _counts(counts, behind)
    rng = np.random.default_rng(seed)
    a = oracle.e4m3.encode(np.clip(rng.standard_normal((rows, k)) * 100, -448, 448))
    a_s = (2.0 ** rng.uniform(-2, 2, (rows, k // 128)) * 1e-2).astype(np.float32)
    # what the rows behind hold must not matter: NaN codes, NaN scales
    a[offsets[-1]:], a_s[offsets[-1]:] = 0x7F, np.nan
    return offsets, a, a_s, E.weights(2 * seed + 1, len(counts), n, k), E.weights(2 * seed + 2, len(counts), n, k)


def _tolerance(a, a_s, offsets, w, w_s):
    t = np.zeros((a.shape[0], w.shape[1]))
    for e in range(w.shape[0]):
        part = slice(offsets[e], offsets[e + 1])
        if offsets[e + 1] > offsets[e]:
            t[part] = oracle.gemm_tolerance(a[part], a_s[part], w[e], w_s[e])
    return t


def _check_gemm(offsets, a, a_s, w, out, got):
    c = want.product(a, a_s, offsets, *w)
    E.within(got, c, _tolerance(a, a_s, offsets, *w) * (1 + E.STEP[out]) + np.abs(c) * E.STEP[out])
    assert not got[offsets[-1]:].any()


def _check_gated(offsets, a, a_s, wg, wu, out, got):
    h, g, u = want.gated(a, a_s, offsets, *wg, *wu)
    dg, du = _tolerance(a, a_s, offsets, *wg), _tolerance(a, a_s, offsets, *wu)
    silu = np.abs(g * oracle.ffn.sigmoid(g))
    off = 1.1 * dg * np.abs(u) + silu * du + 1.1 * dg * du + np.abs(h) * 2.0 ** -20
    E.within(got, h, off * (1 + E.STEP[out]) + np.abs(h) * E.STEP[out] + 1e-30)
    assert not got[offsets[-1]:].any()


def _run(seed, counts, behind, n, k, out):
    offsets, a, a_s, wg, wu = _inputs(seed, counts, behind, n, k)
    on = [U.gpu(v) for v in (a, a_s, offsets)]
    gemm = fb.expert_gemm(*on, *[U.gpu(v) for v in wg], out_dtype=E.TYPES[out])
    gated = fb.expert_gated_ffn(*on, *[U.gpu(v) for v in (*wg, *wu)], out_dtype=E.TYPES[out])
    assert gemm.dtype == gated.dtype == E.TYPES[out] and gemm.shape == gated.shape == (len(a), n)
    _check_gemm(offsets, a, a_s, wg, out, gemm)
    _check_gated(offsets, a, a_s, wg, wu, out, gated)


# rows of the experts: one row; some experts without; around every tile's size; one expert with all; none at all
COUNTS = [[1], [0, 1, 0, 1, 1, 0], [3, 0, 17, 16, 15, 1], [0, 0, 0], [33, 64, 0, 65, 31], [127, 128, 129], [300, 1, 0, 255, 256, 257], [0, 0, 700, 0]]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("n,k", [(1, 128), (130, 256), (320, 640)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_rows(counts, n, k, out):
    G.announce(f"expert products {counts} {n} {k} {out}")
    _run(1, counts, 5, n, k, out)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 63, 64, 65, 127, 128, 129, 255, 256, 257, 388, 640])
@pytest.mark.parametrize("counts", [[2, 1, 0, 3], [70, 0, 30], [200, 300]])
def test_widths(n, counts):
    G.announce(f"expert products {counts} n={n}")
    _run(2, counts, 0, n, 384, "bf16")


@pytest.mark.parametrize("k", [128, 256, 384, 512, 640, 1024, 1152, 2944])
@pytest.mark.parametrize("counts", [[1, 4, 0], [50, 70], [260, 10]])
def test_depths(k, counts):
    G.announce(f"expert products {counts} k={k}")
    _run(3, counts, 1, 144, k, "f32")


@pytest.mark.parametrize("experts,top_k,tokens", [(64, 6, 40), (200, 8, 100), (1024, 2, 300)])
def test_many_experts(experts, top_k, tokens):
    G.announce(f"expert products of {experts}")
    ids = E.choices(1, tokens, top_k, experts, 0.1)
    offsets = E.sort(ids, experts)[0]
    _run(4, np.diff(offsets), tokens * top_k - int(offsets[-1]), 72, 256, "bf16")


def _sampled(seed, counts, behind, n, k, gated):
    """Rows at the experts' first and last, and a few others, of a larger problem."""
    offsets, a, a_s, wg, wu = _inputs(seed, counts, behind, n, k)
    on = [U.gpu(v) for v in (a, a_s, offsets)]
    got = fb.expert_gated_ffn(*on, *[U.gpu(v) for v in (*wg, *wu)]) if gated else fb.expert_gemm(*on, *[U.gpu(v) for v in wg])
    rng, picked, at = np.random.default_rng(seed), [], [0]
    for e, c in enumerate(counts):
        rows = np.unique(np.r_[0, c - 1, min(255, c - 1), min(256, c - 1), rng.integers(0, c, 4)]) if c else np.zeros(0, int)
        picked += list(offsets[e] + rows)
        at.append(len(picked))
    small = np.array(at, np.int32)
    picked = np.array(picked)
    assert not got[offsets[-1]:].any()
    if gated:
        _check_gated(small, a[picked], a_s[picked], wg, wu, "bf16", got[torch.from_numpy(picked).to(got.device)])
    else:
        _check_gemm(small, a[picked], a_s[picked], wg, "bf16", got[torch.from_numpy(picked).to(got.device)])


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("counts,n,k", [([1, 1, 0, 1, 1, 1, 1, 1, 1], 2048, 1024), ([600, 0, 700, 1300], 1100, 1024), ([2100, 300], 2048, 640),
                                        ([90] * 24, 516, 1280), ([20, 3, 0, 45] * 10, 1408, 512)])
def test_larger_sampled_rows(counts, n, k, gated):
    G.announce(f"expert products sampled {len(counts)} experts {sum(counts)} rows {n} {k} gated={gated}")
    _sampled(5, counts, 3, n, k, gated)


@pytest.mark.parametrize("counts,n,k", [([1], 1, 128), ([5, 0, 18], 45, 256), ([129, 40], 130, 128), ([300, 290], 200, 256)])
@pytest.mark.parametrize("gated", [False, True])
def test_writes_stay_inside(counts, n, k, gated):
    G.announce(f"expert products guards {counts} {n} {k}")
    offsets, a, a_s, wg, wu = _inputs(6, counts, 2, n, k)
    on, first, second = [U.gpu(v) for v in (a, a_s, offsets)], [U.gpu(v) for v in wg], [U.gpu(v) for v in wu]
    out, guard = U.guarded_like((len(a), n), torch.bfloat16)
    lib, rest = _ffn_lib.lib(), (out.data_ptr(), 1, len(a), len(counts), n, k, G.stream())
    ptr = [t.data_ptr() for t in (*on, *first, *second)]
    assert (lib.fp8_expert_gated_ffn(*ptr, *rest) if gated else lib.fp8_expert_gemm(*ptr[:5], *rest)) == _lib.OK
    torch.cuda.synchronize()
    guard.check_guards()
    if gated:
        _check_gated(offsets, a, a_s, wg, wu, "bf16", out)
    else:
        _check_gemm(offsets, a, a_s, wg, "bf16", out)


def test_one_expert_is_the_dense_product():
    """With one expert the results meet fp8_gemm's within both bounds."""
    offsets, a, a_s, wg, _ = _inputs(7, [200], 0, 300, 512)
    dense = fb.fp8_gemm(U.gpu(a), U.gpu(a_s), U.gpu(wg[0][0]), U.gpu(wg[1][0]), torch.float32)
    got = fb.expert_gemm(U.gpu(a), U.gpu(a_s), U.gpu(offsets), U.gpu(wg[0]), U.gpu(wg[1]), torch.float32)
    E.within(got, U.values(dense), 2 * _tolerance(a, a_s, offsets, *wg))


def test_input_gradient_is_the_product_with_the_transposed_blocks():
    """dx[r] = dc[r] W[e]: 128 x 128 blocks stay blocks when transposed."""
    offsets, a, a_s, _, _ = _inputs(8, [20, 0, 35], 0, 128, 384)   # dc: [55, 384]
    w, w_s = E.weights(9, 3, 384, 256)
    turned, turned_s = np.ascontiguousarray(w.transpose(0, 2, 1)), np.ascontiguousarray(w_s.transpose(0, 2, 1))
    got = fb.expert_gemm(U.gpu(a), U.gpu(a_s), U.gpu(offsets), U.gpu(turned), U.gpu(turned_s), torch.float32)
    dense = np.zeros((55, 256))
    dc = oracle.e4m3.decode(a) * np.repeat(a_s.astype(np.float64), 128, 1)
    for e in range(3):
        full = oracle.e4m3.decode(w[e]) * np.repeat(np.repeat(w_s[e].astype(np.float64), 128, 0), 128, 1)
        dense[offsets[e]:offsets[e + 1]] = dc[offsets[e]:offsets[e + 1]] @ full
    E.within(got, dense, _tolerance(a, a_s, offsets, turned, turned_s) + np.abs(dense) * 2.0 ** -24)


def test_empty():
    offsets, a, a_s, wg, wu = _inputs(9, [2, 3], 0, 96, 128)
    on = [U.gpu(v) for v in (a, a_s, offsets)]
    none = [U.gpu(v) for v in (a[:0], a_s[:0], np.zeros(3, np.int32))]
    wg, wu = [U.gpu(v) for v in wg], [U.gpu(v) for v in wu]
    assert fb.expert_gemm(*none, *wg).shape == (0, 96) and fb.expert_gated_ffn(*none, *wg, *wu).shape == (0, 96)
    narrow = [wg[0][:, :0].contiguous(), wg[1][:, :0].contiguous()]
    assert fb.expert_gemm(*on, *narrow).shape == (5, 0)


def test_offsets_of_other_contents_touch_nothing_outside():
    """Offsets that expert_sort does not write: unspecified values, and no access outside."""
    _, a, a_s, wg, wu = _inputs(10, [20, 20, 20], 0, 80, 256)
    on, first, second = [U.gpu(v) for v in (a, a_s)], [U.gpu(v) for v in wg], [U.gpu(v) for v in wu]
    for bad in ([-5, 10, 7, 10 ** 9], [60, 0, 60, 0], [2 ** 31 - 1] * 4, [-2 ** 31] * 4, [0, 60, 0, 60]):
        offsets = torch.tensor(bad, dtype=torch.int32, device=G.device())
        for gated in (False, True):
            out, guard = U.guarded_like((60, 80), torch.float32)
            lib, rest = _ffn_lib.lib(), (out.data_ptr(), 0, 60, 3, 80, 256, G.stream())
            ptr = [t.data_ptr() for t in (*on, offsets, *first, *second)]
            assert (lib.fp8_expert_gated_ffn(*ptr, *rest) if gated else lib.fp8_expert_gemm(*ptr[:5], *rest)) == _lib.OK
            torch.cuda.synchronize()
            guard.check_guards()


def test_refusals():
    offsets, a, a_s, wg, wu = _inputs(11, [2, 3], 0, 128, 256)
    a, a_s, offsets, wg, wu = U.gpu(a), U.gpu(a_s), U.gpu(offsets), [U.gpu(v) for v in wg], [U.gpu(v) for v in wu]
    fb.expert_gemm(a, a_s, offsets, *wg)
    for bad in (lambda: fb.expert_gemm(a[:, :128], a_s, offsets, *wg), lambda: fb.expert_gemm(a, a_s[:4], offsets, *wg),
                lambda: fb.expert_gemm(a, a_s, offsets[:2], *wg), lambda: fb.expert_gemm(a, a_s, offsets, wg[0][0], wg[1]),
                lambda: fb.expert_gemm(a, a_s, offsets, wg[0], wg[1][:, :, :1].contiguous()),
                lambda: fb.expert_gated_ffn(a, a_s, offsets, *wg, wu[0][:, :64].contiguous(), wu[1]),
                lambda: fb.expert_gemm(a.cpu(), a_s, offsets, *wg), lambda: fb.expert_gemm(a, a_s, offsets.cpu(), *wg)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fb.expert_gemm(a.float(), a_s, offsets, *wg), lambda: fb.expert_gemm(a, a_s, offsets.long(), *wg),
                lambda: fb.expert_gemm(a, a_s.double(), offsets, *wg), lambda: fb.expert_gemm(a, a_s, offsets, *wg, out_dtype=torch.half)):
        with pytest.raises(TypeError):
            bad()


@pytest.mark.parametrize("counts", [[1, 0, 2], [40, 90, 0], [300, 400, 500]])
def test_graph_replays_and_other_streams(counts):
    """One captured call serves whatever offsets its buffers hold later."""
    n, k, rows = 320, 384, sum(counts)
    G.announce(f"expert products graph {counts}")
    routes = [counts, counts[::-1], [rows, 0, 0], [0, 0, 0]]
    cases = []
    for s, c in enumerate(routes):
        offsets, a, a_s, wg, wu = _inputs(20 + s, c, rows - sum(c), n, k)
        cases.append([U.gpu(v) for v in (a, a_s, offsets, *wg, *wu)])
    static = [t.clone() for t in cases[0]]

    def step(a, a_s, offsets, *w):
        return fb.expert_gemm(a, a_s, offsets, *w[:2]), fb.expert_gated_ffn(a, a_s, offsets, *w)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step(*static)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(other, step(*static)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(*static)
    for case in cases + cases:
        for t, v in zip(static, case):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(captured, step(*case)))
