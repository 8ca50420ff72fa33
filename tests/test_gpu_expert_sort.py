"""expert_sort against a stable sort: equal integers, over sizes from no choice to
many workgroups, both index types, and numbers that are no expert's."""

import numpy as np
import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from fp8_block_scaled_quant_amd import _ffn_lib, _lib
from tests import expert_util as E
from tests import ffn_util as U
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


def _check(ids, experts, got):
    assert isinstance(got, fb.ExpertSort)
    for name, want in zip(("offsets", "rows", "choices"), E.sort(ids, experts)):
        t = getattr(got, name)
        assert t.dtype == torch.int32 and np.array_equal(t.cpu().numpy(), want), name


# one workgroup of one wave, of some, of all; two workgroups and more, with and without a last one that is not full
@pytest.mark.parametrize("tokens,top_k", [(1, 1), (1, 8), (9, 7), (16, 8), (129, 8), (512, 8), (4097, 1), (683, 6), (1024, 8), (2731, 3), (8192, 8),
                                          (70000, 8)])
@pytest.mark.parametrize("experts", [1, 2, 64, 256, 1024])
def test_sizes(tokens, top_k, experts):
    G.announce(f"expert_sort {tokens} x {top_k} of {experts}")
    ids = E.choices(tokens + experts, tokens, top_k, experts, 0.1) if tokens * experts < 1 << 22 else \
        np.random.default_rng(tokens).integers(-2, experts + 2, (tokens, top_k))
    _check(ids, experts, fb.expert_sort(U.gpu(ids), experts))
    _check(ids, experts, fb.expert_sort(U.gpu(ids.astype(np.int32)), experts))


@pytest.mark.parametrize("n", [64, 5000, 40000])
@pytest.mark.parametrize("kind", ["one", "last", "none", "alternating", "far"])
def test_distributions(n, kind):
    """All choices at one expert; none at any; every other one; numbers beyond 32 bits."""
    G.announce(f"expert_sort {kind} {n}")
    ids = {"one": np.full(n, 3), "last": np.full(n, 16), "none": np.full(n, -1), "alternating": np.arange(n) % 2 * 15,
           "far": np.where(np.arange(n) % 3 == 0, (1 << 32) + 5, np.where(np.arange(n) % 3 == 1, -(1 << 40), 7))}[kind].astype(np.int64)
    _check(ids.reshape(-1, 8), 17, fb.expert_sort(U.gpu(ids.reshape(-1, 8)), 17))


def test_no_choices_and_leading_dimensions():
    got = fb.expert_sort(torch.empty(0, 4, dtype=torch.int64, device=G.device()), 5)
    assert got.rows.shape == (0, 4) and got.choices.shape == (0,) and torch.equal(got.offsets.cpu(), torch.zeros(6, dtype=torch.int32))
    ids = E.choices(0, 12, 3, 7)
    got = fb.expert_sort(U.gpu(ids).view(2, 6, 3), 7)
    assert got.rows.shape == (2, 6, 3)
    assert all(torch.equal(a.flatten(), b.flatten()) for a, b in zip(got, fb.expert_sort(U.gpu(ids), 7)))


@pytest.mark.parametrize("n,experts", [(8, 256), (4096, 31), (9000, 1024)])
def test_writes_stay_inside(n, experts):
    G.announce(f"expert_sort guards {n} {experts}")
    ids = E.choices(n, n // 8, 8, experts, 0.2)
    dev = U.gpu(ids)
    lib = _ffn_lib.lib()
    outs = [U.guarded_like((size,), torch.int32) for size in (experts + 1, n, n)]
    nbytes = lib.fp8bsq_expert_sort_workspace(n, experts)
    ws, ws_guard = U.guarded_like((nbytes,), torch.uint8)
    assert lib.fp8bsq_expert_sort(dev.data_ptr(), 8, n, experts, *[t.data_ptr() for t, _ in outs], ws.data_ptr() if nbytes else None, nbytes,
                                  G.stream()) == _lib.OK
    torch.cuda.synchronize()
    for _, guard in outs + [(ws, ws_guard)]:
        guard.check_guards()
    for (t, _), want in zip(outs, E.sort(ids, experts)):
        assert np.array_equal(t.cpu().numpy(), want.reshape(-1))


def test_refusals():
    ids = torch.zeros(4, 2, dtype=torch.int64, device=G.device())
    for bad in (lambda: fb.expert_sort(ids.t(), 4), lambda: fb.expert_sort(ids, 0), lambda: fb.expert_sort(ids.cpu(), 4),
                lambda: fb.expert_sort(ids[0, 0], 4)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        fb.expert_sort(ids.short(), 4)
    for experts in (1025, 1 << 40, (1 << 63) - 1):   # refused, not allocated for
        with pytest.raises(fb.Fp8Error):
            fb.expert_sort(ids, experts)


@pytest.mark.parametrize("tokens", [1, 300, 3000])
def test_graph_replays_and_other_streams(tokens):
    G.announce(f"expert_sort graph {tokens}")
    inputs = [E.choices(s, tokens, 8, 64, 0.1) for s in range(3)]
    static = U.gpu(inputs[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = fb.expert_sort(static, 64)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    _check(inputs[0], 64, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = fb.expert_sort(static, 64)
    for ids in inputs + inputs:
        static.copy_(U.gpu(ids))
        graph.replay()
        torch.cuda.synchronize()
        _check(ids, 64, captured)
        _check(ids, 64, fb.expert_sort(static, 64))
