"""Every kernel of the experts' products, each at sizes that choose it
(test_expert_plans.py asks the rule itself): values, output types, writes, offsets of
any contents, replays, threads.  Bounds as in test_gpu_expert_products.
"""

import functools
import threading

import numpy as np
import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from fp8_block_scaled_quant_amd import _ffn_lib, _lib
from tests import expert_util as E
from tests import ffn_util as U
from tests import gpu_util as G
from tests.test_gpu_expert_products import _check_gated, _check_gemm, _inputs

pytestmark = pytest.mark.gpu

# an expert's rows around every tile's size, and experts without any
AROUND = (300, 1, 0, 255, 256, 257, 128, 129, 127, 513, 0, 700)
FEW = (8, 1, 0, 16, 17, 2, 0, 9) * 4
SOME = (64, 65, 0, 63, 1, 130, 128, 33) * 2

# (gated, counts, rows behind, n, k) -> the kernel; 256-row tiles also: scales by four blocks or by one
SIZES = {
    (False, AROUND * 3, 9, 1027, 512): "many by four",
    (False, AROUND * 3, 9, 1100, 384): "many",
    (False, AROUND * 2, 9, 1285, 640): "many",
    (True, AROUND, 9, 1803, 512): "many by four",
    (True, AROUND * 2, 9, 643, 1024): "many by four",
    (True, AROUND, 9, 1536, 640): "many",
    (False, SOME, 5, 700, 640): "some",
    (True, SOME, 5, 701, 384): "some",
    (False, FEW, 5, 1300, 640): "few",
    (True, FEW, 5, 1301, 256): "few",
    # and of these the tiles are more than 256, so that workgroups go on to a second: two steps of K blocks each, or more
    (False, (17, 1), 0, 3840, 640): "long32",
    (False, (33, 1, 1, 1), 0, 1901, 1152): "long32",
    (True, (17, 1), 0, 1904, 640): "long32",
    (True, (57, 1, 1, 1, 1, 1, 1, 1), 0, 497, 1152): "long32",
    (False, (33, 1, 1, 1), 0, 3839, 1536): "long64",
    (False, (57, 1, 1, 1, 1, 1, 1, 1), 0, 1920, 1664): "long64",
    (True, (17, 1), 0, 3839, 1536): "long64",
    (True, (17, 1, 17, 1), 0, 1900, 2176): "long64",
}
CASES = list(SIZES)


def _name(case):
    gated, counts, behind, n, k = case
    return f"{SIZES[case]}, {'gated' if gated else 'gemm'}, {sum(counts)} rows of {len(counts)} experts, {behind} behind, {n} x {k}"


@functools.lru_cache(maxsize=None)
def _host(case):
    gated, counts, behind, n, k = case
    offsets, a, a_s, wg, wu = _inputs(len(counts) + n + k, list(counts), behind, n, k)
    return offsets, a, a_s, wg, wu if gated else None


def _device(case):
    """(a, a_s, offsets, weights ...) on the GPU."""
    offsets, a, a_s, wg, wu = _host(case)
    return [U.gpu(v) for v in (a, a_s, offsets, *wg, *(wu or ()))]


def _call(case, args, out=torch.bfloat16):
    return (fb.expert_gated_ffn if case[0] else fb.expert_gemm)(*args, out_dtype=out)


def _check(case, got, out):
    offsets, a, a_s, wg, wu = _host(case)
    if case[0]:
        _check_gated(offsets, a, a_s, wg, wu, out, got)
    else:
        _check_gemm(offsets, a, a_s, wg, out, got)


def _into(case, args, out, dtype):
    """The C entry point's call, into `out`."""
    gated, counts, behind, n, k = case
    lib, rest = _ffn_lib.lib(), (out.data_ptr(), dtype, sum(counts) + behind, len(counts), n, k, G.stream())
    ptr = [t.data_ptr() for t in args]
    assert (lib.fp8_expert_gated_ffn if gated else lib.fp8_expert_gemm)(*ptr, *rest) == _lib.OK
    torch.cuda.synchronize()


@pytest.mark.parametrize("case", CASES, ids=_name)
def test_values_and_guards(case):
    G.announce(_name(case))
    args, shape = _device(case), (sum(case[1]) + case[2], case[3])
    for out, dtype in (("bf16", _lib.BF16), ("f32", _lib.F32)):
        got, guard = U.guarded_like(shape, E.TYPES[out])
        _into(case, args, got, dtype)
        guard.check_guards()
        _check(case, got, out)
        assert torch.equal(got, _call(case, args, E.TYPES[out]))


@pytest.mark.parametrize("case", [c for c in CASES if SIZES[c] == "many by four"], ids=_name)
def test_scales_that_start_anywhere(case):
    """On any four bytes: the scales come a block at a time, and the bits are the same."""
    G.announce(_name(case) + ", unaligned scales")
    args = _device(case)
    want = _call(case, args)
    args[1] = torch.cat([args[1].new_zeros(1), args[1].flatten()])[1:].view(args[1].shape)
    assert args[1].data_ptr() % 16 and torch.equal(_call(case, args), want)


def _disorders(experts, rows):
    rng = np.random.default_rng(experts)
    yield np.full(experts + 1, 2 ** 31 - 1)
    yield np.full(experts + 1, -2 ** 31)
    yield np.full(experts + 1, rows // 2)
    yield np.arange(experts + 1)[::-1] * 7 - 5
    yield np.arange(experts + 1) % 2 * rows
    yield np.r_[rows // 3, rng.integers(-rows, 2 * rows, experts)]
    yield np.sort(rng.integers(0, rows + 1, experts + 1))


@pytest.mark.parametrize("case", CASES, ids=_name)
def test_offsets_of_any_contents(case):
    """Offsets that expert_sort does not write touch nothing outside.  What they give is
    unspecified for a caller; the kernels take the largest so far, within the rows, and a
    mistake there shows in the values."""
    _, counts, behind, n, _ = case
    rows, args = sum(counts) + behind, _device(case)
    args[0][rows - behind:] = 0x38   # 1.0, and 1: with other offsets these rows are some expert's
    args[1][rows - behind:] = 1
    for bad in _disorders(len(counts), rows):
        G.announce(f"{_name(case)}, offsets {bad[:4]} ..")
        order = np.maximum.accumulate(np.clip(bad, 0, rows)).astype(np.int32)
        got, guard = U.guarded_like((rows, n), torch.bfloat16)
        args[2] = U.gpu(bad.astype(np.int32))
        _into(case, args, got, _lib.BF16)
        guard.check_guards()
        args[2] = U.gpu(order)
        assert torch.equal(got[order[0]:], _call(case, args)[order[0]:])
        assert not got[order[-1]:].any()


ONE_EACH = [next(c for c in CASES if SIZES[c] == shape and c[0] == gated)
            for shape in ("many by four", "many", "some", "few", "long32", "long64") for gated in (False, True)]


@pytest.mark.parametrize("case", ONE_EACH, ids=_name)
def test_graph_replays_and_other_streams(case):
    """Equal calls give equal bits; a captured one serves whatever its buffers hold later."""
    G.announce(_name(case) + ", graph")
    _, counts, behind, _, _ = case
    args = _device(case)
    args[0][sum(counts):], args[1][sum(counts):] = 0x38, 1
    routes = [counts, counts[::-1], (0,) * (len(counts) - 1) + (sum(counts),), (0,) * len(counts)]
    routes = [U.gpu(np.r_[0, np.cumsum(c)].astype(np.int32)) for c in routes]
    first = _call(case, args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = _call(case, args)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(first, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = _call(case, args)
    for offsets in routes + routes:
        args[2].copy_(offsets)
        captured.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured, _call(case, args))


def test_threads_on_their_own_streams_match_serial_results():
    cases = [(c, _device(c)) for c in ONE_EACH]
    expect = [_call(*c) for c in cases]
    torch.cuda.synchronize()
    errors = []

    def worker(t):
        try:
            stream = torch.cuda.Stream(device=G.device())
            with torch.cuda.stream(stream):
                for it in range(2 * len(cases)):
                    i = (3 * t + it) % len(cases)
                    got = _call(*cases[i])
                    stream.synchronize()
                    if not torch.equal(got, expect[i]):
                        errors.append(f"thread {t} iteration {it}: {_name(cases[i][0])}")
                        return
        except Exception as e:      # reported below, in the test's own thread
            errors.append(f"thread {t}: {e!r}")

    G.announce(f"4 threads x {len(cases)} sizes, own streams")
    threads = [threading.Thread(target=worker, args=(t,)) for t in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join(timeout=100)
    assert not any(th.is_alive() for th in threads), "a worker thread did not finish"
    torch.cuda.synchronize()
    assert not errors, errors
