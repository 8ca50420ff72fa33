"""The expert operators called by several host threads, each on its own stream with
its own inputs: every result is bit-identical to the same call made alone."""

import threading

import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from tests import expert_util as E
from tests import ffn_util as U
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

# tokens, top_k, experts, features: tiles of 16, 64 and 256 rows; a sort over several workgroups
SHAPES = [(1, 8, 16, 256), (60, 4, 8, 384), (700, 4, 8, 256), (2100, 3, 6, 128)]


def _case(i, tokens, top_k, experts, k):
    w = [U.gpu(v) for j in (0, 1) for v in E.weights(2 * i + j, experts, 260, k)]
    return {"ids": U.gpu(E.choices(i, tokens, top_k, experts, 0.1)), "experts": experts, "x": E.normal(i, (tokens, k), "bf16").to(G.device()), "w": w,
            "share": E.normal(i + 9, (tokens, top_k), "f32").to(G.device()), "dout": E.normal(i + 5, (tokens, 260), "bf16").to(G.device())}


def _run(c):
    s = fb.expert_sort(c["ids"], c["experts"])
    a, a_s = fb.expert_dispatch_quant(c["x"], s.rows)
    h = fb.expert_gated_ffn(a, a_s, s.offsets, *c["w"])
    g = fb.expert_gemm(a, a_s, s.offsets, *c["w"][:2])
    out = fb.expert_combine(h, s.rows, c["share"])
    return *s, a.view(torch.uint8), a_s, h, g, out, *fb.expert_combine_backward(c["dout"], g, s.rows, c["share"]), fb.expert_dispatch(c["x"], s.rows)


def test_threads_on_their_own_streams_match_serial_results():
    cases = [_case(i, *shape) for i, shape in enumerate(SHAPES)]
    expect = [_run(c) for c in cases]
    torch.cuda.synchronize()
    errors = []

    def worker(t):
        try:
            stream = torch.cuda.Stream(device=G.device())
            with torch.cuda.stream(stream):
                for it in range(12):
                    i = (t + it) % len(cases)
                    got = _run(cases[i])
                    stream.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, expect[i])):
                        errors.append(f"thread {t} iteration {it} shape {SHAPES[i]}")
                        return
        except Exception as e:      # reported below, in the test's own thread
            errors.append(f"thread {t}: {e!r}")

    G.announce(f"4 threads x {len(SHAPES)} shapes, own streams")
    threads = [threading.Thread(target=worker, args=(t,)) for t in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join(timeout=120)
    assert not any(th.is_alive() for th in threads), "a worker thread did not finish"
    torch.cuda.synchronize()
    assert not errors, errors
