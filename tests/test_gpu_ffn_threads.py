"""The feed-forward operators called by several host threads, each on its own stream
with its own inputs: every result is bit-identical to the same call made alone."""

import threading

import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from tests import ffn_util as U
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

# decode; 128 x 128 tiles; these with the contraction in parts; 256 x 256 tiles
SHAPES = [(1, 2304, 1024), (40, 640, 512), (65, 1024, 896), (1037, 384, 3456)]


def _case(i, m, f, k):
    gen = torch.Generator(G.device()).manual_seed(i)
    randn = lambda *shape: torch.randn(*shape, generator=gen, device=G.device())  # noqa: E731
    return {"x": randn(m, k).bfloat16(), "dh": (randn(m, f) * 1e-3).bfloat16(), "w": [U.gpu(v) for j in (0, 1) for v in U.weight(2 * i + j, f, k)],
            "wide": randn(f, k).bfloat16(), "grads": [randn(100 * j + i + 1) for j in range(40)]}


def _run(c):
    h, g, u = fb.gated_ffn(c["x"], *c["w"], "ue8m0", save=True)
    grads = fb.gated_ffn_backward(c["dh"], c["x"], g, u, *c["w"])
    q, s = fb.fp4_weight_quant(c["wide"])
    y = fb.fp4_gemv(c["x"], q, s, torch.float32)
    outs = [torch.empty_like(t) for t in c["grads"]]
    norm = fb.clip_grad_norm(c["grads"], 1.0, out=outs)
    return h, g, u, *grads, q, s, y, norm, *outs


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
