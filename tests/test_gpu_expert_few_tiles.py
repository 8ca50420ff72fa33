"""The experts' products where few tiles cover the outputs and K is long: K blocks that
do and do not fill steps of four, more tiles than an even spread would take, and the
sizes from which on the other kernels take over.  Bounds as in
test_gpu_expert_products.
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from tests import ffn_util as U
from tests import gpu_util as G
from tests.test_gpu_expert_products import _inputs, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [512, 640, 768, 896, 1024, 1152, 2176])
@pytest.mark.parametrize("counts", [[1], [0, 2, 1, 0], [16], [17, 0, 15], [40, 1, 1, 0, 3], [130], [0, 0]])
def test_blocks(counts, k):
    G.announce(f"few tiles {counts} k={k}")
    _run(21, counts, 3, 100, k, "bf16")


@pytest.mark.parametrize("n", [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_widths(n, out):
    G.announce(f"few tiles n={n} {out}")
    _run(22, [1, 0, 18], 2, n, 768, out)


# one expert's 17 rows are two tiles, where the average says hardly more than one: a
# workgroup gets several tiles of the sizes at which 32 and 64 rows of weights still fit
@pytest.mark.parametrize("n,k", [(1904, 640), (3840, 640), (3840, 1536), (7680, 1536)])
def test_more_tiles_than_workgroups(n, k):
    G.announce(f"few tiles {n} x {k}")
    _run(23, [17, 1], 1, n, k, "bf16")


# around the largest numbers of tiles, and past them
@pytest.mark.parametrize("counts", [[1, 2], [20, 33], [0, 1, 100]])
@pytest.mark.parametrize("n,k", [(4096, 640), (4112, 1536), (8200, 640), (8200, 1664)])
def test_borders(counts, n, k):
    G.announce(f"few tiles {counts} {n} x {k}")
    _run(24, counts, 2, n, k, "bf16")


def test_many_experts():
    G.announce("few tiles, 1024 experts")
    counts = [0] * 1024
    for e in (0, 5, 511, 512, 1000, 1023):
        counts[e] = 1 + e % 3
    _run(25, counts, 4, 48, 640, "bf16")


@pytest.mark.parametrize("k", [640, 2048])
def test_repeats(k):
    """Equal calls, also replayed, give equal bits."""
    G.announce(f"few tiles, repeated, k={k}")
    offsets, a, a_s, wg, wu = _inputs(26, [3, 0, 17, 1], 2, 200, k)
    on = [U.gpu(v) for v in (a, a_s, offsets)]
    gate, up = [U.gpu(v) for v in wg], [U.gpu(v) for v in wu]
    call = lambda: (fb.expert_gemm(*on, *gate), fb.expert_gated_ffn(*on, *gate, *up))
    first = call()
    for _ in range(20):
        assert all(torch.equal(x, y) for x, y in zip(first, call()))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(3):
        for x in got:
            x.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(first, got))


@pytest.mark.parametrize("offsets", [[0, 50, 20, 90], [-5, 3, 1000, 7], [9, 9, 9, 9], [2 ** 31 - 1, -2 ** 31, 40, 40]])
def test_offsets_out_of_order(offsets):
    """Unspecified outputs, but the call ends and takes no other rows than there are."""
    G.announce(f"few tiles, offsets {offsets}")
    rows, n, k = 60, 72, 768
    _, a, a_s, wg, wu = _inputs(27, [20, 20, 20], 0, n, k)
    on = [U.gpu(v) for v in (a, a_s, np.array(offsets, np.int64).astype(np.int32))]
    got = fb.expert_gated_ffn(*on, *[U.gpu(v) for v in (*wg, *wu)])
    torch.cuda.synchronize()
    assert got.shape == (rows, n)
