"""Gradient lists that fill the tables of kernel arguments to the last entry: every
tensor's value tells which entry was read, eagerly and in a replayed graph."""

import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("count", [255, 256, 257, 512, 600])
def test_every_entry_eagerly_and_from_a_graph(count):
    G.announce(f"clip table of {count} tensors")
    dev = G.device()
    first = [torch.full((3 + i % 5,), (i + 1) / 64, device=dev, dtype=(torch.float32, torch.bfloat16)[i % 7 == 0]) for i in range(count)]
    grads, outs = [t.clone() for t in first], [torch.empty_like(t) for t in first]

    def check(norm, factor):
        total = sum(float((t.double() * factor).square().sum()) for t in first) ** 0.5
        assert abs(float(norm) - total) <= 1e-6 * total
        for t, o in zip(first, outs):
            want = t.double() * factor / (2 * factor)
            assert torch.all((o.double() - want).abs() <= want.abs() * (2.0 ** -8 if t.dtype == torch.bfloat16 else 2.0 ** -21))

    half = sum(float(t.double().square().sum()) for t in first) ** 0.5 / 2   # clips to this norm
    check(fb.clip_grad_norm(grads, half, out=outs, eps=0.0), 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fb.clip_grad_norm(grads, half, out=outs, eps=0.0)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = fb.clip_grad_norm(grads, half, out=outs, eps=0.0)
    for factor in (1, 4, 2, 8):
        for g, t in zip(grads, first):
            g.copy_(t * factor)
        [o.zero_() for o in outs]
        graph.replay()
        torch.cuda.synchronize()
        check(norm, factor)
