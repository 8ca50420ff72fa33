"""Gradients that share memory: refused where one would be written, since the
workgroups that scale them run in any order; the norm alone takes them."""

import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _flat(dtype=F32, n=4000):
    return torch.ones(n, dtype=dtype, device=G.device())


def _refused(grads):
    before = [t.clone() for t in grads]
    for kw in ({}, {"out": list(grads)}):
        with pytest.raises(ValueError, match="overlap"):
            fb.clip_grad_norm(grads, 0.5, **kw)
    assert all(torch.equal(p, q) for p, q in zip(before, grads))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place(dtype):
    a, b = _flat(dtype), _flat(dtype)
    _refused([a, a])
    _refused([b, a, b[:3], _flat(dtype)])                 # a view of another
    _refused([a[:2001], b, a[2000:]])                     # one element shared
    _refused([a.view(40, 100), b, a[17:18]])
    _refused([a] + [_flat(dtype, 5) for _ in range(300)] + [a])
    norm = fb.clip_grad_norm([a[2000:], b, a[:2000]], 0.5)          # neighbours in any order
    assert abs(float(norm) - 8000 ** 0.5) < 1e-3 and abs(float(fb.grad_norm([a, b])) - 0.5) < 2e-3


def test_in_place_across_types():
    raw = _flat(F32)
    _refused([raw, raw.view(BF)[10:20]])
    fb.clip_grad_norm([raw[:1000], raw[1000:].view(BF)], 1e9)


def test_read_twice_and_written_apart():
    a, o, p = _flat(), _flat(), _flat()
    norm = fb.clip_grad_norm([a, a, a[5:]], 0.5, out=[o, p[:4000], torch.empty_like(a[5:])])
    assert abs(float(norm) - 11995 ** 0.5) < 1e-3 and torch.equal(o, p) and float(a.min()) == 1.0


def test_empty_tensors_overlap_nothing():
    a = _flat()
    fb.clip_grad_norm([a, a[7:7], a[:0], a[4000:]], 1e9)


def test_norm_of_shared_tensors():
    a = _flat()
    assert abs(float(fb.grad_norm([a, a, a[:2000]])) - 100.0) < 1e-4
