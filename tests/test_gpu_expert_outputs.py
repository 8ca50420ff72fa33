"""The expert operators' outputs as tensors that a program keeps: saved and loaded,
copied, made in inference mode, used on another stream, and checkpointed through."""

import copy
import io

import pytest
import torch
from torch.utils.checkpoint import checkpoint

import fp8_block_scaled_quant_amd as fb
from tests import expert_util as E
from tests import ffn_util as U
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


def _bits(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


def _same(got, want):
    return all(a.dtype == b.dtype and torch.equal(_bits(a), _bits(b)) for a, b in zip(got, want, strict=True))


def _case(tokens, h=256, top_k=3, experts=5):
    ids = U.gpu(E.choices(tokens, tokens, top_k, experts, 0.2))
    return ids, E.normal(1, (tokens, h), "bf16").to(G.device()), torch.softmax(E.normal(2, (tokens, top_k), "f32"), 1).to(G.device())


def _all(ids, x, w):
    s = fb.expert_sort(ids, 5)
    a, a_s = fb.expert_dispatch_quant(x, s.rows)
    y = fb.expert_dispatch(x, s.rows)
    return [*s, a, a_s, y, fb.expert_combine(y, s.rows, w), *fb.expert_combine_backward(x, y, s.rows, w)]


# outputs of the smallest calls, and of ones with 2^20 elements and more
SIZES = [1, 40, 1500]


@pytest.mark.parametrize("tokens", SIZES)
def test_saved_loaded_and_copied(tokens):
    """Together and alone; a tensor written in place changes no other."""
    got = _all(*_case(tokens))
    want = [t.clone() for t in got]
    file = io.BytesIO()
    torch.save(got, file)
    file.seek(0)
    assert _same(torch.load(file, weights_only=True), want) and _same(copy.deepcopy(got), want)
    for i, t in enumerate(got):
        file = io.BytesIO()
        torch.save(t, file)
        file.seek(0)
        assert _same([torch.load(file, weights_only=True)], [want[i]])
        versions = [o._version for o in got]
        t.zero_()
        assert [o._version for o in got] == [v + (i == j) for j, v in enumerate(versions)]
        assert _same(got[i + 1:], want[i + 1:])


@pytest.mark.parametrize("tokens", SIZES)
def test_inference_mode(tokens):
    case = _case(tokens)
    want = _all(*case)
    with torch.inference_mode():
        got = _all(*case)
        assert all(t.is_inference() for t in got)
        assert _same(got, want)
    assert not any(t.is_inference() or t.requires_grad for t in want)


@pytest.mark.parametrize("tokens", SIZES)
def test_freed_while_another_stream_reads(tokens):
    """record_stream holds each output's memory for the stream that still reads it."""
    case = _case(tokens)
    want = [t.clone() for t in _all(*case)]
    side = torch.cuda.Stream()
    busy = torch.randn(2048, 2048, device=G.device())
    for _ in range(3):
        got = _all(*case)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(10):
                busy = torch.tanh(busy @ busy)
            kept = []
            for t in got:
                t.record_stream(side)
                kept.append(t.clone())
        del got, t
        for _ in range(4):   # what a freed block would be handed out for
            other = _all(case[0].roll(1, 0), case[1] + 1, case[2])
            del other
        torch.cuda.synchronize()
        assert _same(kept, want)


def test_checkpointed():
    ids, x, w = _case(37)
    rows = fb.expert_sort(ids, 5).rows
    x, w = x.float().requires_grad_(), w.requires_grad_()

    def step(x, w):
        return fb.expert_combine(torch.tanh(fb.expert_dispatch(x, rows)), rows, w)

    want = torch.autograd.grad(step(x, w).square().sum(), (x, w))
    assert _same(torch.autograd.grad(checkpoint(step, x, w, use_reentrant=False).square().sum(), (x, w)), want)


def test_layer_copied_and_restored():
    gen = torch.Generator(G.device()).manual_seed(1)
    layer = fb.Experts.from_weights(*(torch.randn(5, *s, generator=gen, device=G.device()) * 0.06 for s in ((384, 256), (384, 256), (256, 384))))
    ids, x, w = _case(20)
    want = layer(x, ids, w)
    again = fb.Experts(5, 256, 384, device=G.device())
    again.load_state_dict(layer.state_dict())
    assert torch.equal(again(x, ids, w), want) and torch.equal(copy.deepcopy(layer)(x, ids, w), want)
