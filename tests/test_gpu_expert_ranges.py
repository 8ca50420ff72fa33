"""Sizes beyond the expert operators' ranges are refused as such, by the library's
status, and not by a failed allocation of their outputs (several TB here)."""

import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from fp8_block_scaled_quant_amd import _lib
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

MOST_ROWS, MOST_FEATURES = 65535 * 16, 1 << 21


def _zeros(*shape, dtype=torch.uint8):
    return torch.zeros(*shape, dtype=dtype, device=G.device())


def _refused(call):
    with pytest.raises(fb.Fp8Error) as e:
        call()
    assert e.value.status == _lib.ERANGE


@pytest.mark.parametrize("gated", [False, True])
def test_products(gated):
    call = fb.expert_gated_ffn if gated else fb.expert_gemm
    for rows, experts, f in ((MOST_ROWS + 1, 1, MOST_FEATURES), (MOST_ROWS, 1, MOST_FEATURES + 1), (MOST_ROWS, 1025, 1 << 16)):
        G.announce(f"expert products' ranges {rows} {experts} {f} gated={gated}")
        w = (_zeros(experts, f, 128), _zeros(experts, -(-f // 128), 1, dtype=torch.float32))
        a, a_s, offsets = _zeros(rows, 128), _zeros(rows, 1, dtype=torch.float32), _zeros(experts + 1, dtype=torch.int32)
        _refused(lambda: call(a, a_s, offsets, *w, *(w if gated else ())))
        del w, a


@pytest.mark.parametrize("h,top_k", [(MOST_FEATURES + 128, 1 << 20), (1 << 12, 1 << 31)])
def test_rows(h, top_k):
    G.announce(f"expert rows' ranges {h} {top_k}")
    x, rows = _zeros(1, h, dtype=torch.bfloat16), _zeros(1, top_k, dtype=torch.int32)
    _refused(lambda: fb.expert_dispatch(x, rows))
    _refused(lambda: fb.expert_dispatch_quant(x, rows))


def test_rows_too_long_to_combine():
    h = MOST_FEATURES + 1
    y, rows, dout = _zeros(2, h, dtype=torch.bfloat16), _zeros(1, 2, dtype=torch.int32), _zeros(1, h, dtype=torch.bfloat16)
    _refused(lambda: fb.expert_combine(y, rows))
    _refused(lambda: fb.expert_combine_backward(dout, y, rows))


def test_nothing_to_do_is_within_every_range():
    w, w_s = _zeros(1025, 1, 128), _zeros(1025, 1, 1, dtype=torch.float32)
    none = _zeros(0, 128), _zeros(0, 1, dtype=torch.float32), _zeros(1026, dtype=torch.int32)
    assert fb.expert_gemm(*none, w, w_s).shape == (0, 1) and fb.expert_gated_ffn(*none, w, w_s, w, w_s).shape == (0, 1)
    h, rows = MOST_FEATURES + 128, _zeros(0, 2, dtype=torch.int32)
    x = _zeros(0, h, dtype=torch.bfloat16)
    assert fb.expert_dispatch(x, rows).shape == (0, h) and fb.expert_combine(x, rows).shape == (0, h)
    assert fb.expert_dispatch_quant(x, rows)[0].shape == (0, h)
