"""Sizes beyond the entry points' ranges are refused as such from Python too."""

import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from fp8_block_scaled_quant_amd import _lib
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,f,k", [(1 << 20, 128, 128), (1, 128, (1 << 21) + 128)])
def test_out_of_range_sizes_say_so(m, f, k):
    dev = G.device()
    x = torch.zeros(m, k, dtype=torch.bfloat16, device=dev)
    w = torch.zeros(f, k, dtype=torch.uint8, device=dev)
    s = torch.ones(f // 128, k // 128, device=dev)
    acts = [torch.zeros(m, f, dtype=torch.bfloat16, device=dev)] * 3
    for call in (lambda: fb.gated_ffn(x, w, s, w, s), lambda: fb.gated_ffn_backward(acts[0], x, *acts[1:], w, s, w, s)):
        with pytest.raises(fb.Fp8Error) as e:
            call()
        assert e.value.status == _lib.ERANGE
