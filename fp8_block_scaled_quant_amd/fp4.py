"""4-bit weights: E2M1 codes, two to a byte, with one E8M0 scale per 32 weights
of a row, and the matrix-vector product that reads them in the decode step.
"""

import torch

from . import _DTYPE, _ffn_lib


def fp4_weight_quant(w: torch.Tensor):
    """Quantize a 2-D bf16/fp32 weight [N, K] (K a multiple of 32).

    Returns ``q`` (uint8 [N, K/2], the code of the even weight in a byte's low
    half) and ``s`` (uint8 [N, K/32], E8M0: scale = 2^(s - 127), the smallest
    power of two with max|w| <= 6 * scale).
    """
    return _ffn_lib.ext().fp4_weight_quant(w)


def fp4_gemv(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
             bias: torch.Tensor = None) -> torch.Tensor:
    """``y = x W^T (+ bias)`` with the 4-bit weight ``(q, s)`` [N, K].

    ``x`` [..., K] bf16 or fp32: one matrix-vector product per row, made for the
    few rows of a decode step.  ``bias`` [N] has ``out_dtype`` and is added before
    the output rounding.  Returns [..., N].
    """
    if out_dtype not in _DTYPE:
        raise TypeError("out_dtype must be float32 or bfloat16")
    return _ffn_lib.ext().fp4_gemv(x, q, s, _DTYPE[out_dtype], bias)
