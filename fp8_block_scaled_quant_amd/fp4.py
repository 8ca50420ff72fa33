"""4-bit weights: E2M1 codes, two to a byte, with one E8M0 scale per 32 weights
of a row, and the matrix-vector product that reads them in the decode step.
"""

import torch

from . import _DTYPE, _ffn_lib, _require_gpu, _stream_handle

GROUP = 32


def fp4_weight_quant(w: torch.Tensor):
    """Quantize a 2-D bf16/fp32 weight [N, K] (K a multiple of 32).

    Returns ``q`` (uint8 [N, K/2], the code of the even weight in a byte's low
    half) and ``s`` (uint8 [N, K/32], E8M0: scale = 2^(s - 127), the smallest
    power of two with max|w| <= 6 * scale).
    """
    _require_gpu(w)
    if w.dtype not in _DTYPE:
        raise TypeError("fp4_weight_quant takes bf16 or fp32 input")
    if w.dim() != 2:
        raise ValueError("weight must be 2-D")
    n, k = w.shape
    if k % GROUP != 0:
        raise ValueError(f"K must be a multiple of {GROUP}")
    q = torch.empty((n, k // 2), dtype=torch.uint8, device=w.device)
    s = torch.empty((n, k // GROUP), dtype=torch.uint8, device=w.device)
    if n and k:
        _ffn_lib.check(_ffn_lib.lib().fp4_weight_quant(w.data_ptr(), _DTYPE[w.dtype], n, k, q.data_ptr(),
                                                       s.data_ptr(), _stream_handle(w)))
    return q, s


def fp4_gemv(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
             bias: torch.Tensor = None) -> torch.Tensor:
    """``y = x W^T (+ bias)`` with the 4-bit weight ``(q, s)`` [N, K].

    ``x`` [..., K] bf16 or fp32: one matrix-vector product per row, made for the
    few rows of a decode step.  ``bias`` [N] has ``out_dtype`` and is added before
    the output rounding.  Returns [..., N].
    """
    _require_gpu(x, q, s, *(() if bias is None else (bias,)))
    if x.dtype not in _DTYPE:
        raise TypeError("fp4_gemv takes bf16 or fp32 activations")
    if out_dtype not in _DTYPE:
        raise TypeError("out_dtype must be float32 or bfloat16")
    if q.dtype != torch.uint8 or s.dtype != torch.uint8:
        raise TypeError("4-bit codes and their scales are uint8")
    k = x.shape[-1]
    if k <= 0 or k % GROUP != 0:
        raise ValueError(f"K must be a positive multiple of {GROUP}")
    if q.dim() != 2 or q.shape[1] != k // 2:
        raise ValueError("q must be [N, K/2] with x's K")
    n = q.shape[0]
    if tuple(s.shape) != (n, k // GROUP):
        raise ValueError(f"s must be [N, K/{GROUP}]")
    if bias is not None and (bias.dtype != out_dtype or tuple(bias.shape) != (n,)):
        raise ValueError(f"bias must be [{n}] of the output dtype {out_dtype}")
    m = x.numel() // k
    y = torch.empty(x.shape[:-1] + (n,), dtype=out_dtype, device=x.device)
    if m and n:
        _ffn_lib.check(_ffn_lib.lib().fp4_gemv(
            x.data_ptr(), _DTYPE[x.dtype], q.data_ptr(), s.data_ptr(), None if bias is None else bias.data_ptr(),
            y.data_ptr(), _DTYPE[out_dtype], m, n, k, _stream_handle(x)))
    return y
