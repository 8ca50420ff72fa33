"""The gated feed-forward block on block-scaled E4M3 weights: the two products,
the activation and their backward pass, and a training module over them.

A weight is the pair ``weight_quant`` returns: E4M3 codes ``[F, K]`` and FP32
scales ``[ceil(F/128), ceil(K/128)]``.  Everything runs in the library's HIP
kernels; tensors on the CPU raise.
"""

import torch

from . import _DTYPE, _SCALE_FMT, _codes, _ffn_lib, _require_gpu, _stream_handle, weight_quant


def _weight(name, w, w_s, f, k):
    if w.dim() != 2 or tuple(w.shape) != (f, k):
        raise ValueError(f"{name} must be [{f}, {k}], got {tuple(w.shape)}")
    if w_s.dtype != torch.float32:
        raise TypeError("scales must be float32")
    if tuple(w_s.shape) != (-(-f // 128), k // 128):
        raise ValueError(f"{name}'s scales must be [ceil(F/128), K/128]")


def gated_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_gate_s: torch.Tensor, w_up: torch.Tensor,
              w_up_s: torch.Tensor, scale_fmt=None, out_dtype: torch.dtype = torch.bfloat16, save: bool = False):
    """``h = silu(g) * u`` with ``g = Q(x) W_gate^T`` and ``u = Q(x) W_up^T``.

    ``x`` [..., K] bf16 or fp32, quantized as ``act_quant(x, 128, scale_fmt)``;
    both weights [F, K] with their block scales.  Returns ``h`` [..., F] in
    ``out_dtype``, or with ``save`` the tuple ``(h, g, u)``: what
    ``gated_ffn_backward`` takes.
    """
    w_gate, w_up = _codes(w_gate), _codes(w_up)
    _require_gpu(x, w_gate, w_gate_s, w_up, w_up_s)
    if x.dtype not in _DTYPE:
        raise TypeError("gated_ffn takes bf16 or fp32 activations")
    if scale_fmt not in _SCALE_FMT:
        raise ValueError(f"unknown scale_fmt {scale_fmt!r}")
    if out_dtype not in _DTYPE:
        raise TypeError("out_dtype must be float32 or bfloat16")
    k = x.shape[-1]
    if k <= 0 or k % 128 != 0:
        raise ValueError("K must be a positive multiple of 128")
    f = w_gate.shape[0]
    _weight("w_gate", w_gate, w_gate_s, f, k)
    _weight("w_up", w_up, w_up_s, f, k)
    m = x.numel() // k
    shape = x.shape[:-1] + (f,)
    h = torch.empty(shape, dtype=out_dtype, device=x.device)
    g, u = (torch.empty_like(h), torch.empty_like(h)) if save else (None, None)
    if m and f:
        lib = _ffn_lib.lib()
        nbytes = lib.fp8_gated_ffn_workspace(m, f, k)
        # torch's allocator keeps the workspace from being reused until the
        # work queued on this stream has passed it
        ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
        _ffn_lib.check(lib.fp8_gated_ffn(
            x.data_ptr(), _DTYPE[x.dtype], _SCALE_FMT[scale_fmt], w_gate.data_ptr(), w_gate_s.data_ptr(),
            w_up.data_ptr(), w_up_s.data_ptr(), h.data_ptr(), g.data_ptr() if save else None,
            u.data_ptr() if save else None, _DTYPE[out_dtype], m, f, k, ws.data_ptr(), nbytes, _stream_handle(x)))
    return (h, g, u) if save else h


def gated_ffn_backward(dh: torch.Tensor, x: torch.Tensor, g: torch.Tensor, u: torch.Tensor, w_gate: torch.Tensor,
                       w_gate_s: torch.Tensor, w_up: torch.Tensor, w_up_s: torch.Tensor,
                       out_dtype: torch.dtype = torch.bfloat16, input_grad: bool = True, weight_grad: bool = True):
    """Gradients of ``gated_ffn`` from ``dh`` [..., F], its input ``x`` [..., K]
    and the ``g``, ``u`` it saved.

    Returns ``(dx [..., K], dw_gate [F, K], dw_up [F, K])`` in ``out_dtype``;
    with ``input_grad`` or ``weight_grad`` false, None in their place (and the
    work they need is not done).  The three products run on E4M3: the gradients
    (and, for the weights, ``x``) are rounded with one power-of-two scale per 128
    values along each contraction.  F must be a multiple of 128.
    """
    w_gate, w_up = _codes(w_gate), _codes(w_up)
    _require_gpu(dh, x, g, u, w_gate, w_gate_s, w_up, w_up_s)
    if dh.dtype not in _DTYPE or any(t.dtype != dh.dtype for t in (x, g, u)):
        raise TypeError("dh, x, g and u must all be bf16 or all fp32")
    if out_dtype not in _DTYPE:
        raise TypeError("out_dtype must be float32 or bfloat16")
    f, k = dh.shape[-1], x.shape[-1]
    if f <= 0 or f % 128 != 0 or k <= 0 or k % 128 != 0:
        raise ValueError("F and K must be positive multiples of 128")
    if g.shape != dh.shape or u.shape != dh.shape or x.shape[:-1] != dh.shape[:-1]:
        raise ValueError("g and u must have dh's shape, and x its leading dimensions")
    _weight("w_gate", w_gate, w_gate_s, f, k)
    _weight("w_up", w_up, w_up_s, f, k)
    m = x.numel() // k
    dx = torch.empty(x.shape, dtype=out_dtype, device=x.device) if input_grad else None
    dwg, dwu = (torch.empty((f, k), dtype=out_dtype, device=x.device) for _ in range(2)) if weight_grad else (None, None)
    if weight_grad or (input_grad and m):
        lib = _ffn_lib.lib()
        nbytes = lib.fp8_gated_ffn_backward_workspace(m, f, k)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
        _ffn_lib.check(lib.fp8_gated_ffn_backward(
            dh.data_ptr(), x.data_ptr(), g.data_ptr(), u.data_ptr(), _DTYPE[dh.dtype], w_gate.data_ptr(),
            w_gate_s.data_ptr(), w_up.data_ptr(), w_up_s.data_ptr(), dx.data_ptr() if input_grad else None,
            dwg.data_ptr() if weight_grad else None, dwu.data_ptr() if weight_grad else None, _DTYPE[out_dtype],
            m, f, k, ws.data_ptr(), nbytes, _stream_handle(x)))
    return dx, dwg, dwu


class _GatedFFNFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, scale_fmt):
        wg, wg_s = weight_quant(w_gate.detach())
        wu, wu_s = weight_quant(w_up.detach())
        x = x.contiguous()
        h, g, u = gated_ffn(x, wg, wg_s, wu, wu_s, scale_fmt, x.dtype, save=True)
        ctx.save_for_backward(x, g, u, wg, wg_s, wu, wu_s)
        return h

    @staticmethod
    def backward(ctx, dh):
        weight_grad = ctx.needs_input_grad[1] or ctx.needs_input_grad[2]
        x, *saved = ctx.saved_tensors
        dx, dwg, dwu = gated_ffn_backward(dh.contiguous(), x, *saved, out_dtype=x.dtype,
                                          input_grad=ctx.needs_input_grad[0], weight_grad=weight_grad)
        return dx, dwg, dwu, None


class GatedFFN(torch.nn.Module):
    """Trainable ``h = silu(x W_gate^T) * (x W_up^T)`` with E4M3 products.

    Master weights ``w_gate``, ``w_up`` [F, K] are kept in ``dtype`` (bf16 or
    fp32) and quantized per 128 x 128 tile in every forward pass; activations and
    gradients have the same dtype.
    """

    def __init__(self, in_features: int, hidden_features: int, dtype: torch.dtype = torch.bfloat16, scale_fmt=None,
                 device=None):
        super().__init__()
        if in_features <= 0 or in_features % 128 != 0 or hidden_features <= 0 or hidden_features % 128 != 0:
            raise ValueError("in_features and hidden_features must be positive multiples of 128")
        if dtype not in _DTYPE:
            raise ValueError("dtype must be bfloat16 or float32")
        if scale_fmt not in _SCALE_FMT:
            raise ValueError(f"unknown scale_fmt {scale_fmt!r}")
        self.in_features, self.hidden_features, self.scale_fmt = in_features, hidden_features, scale_fmt
        shape = (hidden_features, in_features)
        self.w_gate = torch.nn.Parameter(torch.randn(shape, dtype=dtype, device=device) * in_features ** -0.5)
        self.w_up = torch.nn.Parameter(torch.randn(shape, dtype=dtype, device=device) * in_features ** -0.5)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        if x.shape[-1] != self.in_features:
            raise ValueError(f"expected last dimension {self.in_features}, got {x.shape[-1]}")
        return _GatedFFNFunction.apply(x.to(self.w_gate.dtype), self.w_gate, self.w_up, self.scale_fmt)

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, hidden_features={self.hidden_features}, "
                f"dtype={self.w_gate.dtype}, scale_fmt={self.scale_fmt}")
