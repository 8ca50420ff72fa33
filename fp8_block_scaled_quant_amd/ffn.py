"""The gated feed-forward block on block-scaled E4M3 weights: the two products,
the activation and their backward pass, and a training module over them.

A weight is the pair ``weight_quant`` returns: E4M3 codes ``[F, K]`` and FP32
scales ``[ceil(F/128), ceil(K/128)]``.  Everything runs in the library's HIP
kernels; tensors on the CPU raise.
"""

import torch

from . import _DTYPE, _SCALE_FMT, _ffn_lib, weight_quant


def _format(scale_fmt):
    if scale_fmt not in _SCALE_FMT:
        raise ValueError(f"unknown scale_fmt {scale_fmt!r}")
    return _SCALE_FMT[scale_fmt]


def _out(dtype):
    if dtype not in _DTYPE:
        raise TypeError("out_dtype must be float32 or bfloat16")
    return _DTYPE[dtype]


def gated_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_gate_s: torch.Tensor, w_up: torch.Tensor,
              w_up_s: torch.Tensor, scale_fmt=None, out_dtype: torch.dtype = torch.bfloat16, save: bool = False):
    """``h = silu(g) * u`` with ``g = Q(x) W_gate^T`` and ``u = Q(x) W_up^T``.

    ``x`` [..., K] bf16 or fp32, quantized as ``act_quant(x, 128, scale_fmt)``;
    both weights [F, K] with their block scales.  Returns ``h`` [..., F] in
    ``out_dtype``, or with ``save`` the tuple ``(h, g, u)``: what
    ``gated_ffn_backward`` takes.  Autograd does not see the call: ``GatedFFN``
    is the differentiable form.
    """
    return _ffn_lib.ext().gated_ffn(x, w_gate, w_gate_s, w_up, w_up_s, _format(scale_fmt), _out(out_dtype), save)


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
    return _ffn_lib.ext().gated_ffn_backward(dh, x, g, u, w_gate, w_gate_s, w_up, w_up_s, _out(out_dtype), input_grad,
                                             weight_grad)


def _operand(t):
    """``t`` as the library takes it, contiguous and 16-byte aligned: a contiguous
    view (a piece of a flattened ``cat``, say) may start anywhere."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class _FirstOrder(torch.autograd.Function):
    """Hands gradients on; differentiating them raises.

    They come from the native kernels without a graph: without this, a backward
    pass with ``create_graph`` would take them for constants.
    """

    @staticmethod
    def forward(ctx, anchor, *grads):
        return grads

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("GatedFFN has no second-order gradients: its backward pass is not differentiable")


class _GatedFFNFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, scale_fmt, save):
        wg, wg_s = weight_quant(w_gate.detach())
        wu, wu_s = weight_quant(w_up.detach())
        x = _operand(x)
        if not save:   # g and u need not be stored
            return gated_ffn(x, wg, wg_s, wu, wu_s, scale_fmt, x.dtype)
        h, g, u = gated_ffn(x, wg, wg_s, wu, wu_s, scale_fmt, x.dtype, save=True)
        ctx.save_for_backward(x, g, u, wg, wg_s, wu, wu_s)
        return h

    @staticmethod
    def backward(ctx, dh):
        weight_grad = ctx.needs_input_grad[1] or ctx.needs_input_grad[2]
        x, *saved = ctx.saved_tensors
        grads = gated_ffn_backward(_operand(dh), x, *saved, out_dtype=x.dtype,
                                   input_grad=ctx.needs_input_grad[0], weight_grad=weight_grad)
        if torch.is_grad_enabled():   # create_graph; dh need not have a graph for the gradients to depend on x and the weights
            grads = _FirstOrder.apply(torch.zeros((), requires_grad=True), *grads)
        return *grads, None, None


class GatedFFN(torch.nn.Module):
    """Trainable ``h = silu(x W_gate^T) * (x W_up^T)`` with E4M3 products.

    Master weights ``w_gate``, ``w_up`` [F, K] are kept in ``dtype`` (bf16 or
    fp32) and quantized per 128 x 128 tile in every forward pass; activations and
    gradients have the same dtype.  First-order gradients only: differentiating
    them, or forward-mode differentiation, raises.
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
        x = x.to(self.w_gate.dtype)
        # without gradients too: the function refuses a forward-mode tangent, a plain call would drop it
        return _GatedFFNFunction.apply(x, self.w_gate, self.w_up, self.scale_fmt, torch.is_grad_enabled())

    def extra_repr(self) -> str:
        return (f"in_features={self.in_features}, hidden_features={self.hidden_features}, "
                f"dtype={self.w_gate.dtype}, scale_fmt={self.scale_fmt}")
