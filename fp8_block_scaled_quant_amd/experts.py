"""The feed-forward block behind a router: tokens go to a few of many experts each.

A token's row is sorted to its experts (``expert_sort``, ``expert_dispatch``), each
expert's rows meet its own block-scaled E4M3 weights (``expert_gated_ffn``,
``expert_gemm``), and the weighted results come back to the token
(``expert_combine``).  Nothing is read back to the host in between: the tensors'
sizes depend on the number of choices alone.  Everything runs in the library's HIP
kernels; tensors on the CPU raise.
"""

from typing import NamedTuple

import torch

from . import _DTYPE, _ffn_lib, act_quant, weight_quant
from .ffn import _format, _operand, _out


class ExpertSort(NamedTuple):
    """Where ``expert_sort`` puts n choices.

    The three lie in one allocation, which any of them keeps in use: ``clone`` one that is
    to be kept, saved or resized alone.
    """

    offsets: torch.Tensor   # [num_experts + 1] int32: expert e has the rows offsets[e] .. offsets[e + 1] - 1
    rows: torch.Tensor      # [..., top_k] int32: a choice's row r, or ~r (negative) where it takes no part
    choices: torch.Tensor   # [n] int32: a row's choice


def expert_sort(experts: torch.Tensor, num_experts: int) -> ExpertSort:
    """Sort the choices ``experts`` [..., top_k] (int32 or int64 expert numbers) by
    expert, keeping their order within each.

    A number outside 0 .. num_experts - 1 (a padded token's, or an expert's of
    another rank) takes no part: its row is one of those behind the experts'.  At
    most 1024 experts.
    """
    return ExpertSort(*_ffn_lib.ext().expert_sort(experts, num_experts))


class _FirstOrder(torch.autograd.Function):
    """Hands gradients on; differentiating them raises, where a backward pass with
    ``create_graph`` would otherwise take them for constants."""

    @staticmethod
    def forward(ctx, anchor, *grads):
        return grads

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("expert_combine with weights has no second-order gradients: its backward pass is not differentiable")


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, rows):
        ctx.save_for_backward(rows)
        return _ffn_lib.ext().expert_dispatch(x, rows, False)

    @staticmethod
    def backward(ctx, dy):
        return expert_combine(dy.contiguous(), *ctx.saved_tensors), None


class _Sum(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, rows):
        ctx.save_for_backward(rows)
        return _ffn_lib.ext().expert_combine(y, rows, None, False)

    @staticmethod
    def backward(ctx, dout):
        return expert_dispatch(dout.contiguous(), *ctx.saved_tensors), None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, rows, weights):
        ctx.save_for_backward(y, rows, weights)
        return _ffn_lib.ext().expert_combine(y, rows, weights, False)

    @staticmethod
    def backward(ctx, dout):
        need_y, _, need_weights = ctx.needs_input_grad
        dy, dweights = expert_combine_backward(dout.contiguous(), *ctx.saved_tensors, need_y, need_weights)
        if torch.is_grad_enabled():   # create_graph
            dy, dweights = _FirstOrder.apply(torch.zeros((), requires_grad=True), dy, dweights)
        return dy, None, dweights


def expert_dispatch(x: torch.Tensor, rows: torch.Tensor) -> torch.Tensor:
    """The tokens' rows ``x`` [..., H] (bf16 or fp32) in sorted order, [n, H]: row
    ``rows[t, j]`` is ``x[t]``; the rows behind the experts' are zero.

    ``rows`` [..., top_k] is ``expert_sort``'s.  Differentiable, to any order.
    """
    y = _ffn_lib.ext().expert_dispatch(x, rows, True)
    return _Dispatch.apply(x, rows) if y is None else y   # None: autograd has to see the call


def expert_dispatch_quant(x: torch.Tensor, rows: torch.Tensor, scale_fmt=None):
    """``act_quant(expert_dispatch(x, rows), 128, scale_fmt)``, each token quantized
    once: ``y`` (float8_e4m3fn [n, H]) and ``s`` (float32 [n, H / 128]).  Autograd does
    not see this call, nor the products'."""
    return _ffn_lib.ext().expert_dispatch_quant(x, rows, _format(scale_fmt))


def expert_combine(y: torch.Tensor, rows: torch.Tensor, weights: torch.Tensor = None) -> torch.Tensor:
    """``out[t] = sum_j weights[t, j] * y[rows[t, j]]`` [..., H], in ``y``'s type.

    ``y`` [n, H] bf16 or fp32 in sorted order; ``weights`` [..., top_k] bf16 or fp32,
    or None: ones.  Sums are FP32, in j's order; choices that take no part are left
    out, whatever their rows hold.  Differentiable in ``y`` and ``weights`` (with
    weights, to first order).
    """
    out = _ffn_lib.ext().expert_combine(y, rows, weights, True)
    if out is not None:
        return out
    return _Sum.apply(y, rows) if weights is None else _Combine.apply(y, rows, weights)


def expert_combine_backward(dout: torch.Tensor, y: torch.Tensor, rows: torch.Tensor, weights: torch.Tensor = None,
                            row_grad: bool = True, weight_grad: bool = True):
    """Gradients of ``expert_combine`` from ``dout`` [..., H]: ``dy`` [n, H] (zero in
    the rows behind) and ``dweights`` [..., top_k] (zero where a choice takes no
    part), or None in the place of one that is not asked for."""
    return _ffn_lib.ext().expert_combine_backward(dout, y, rows, weights, row_grad, weight_grad)


def expert_gemm(a: torch.Tensor, a_s: torch.Tensor, offsets: torch.Tensor, b: torch.Tensor, b_s: torch.Tensor,
                out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """``c[r] = a[r] b[e]^T`` for each expert e's rows, ``offsets[e] <= r < offsets[e + 1]``.

    ``a`` [n, K] E4M3 with ``a_s`` [n, K/128]; ``b`` [E, N, K] E4M3 with ``b_s``
    [E, ceil(N/128), K/128]: ``fp8_gemm`` of every expert, in one call.  Returns
    [n, N]; the rows behind are zero.  At most 65535 * 16 rows.

    Equal calls give equal bits.  From K = 640 on, a row's last bits can change with the
    number of rows that come along (another kernel adds the K blocks in another order).
    """
    return _ffn_lib.ext().expert_gemm(a, a_s, offsets, b, b_s, _out(out_dtype))


def expert_gated_ffn(a: torch.Tensor, a_s: torch.Tensor, offsets: torch.Tensor, w_gate: torch.Tensor,
                     w_gate_s: torch.Tensor, w_up: torch.Tensor, w_up_s: torch.Tensor,
                     out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """``h[r] = silu(a[r] w_gate[e]^T) * (a[r] w_up[e]^T)`` for each expert's rows, as
    ``expert_gemm``; both weights [E, F, K].  Returns [n, F]."""
    return _ffn_lib.ext().expert_gated_ffn(a, a_s, offsets, w_gate, w_gate_s, w_up, w_up_s, _out(out_dtype))


class Experts(torch.nn.Module):
    """``out[t] = sum_j weights[t, j] * (silu(x W_gate^T) * (x W_up^T)) W_down^T`` with
    the weights of the experts that ``experts[t]`` names, held as E4M3 codes and
    128 x 128 block scales.

    A call takes up to 65535 * 16 choices, the products' rows.  A token's output does not
    depend on which tokens come with it; with K or F of 640 and more its last bits can
    depend on how many do, as ``expert_gemm``'s.

    Parameters (frozen; this is an inference layer): ``w_gate``, ``w_up`` [E, F, K] and
    ``w_down`` [E, K, F] float8_e4m3fn, with their ``.._scale``.  ``scale_fmt`` is the
    activations' act_quant scale format, ``dtype`` the outputs', bf16 or fp32.
    """

    def __init__(self, num_experts: int, in_features: int, hidden_features: int, dtype: torch.dtype = torch.bfloat16,
                 scale_fmt=None, device=None):
        super().__init__()
        if not 0 < num_experts <= 1024:
            raise ValueError("num_experts must be between 1 and 1024")
        if in_features <= 0 or in_features % 128 != 0 or hidden_features <= 0 or hidden_features % 128 != 0:
            raise ValueError("in_features and hidden_features must be positive multiples of 128")
        if dtype not in _DTYPE:
            raise ValueError("dtype must be bfloat16 or float32")
        _format(scale_fmt)
        self.num_experts, self.in_features, self.hidden_features = num_experts, in_features, hidden_features
        self.dtype, self.scale_fmt = dtype, scale_fmt
        for name, shape in (("w_gate", (hidden_features, in_features)), ("w_up", (hidden_features, in_features)),
                            ("w_down", (in_features, hidden_features))):
            codes = torch.zeros(num_experts, *shape, dtype=torch.float8_e4m3fn, device=device)
            scales = torch.ones(num_experts, shape[0] // 128, shape[1] // 128, device=device)
            setattr(self, name, torch.nn.Parameter(codes, requires_grad=False))
            setattr(self, name + "_scale", torch.nn.Parameter(scales, requires_grad=False))

    @classmethod
    def from_weights(cls, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor, **kwargs) -> "Experts":
        """Quantize bf16/fp32 GPU weights [E, F, K], [E, F, K] and [E, K, F] per 128 x 128 tile."""
        experts, hidden, features = w_gate.shape
        if w_up.shape != w_gate.shape or w_down.shape != (experts, features, hidden):
            raise ValueError("w_up must have w_gate's shape [E, F, K], and w_down be [E, K, F]")
        layer = cls(experts, features, hidden, device=w_gate.device, **kwargs)
        for name, w in (("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down)):
            # whole tiles an expert: those of all experts are the tiles of one tall weight
            codes, scales = weight_quant(w.detach().contiguous().flatten(0, 1))
            getattr(layer, name).data.copy_(codes.view(w.shape))
            getattr(layer, name + "_scale").data.copy_(scales.view(getattr(layer, name + "_scale").shape))
        return layer

    @torch.no_grad()
    def forward(self, x: torch.Tensor, experts: torch.Tensor, weights: torch.Tensor) -> torch.Tensor:
        """``x`` [..., K]; ``experts`` and ``weights`` [..., top_k], a router's choices."""
        if x.shape[-1] != self.in_features:
            raise ValueError(f"expected last dimension {self.in_features}, got {x.shape[-1]}")
        x = _operand(x.to(self.dtype))
        offsets, rows, _ = expert_sort(experts.contiguous(), self.num_experts)
        a, a_s = expert_dispatch_quant(x, rows, self.scale_fmt)
        h = expert_gated_ffn(a, a_s, offsets, self.w_gate, self.w_gate_scale, self.w_up, self.w_up_scale, self.dtype)
        a, a_s = act_quant(h, 128, self.scale_fmt)
        y = expert_gemm(a, a_s, offsets, self.w_down, self.w_down_scale, self.dtype)
        return expert_combine(y, rows, weights.contiguous())

    def extra_repr(self) -> str:
        return (f"num_experts={self.num_experts}, in_features={self.in_features}, hidden_features={self.hidden_features}, "
                f"dtype={self.dtype}, scale_fmt={self.scale_fmt}")
