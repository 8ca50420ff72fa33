"""The global norm of many gradient tensors, and clipping by it."""

import torch

from . import _ffn_lib


def _list(tensors):
    return [tensors] if isinstance(tensors, torch.Tensor) else list(tensors)


def grad_norm(grads) -> torch.Tensor:
    """``sqrt`` of the sum of squares over all tensors (a 0-dim float32 tensor)."""
    return _ffn_lib.ext().clip_grad_norm(_list(grads), None, 0.0, 0.0)


def clip_grad_norm(grads, max_norm: float, out=None, eps: float = 1e-6) -> torch.Tensor:
    """Scale all gradients by ``min(1, max_norm / (norm + eps))``, ``norm`` being
    their common 2-norm, which is returned (0-dim float32, before clipping).

    ``grads``: contiguous bf16/fp32 tensors on one GPU, or one tensor; views at
    any offset are fine.  They are clipped in place, and then may not overlap (the
    same tensor twice raises), or into ``out``: tensors of the same shapes and
    dtypes that overlap neither each other nor any gradient (not checked).  A NaN
    gradient makes the norm and every result NaN.
    """
    if not max_norm >= 0.0 or not eps >= 0.0:
        raise ValueError("max_norm and eps must not be negative")
    grads = _list(grads)
    return _ffn_lib.ext().clip_grad_norm(grads, grads if out is None else _list(out), max_norm, eps)
