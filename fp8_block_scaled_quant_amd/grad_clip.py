"""The global norm of many gradient tensors, and clipping by it."""

from array import array

import torch

from . import _DTYPE, _ffn_lib, _stream_handle


def _table(tensors):
    """Addresses of contiguous bf16/fp32 tensors on one GPU, and that device."""
    devices = {t.device for t in tensors}
    if len(devices) != 1:
        raise ValueError("all tensors must be on the same device")
    device = devices.pop()
    if device.type != "cuda":
        raise ValueError("fp8_block_scaled_quant_amd runs on the GPU only: tensor is on " + str(device))
    if not all([t.is_contiguous() for t in tensors]):
        raise ValueError("tensors must be contiguous")
    return array("Q", [t.data_ptr() for t in tensors]), device


def _run(grads, max_norm, out, eps):
    if isinstance(grads, torch.Tensor):
        grads = [grads]
    grads = list(grads)
    if not grads:
        raise ValueError("no gradients given")
    ptrs, device = _table(grads)
    try:
        dtypes = array("i", [_DTYPE[t.dtype] for t in grads])
    except KeyError:
        raise TypeError("gradients must be bf16 or fp32") from None
    numels = array("q", [t.numel() for t in grads])
    outs = None
    if out is grads:
        outs = ptrs
    elif out is not None:
        out = [out] if isinstance(out, torch.Tensor) else list(out)
        if [t.shape for t in out] != [t.shape for t in grads] or [t.dtype for t in out] != [t.dtype for t in grads]:
            raise ValueError("out must match the gradients' number, shapes and dtypes")
        outs, out_device = _table(out)
        if out_device != device:
            raise ValueError("all tensors must be on the same device")
    lib = _ffn_lib.lib()
    nbytes = lib.fp8bsq_clip_grad_norm_workspace(len(grads))
    norm = torch.empty((), dtype=torch.float32, device=device)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    _ffn_lib.check(lib.fp8bsq_clip_grad_norm(
        ptrs.buffer_info()[0], outs.buffer_info()[0] if outs is not None else None, numels.buffer_info()[0],
        dtypes.buffer_info()[0], len(grads), max_norm, eps, norm.data_ptr(), ws.data_ptr(), nbytes,
        _stream_handle(norm)))
    return norm


def grad_norm(grads) -> torch.Tensor:
    """``sqrt`` of the sum of squares over all tensors (a 0-dim float32 tensor)."""
    return _run(grads, 0.0, None, 0.0)


def clip_grad_norm(grads, max_norm: float, out=None, eps: float = 1e-6) -> torch.Tensor:
    """Scale all gradients by ``min(1, max_norm / (norm + eps))``, ``norm`` being
    their common 2-norm, which is returned (0-dim float32, before clipping).

    ``grads``: contiguous bf16/fp32 tensors on one GPU, or one tensor; views at
    any offset are fine.  They are clipped in place, or into ``out`` (tensors of
    the same shapes and dtypes that overlap no gradient).  A NaN gradient makes
    the norm and every result NaN.
    """
    if not max_norm >= 0.0 or not eps >= 0.0:
        raise ValueError("max_norm and eps must not be negative")
    if isinstance(grads, torch.Tensor):
        grads = [grads]
    grads = list(grads)
    return _run(grads, max_norm, grads if out is None else out, eps)
