"""Loading ``libfp8bsq_ffn.so`` (the feed-forward operators) for ctypes.

Built in-tree beside ``libfp8bsq.so``, which it links and finds next to itself.
Loading it initializes nothing on the GPU.
"""

import ctypes
import os

from . import _lib

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfp8bsq_ffn.so")

# every symbol include/fp8bsq_ffn.h declares
EXPORTS = ("fp8_gated_ffn", "fp8_gated_ffn_workspace", "fp8_gated_ffn_backward", "fp8_gated_ffn_backward_workspace",
           "fp4_weight_quant", "fp4_gemv", "fp8bsq_clip_grad_norm", "fp8bsq_clip_grad_norm_workspace",
           "fp8bsq_expert_sort", "fp8bsq_expert_sort_workspace", "fp8bsq_expert_dispatch", "fp8_expert_dispatch_quant",
           "fp8bsq_expert_combine", "fp8bsq_expert_combine_backward", "fp8_expert_gemm", "fp8_expert_gated_ffn")

_LIB = None


def load_library(path: str = None) -> ctypes.CDLL:
    """Load the shared library and declare argument types; raises if absent."""
    global _LIB
    if _LIB is not None and path is None:
        return _LIB
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise ImportError(
            f"{p} is missing: build the HIP library first (python -m fp8_block_scaled_quant_amd.build)")
    lib = ctypes.CDLL(p)
    i64, i32, vp, size, f32 = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_float
    lib.fp8_gated_ffn.argtypes = [vp, i32, i32, vp, vp, vp, vp, vp, vp, vp, i32, i64, i64, i64, vp, size, vp]
    lib.fp8_gated_ffn_backward.argtypes = [vp, vp, vp, vp, i32, vp, vp, vp, vp, vp, vp, vp, i32, i64, i64, i64,
                                           vp, size, vp]
    lib.fp4_weight_quant.argtypes = [vp, i32, i64, i64, vp, vp, vp]
    lib.fp4_gemv.argtypes = [vp, i32, vp, vp, vp, vp, i32, i64, i64, i64, vp]
    lib.fp8bsq_clip_grad_norm.argtypes = [vp, vp, vp, vp, i64, f32, f32, vp, vp, size, vp]
    lib.fp8bsq_expert_sort.argtypes = [vp, i32, i64, i64, vp, vp, vp, vp, size, vp]
    lib.fp8bsq_expert_dispatch.argtypes = [vp, i32, vp, i64, i64, i64, vp, vp]
    lib.fp8_expert_dispatch_quant.argtypes = [vp, i32, i32, vp, i64, i64, i64, vp, vp, vp]
    lib.fp8bsq_expert_combine.argtypes = [vp, i32, vp, vp, i32, i64, i64, i64, vp, vp]
    lib.fp8bsq_expert_combine_backward.argtypes = [vp, vp, i32, vp, vp, i32, i64, i64, i64, vp, vp, vp]
    lib.fp8_expert_gemm.argtypes = [vp, vp, vp, vp, vp, vp, i32, i64, i64, i64, i64, vp]
    lib.fp8_expert_gated_ffn.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i64, i64, i64, i64, vp]
    for name in ("fp8_gated_ffn", "fp8_gated_ffn_backward", "fp4_weight_quant", "fp4_gemv", "fp8bsq_clip_grad_norm",
                 "fp8bsq_expert_sort", "fp8bsq_expert_dispatch", "fp8_expert_dispatch_quant", "fp8bsq_expert_combine",
                 "fp8bsq_expert_combine_backward", "fp8_expert_gemm", "fp8_expert_gated_ffn"):
        getattr(lib, name).restype = i32
    for name in ("fp8_gated_ffn_workspace", "fp8_gated_ffn_backward_workspace"):
        getattr(lib, name).argtypes = [i64, i64, i64]
        getattr(lib, name).restype = size
    lib.fp8bsq_clip_grad_norm_workspace.argtypes = [i64]
    lib.fp8bsq_expert_sort_workspace.argtypes = [i64, i64]
    for name in ("fp8bsq_clip_grad_norm_workspace", "fp8bsq_expert_sort_workspace"):
        getattr(lib, name).restype = size
    if path is None:
        _LIB = lib
    return lib


def lib() -> ctypes.CDLL:
    return _LIB or load_library()


_EXT = None


def ext():
    """The native Python binding over the library (``_ffn_ext.so``); raises if absent."""
    global _EXT
    if _EXT is None:
        load_library()
        _lib.lib()
        try:
            from . import _ffn_ext
        except ImportError as e:
            raise ImportError("fp8_block_scaled_quant_amd/_ffn_ext.so is missing or does not load: build the HIP "
                              "library first (python -m fp8_block_scaled_quant_amd.build)") from e
        _EXT = _ffn_ext
    return _EXT
