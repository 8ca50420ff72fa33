"""What the expert operators' C ABI layer hands on: the launcher each entry point
calls, with which arguments, and how a launch error comes back.

Only the host-stub build of the layer can answer; test_expert_abi_sanitized.py makes
it and runs this file with FP8BSQ_EXPERT_TEST_LIB naming it.
"""

import ctypes
import os

import pytest

from fp8_block_scaled_quant_amd import _ffn_lib, _lib

LIB_PATH = os.environ.get("FP8BSQ_EXPERT_TEST_LIB")
P, S = 4096, 0x7000

pytestmark = pytest.mark.skipif(not LIB_PATH, reason="needs the host-stub build (test_expert_abi_sanitized.py)")


@pytest.fixture(scope="module")
def lib():
    lib = _ffn_lib.load_library(LIB_PATH)
    lib._fp8bsq_stub_last.restype = ctypes.c_int
    lib._fp8bsq_stub_last.argtypes = [ctypes.c_char_p, ctypes.c_int, ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_void_p)]
    return lib


def _last(lib, ints, ptrs):
    name, i, p = ctypes.create_string_buffer(64), (ctypes.c_int64 * 16)(), (ctypes.c_void_p * 20)()
    lib._fp8bsq_stub_last(name, 64, i, p)
    return name.value.decode(), list(i)[:ints], [v or 0 for v in list(p)[:ptrs]]


def _at(n):
    return [P + 256 * j for j in range(n)]


def _fails_once(lib, call):
    lib._fp8bsq_stub_fail_next()
    assert call() == _lib.ELAUNCH and call() == _lib.OK


def test_sort(lib):
    ids, off, rows, cho, ws = _at(5)
    need = lib.fp8bsq_expert_sort_workspace(200, 64)
    assert need == 200064
    call = lambda: lib.fp8bsq_expert_sort(ids, 8, 200, 64, off, rows, cho, ws, need, S)  # noqa: E731
    assert call() == _lib.OK and _last(lib, 3, 6) == ("expert_sort", [1, 200, 64], [ids, off, rows, cho, ws, S])
    assert lib.fp8bsq_expert_sort(ids, 8, 200, 64, off, rows, cho, ws, need - 1, S) == _lib.ESCRATCH
    assert lib.fp8bsq_expert_sort(ids, 4, 7, 3, off, rows, cho, None, 0, S) == _lib.OK
    assert _last(lib, 3, 6) == ("expert_sort", [0, 7, 3], [ids, off, rows, cho, 0, S])
    # no choices: the offsets alone
    assert lib.fp8bsq_expert_sort(None, 4, 0, 3, off, None, None, None, 0, S) == _lib.OK
    assert _last(lib, 3, 6) == ("expert_sort", [0, 0, 3], [0, off, 0, 0, 0, S])
    _fails_once(lib, call)


def test_rows(lib):
    x, rows, y, s, w, dy, dw = _at(7)
    dispatch = lambda: lib.fp8bsq_expert_dispatch(x, 1, rows, 5, 2, 70, y, S)  # noqa: E731
    assert dispatch() == _lib.OK and _last(lib, 4, 4) == ("expert_dispatch", [1, 5, 2, 70], [x, rows, y, S])
    quant = lambda: lib.fp8_expert_dispatch_quant(x, 0, 1, rows, 5, 2, 256, y, s, S)  # noqa: E731
    assert quant() == _lib.OK and _last(lib, 5, 5) == ("expert_dispatch_quant", [0, 1, 5, 2, 256], [x, rows, y, s, S])
    combine = lambda: lib.fp8bsq_expert_combine(y, 0, rows, w, 1, 5, 2, 70, x, S)  # noqa: E731
    assert combine() == _lib.OK and _last(lib, 5, 5) == ("expert_combine", [0, 1, 5, 2, 70], [y, rows, w, x, S])
    assert lib.fp8bsq_expert_combine(y, 1, rows, None, 0, 5, 2, 70, x, S) == _lib.OK and _last(lib, 5, 3)[1:] == ([1, 0, 5, 2, 70], [y, rows, 0])
    back = lambda: lib.fp8bsq_expert_combine_backward(x, y, 1, rows, w, 0, 5, 2, 70, dy, dw, S)  # noqa: E731
    assert back() == _lib.OK and _last(lib, 5, 7) == ("expert_combine_backward", [1, 0, 5, 2, 70], [x, y, rows, w, dy, dw, S])
    # y is needed for the weights' gradient alone
    assert lib.fp8bsq_expert_combine_backward(x, None, 1, rows, w, 0, 5, 2, 70, dy, None, S) == _lib.OK
    assert _last(lib, 5, 7)[2] == [x, 0, rows, w, dy, 0, S]
    for call in (dispatch, quant, combine, back):
        _fails_once(lib, call)


def test_products(lib):
    a, a_s, off, w0, w0_s, w1, w1_s, out = _at(8)
    gemm = lambda: lib.fp8_expert_gemm(a, a_s, off, w0, w0_s, out, 0, 9, 3, 70, 256, S)  # noqa: E731
    assert gemm() == _lib.OK and _last(lib, 5, 9) == ("expert_product", [0, 9, 3, 70, 256], [a, a_s, off, w0, w0_s, 0, 0, out, S])
    gated = lambda: lib.fp8_expert_gated_ffn(a, a_s, off, w0, w0_s, w1, w1_s, out, 1, 9, 3, 70, 256, S)  # noqa: E731
    assert gated() == _lib.OK and _last(lib, 5, 9) == ("expert_product", [1, 9, 3, 70, 256], [a, a_s, off, w0, w0_s, w1, w1_s, out, S])
    for call in (gemm, gated):
        _fails_once(lib, call)
