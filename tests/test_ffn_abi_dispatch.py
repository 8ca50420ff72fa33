"""What the feed-forward C ABI layer hands on: the launcher each entry point calls,
with which arguments, and how a launch error comes back.

Only the host-stub build of the layer (ffn_abi.cpp over
tests/ffn_abi_host_stub.cpp) can answer; test_ffn_abi_sanitized.py makes it, under
AddressSanitizer and UndefinedBehaviorSanitizer, and runs this file with
FP8BSQ_FFN_TEST_LIB naming it.
"""

import array
import ctypes
import os

import pytest

from fp8_block_scaled_quant_amd import _ffn_lib, _lib

LIB_PATH = os.environ.get("FP8BSQ_FFN_TEST_LIB")
P, S = 4096, 0x7000
BIG = 1 << 40

pytestmark = pytest.mark.skipif(not LIB_PATH, reason="needs the host-stub build (test_ffn_abi_sanitized.py)")


@pytest.fixture(scope="module")
def lib():
    lib = _ffn_lib.load_library(LIB_PATH)
    lib._fp8bsq_stub_last.restype = ctypes.c_int
    lib._fp8bsq_stub_last.argtypes = [ctypes.c_char_p, ctypes.c_int, ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_void_p)]
    return lib


def _last(lib):
    name, ints, ptrs = ctypes.create_string_buffer(64), (ctypes.c_int64 * 16)(), (ctypes.c_void_p * 20)()
    n = lib._fp8bsq_stub_last(name, 64, ints, ptrs)
    return n, name.value.decode(), list(ints), [p or 0 for p in ptrs]


def _at(*i):
    return [P + 256 * j for j in i]


def test_gated_ffn(lib):
    x, wg, wgs, wu, wus, h, g, u, ws = _at(*range(9))
    assert lib.fp8_gated_ffn(x, 1, 1, wg, wgs, wu, wus, h, g, u, 0, 5, 300, 512, ws, BIG, S) == _lib.OK
    n, name, ints, ptrs = _last(lib)
    assert name == "gated_ffn" and ints[:6] == [1, 1, 0, 5, 300, 512]
    assert ptrs[:10] == [x, wg, wgs, wu, wus, h, g, u, ws, S]
    need = lib.fp8_gated_ffn_workspace(5, 300, 512)
    assert need == 5 * 1000000 + 300 * 1000 + 512
    assert lib.fp8_gated_ffn(x, 0, 0, wg, wgs, wu, wus, h, None, None, 1, 5, 300, 512, ws, need, None) == _lib.OK
    assert _last(lib)[2][:3] == [0, 0, 1] and _last(lib)[3][6:8] == [0, 0]
    assert lib.fp8_gated_ffn(x, 0, 0, wg, wgs, wu, wus, h, None, None, 1, 5, 300, 512, ws, need - 1, None) == _lib.ESCRATCH
    assert lib.fp8_gated_ffn(x, 0, 0, wg, wgs, wu, wus, h, None, None, 1, 0, 300, 512, ws, 0, None) == _lib.OK
    assert _last(lib)[0] == n + 1                          # neither queued anything
    lib._fp8bsq_stub_fail_next()
    assert lib.fp8_gated_ffn(x, 1, 1, wg, wgs, wu, wus, h, g, u, 0, 5, 300, 512, ws, BIG, S) == _lib.ELAUNCH


def test_gated_ffn_backward(lib):
    dh, x, g, u, wg, wgs, wu, wus, dx, dwg, dwu, ws = _at(*range(12))
    call = lambda **k: lib.fp8_gated_ffn_backward(  # noqa: E731
        *[k.get(n, v) for n, v in dict(dh=dh, x=x, g=g, u=u, id=1, wg=wg, wgs=wgs, wu=wu, wus=wus, dx=dx, dwg=dwg, dwu=dwu, od=0, m=7,
                                       f=256, k=384, ws=ws, size=BIG, st=S).items()])
    assert call() == _lib.OK
    n, name, ints, ptrs = _last(lib)
    assert name == "gated_ffn_backward" and ints[:5] == [1, 0, 7, 256, 384]
    assert ptrs[:13] == [dh, x, g, u, wg, wgs, wu, wus, dx, dwg, dwu, ws, S]
    # either product alone does without the other's operands
    assert call(dwg=None, dwu=None, x=None) == _lib.OK and _last(lib)[3][8:11] == [dx, 0, 0]
    assert call(dx=None, wg=None, wgs=None, wu=None, wus=None) == _lib.OK and _last(lib)[3][8:11] == [0, dwg, dwu]
    # no tokens: the zero gradients, from nothing
    assert call(m=0, ws=None, size=0) == _lib.OK
    count, _, ints, ptrs = _last(lib)
    assert ints[:5] == [1, 0, 0, 256, 384] and ptrs[:13] == [0] * 9 + [dwg, dwu, 0, S]
    assert call(m=0, dwg=None, dwu=None) == _lib.OK and call(dx=None, dwg=None, dwu=None) == _lib.OK
    assert _last(lib)[0] == count
    lib._fp8bsq_stub_fail_next()
    assert call() == _lib.ELAUNCH
    lib._fp8bsq_stub_fail_next()
    assert call(m=0) == _lib.ELAUNCH


def test_fp4(lib):
    w, q, s, x, b, y = _at(*range(6))
    assert lib.fp4_weight_quant(w, 0, 9, 96, q, s, S) == _lib.OK
    _, name, ints, ptrs = _last(lib)
    assert name == "fp4_weight_quant" and ints[:3] == [0, 9, 96] and ptrs[:4] == [w, q, s, S]
    assert lib.fp4_gemv(x, 1, q, s, b, y, 0, 3, 9, 96, S) == _lib.OK
    _, name, ints, ptrs = _last(lib)
    assert name == "fp4_gemv" and ints[:5] == [1, 0, 3, 9, 96] and ptrs[:6] == [x, q, s, b, y, S]
    for call in (lambda: lib.fp4_weight_quant(w, 1, 9, 96, q, s, S), lambda: lib.fp4_gemv(x, 1, q, s, None, y, 0, 3, 9, 96, S)):
        lib._fp8bsq_stub_fail_next()
        assert call() == _lib.ELAUNCH and call() == _lib.OK


@pytest.mark.parametrize("count", [0, 1, 300])
def test_clip(lib, count):
    grads, outs = array.array("Q", [P + 4 * i for i in range(count)]), array.array("Q", [2 * P + 4 * i for i in range(count)])
    numels, dtypes = array.array("q", [i % 5 for i in range(count)]), array.array("i", [i % 2 for i in range(count)])
    at = lambda a: a.buffer_info()[0] if count else None  # noqa: E731
    need = lib.fp8bsq_clip_grad_norm_workspace(count)
    for out in (outs, None):
        assert lib.fp8bsq_clip_grad_norm(at(grads), at(out) if out else None, at(numels), at(dtypes), count, 3.0, 2.0, P, 2 * P, need,
                                         S) == _lib.OK
        _, name, ints, ptrs = _last(lib)
        total = sum(grads) + (sum(outs) if out else 0)
        assert name == "clip_grad_norm" and ints[:6] == [count, sum(numels), sum(dtypes), total, 3, 2] and ptrs[:3] == [P, 2 * P, S]
        assert ints[6] == (1 if out and count else 0)
    assert lib.fp8bsq_clip_grad_norm(at(grads), None, at(numels), at(dtypes), count, 3.0, 2.0, P, 2 * P, need - 1, S) == _lib.ESCRATCH
    assert lib.fp8bsq_clip_grad_norm_workspace(-1) == 0
