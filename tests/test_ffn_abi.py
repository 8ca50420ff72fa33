"""C-ABI checks of the feed-forward library that need no GPU: it exports exactly
the symbols include/fp8bsq_ffn.h declares and rejects bad arguments with the
documented status codes before touching HIP (the pointers passed are never
dereferenced), and the Python functions refuse what they do not take."""

import array
import os
import re
import subprocess

import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from fp8_block_scaled_quant_amd import _ffn_lib, _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 4096   # never dereferenced
BIG = 1 << 62


@pytest.fixture(scope="module")
def lib():
    return _ffn_lib.load_library()


def test_exports_match_the_header(lib):
    text = open(os.path.join(ROOT, "include", "fp8bsq_ffn.h")).read()
    declared = set(re.findall(r"^FP8BSQ_API\s+[\w\s\*]*?\b(\w+)\s*\(", text, flags=re.M))
    assert declared == set(_ffn_lib.EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", _ffn_lib.LIB_PATH], capture_output=True, text=True)
    exported = {line.split()[-1] for line in out.stdout.splitlines() if " T " in line}
    assert {s for s in exported if not s.startswith("_")} == declared


def _with(args, **changed):
    args = list(args)
    for i, v in changed.items():
        args[int(i[1:])] = v
    return args


def test_gated_ffn_validation(lib):
    #      x  xd fmt wg ws wu us h  g     u     od m  f    k    ws bytes stream
    ok = (P, 1, 0, P, P, P, P, P, None, None, 1, 4, 256, 512, P, BIG, None)
    call = lambda **kw: lib.fp8_gated_ffn(*_with(ok, **kw))  # noqa: E731
    for bad in (dict(a0=None), dict(a3=None), dict(a6=None), dict(a7=None), dict(a14=None), dict(a8=P), dict(a9=P),
                dict(a1=2), dict(a2=2), dict(a10=-1), dict(a11=-1), dict(a12=-1), dict(a13=0), dict(a13=-128)):
        assert call(**bad) == _lib.EINVAL, bad
    assert call(a13=200) == _lib.ESHAPE
    for bad in (dict(a0=P + 8), dict(a3=P + 4), dict(a4=P + 2), dict(a7=P + 1), dict(a8=P + 1, a9=P), dict(a14=P + 16)):
        assert call(**bad) == _lib.EALIGN, bad
    assert call(a11=1 << 40) == _lib.ERANGE and call(a12=1 << 31) == _lib.ERANGE
    assert call(a15=lib.fp8_gated_ffn_workspace(4, 256, 512) - 1) == _lib.ESCRATCH
    # empty outputs: before any pointer is looked at
    assert lib.fp8_gated_ffn(*([None, 1, 0] + [None] * 7 + [1, 0, 256, 512, None, 0, None])) == _lib.OK
    assert lib.fp8_gated_ffn(*([None, 1, 0] + [None] * 7 + [1, 4, 0, 512, None, 0, None])) == _lib.OK
    for sizes in ((0, 256, 512), (4, 256, 500), (-1, 256, 512)):
        assert lib.fp8_gated_ffn_workspace(*sizes) == 0


def test_gated_ffn_backward_validation(lib):
    #     dh x  g  u  id wg ws wu us dx dg du od m  f    k    ws bytes stream
    ok = (P, P, P, P, 1, P, P, P, P, P, P, P, 1, 4, 256, 512, P, BIG, None)
    call = lambda **kw: lib.fp8_gated_ffn_backward(*_with(ok, **kw))  # noqa: E731
    for bad in (dict(a0=None), dict(a1=None), dict(a2=None), dict(a5=None), dict(a8=None), dict(a10=None), dict(a11=None),
                dict(a16=None), dict(a4=3), dict(a12=3), dict(a13=-1), dict(a14=0), dict(a15=0)):
        assert call(**bad) == _lib.EINVAL, bad
    assert call(a14=200) == _lib.ESHAPE and call(a15=200) == _lib.ESHAPE
    for bad in (dict(a0=P + 8), dict(a1=P + 8), dict(a3=P + 2), dict(a5=P + 8), dict(a6=P + 2), dict(a9=P + 2), dict(a16=P + 64)):
        assert call(**bad) == _lib.EALIGN, bad
    assert call(a13=1 << 40) == _lib.ERANGE and call(a14=1 << 30) == _lib.ERANGE
    assert call(a17=lib.fp8_gated_ffn_backward_workspace(4, 256, 512) - 1) == _lib.ESCRATCH
    assert call(a9=None, a10=None, a11=None) == _lib.OK            # nothing asked for
    assert call(a13=0, a10=None, a11=None, a9=None) == _lib.OK
    assert lib.fp8_gated_ffn_backward_workspace(4, 200, 512) == 0


def test_fp4_validation(lib):
    quant = lambda **kw: lib.fp4_weight_quant(*_with((P, 1, 8, 64, P, P, None), **kw))  # noqa: E731
    for bad in (dict(a0=None), dict(a4=None), dict(a5=None), dict(a1=2), dict(a2=-1), dict(a3=-32)):
        assert quant(**bad) == _lib.EINVAL, bad
    assert quant(a3=48) == _lib.ESHAPE
    assert quant(a0=P + 8) == _lib.EALIGN and quant(a4=P + 2) == _lib.EALIGN
    assert quant(a2=1 << 31) == _lib.ERANGE
    assert lib.fp4_weight_quant(None, 1, 0, 64, None, None, None) == _lib.OK
    #       x  xd q  s  bias y  yd m  n  k   stream
    gemv = lambda **kw: lib.fp4_gemv(*_with((P, 1, P, P, None, P, 1, 2, 8, 64, None), **kw))  # noqa: E731
    for bad in (dict(a0=None), dict(a2=None), dict(a3=None), dict(a5=None), dict(a1=2), dict(a6=2), dict(a7=-1), dict(a9=0)):
        assert gemv(**bad) == _lib.EINVAL, bad
    assert gemv(a9=80) == _lib.ESHAPE
    for bad in (dict(a0=P + 8), dict(a2=P + 8), dict(a4=P + 1), dict(a5=P + 1)):
        assert gemv(**bad) == _lib.EALIGN, bad
    assert gemv(a7=1 << 40) == _lib.ERANGE and gemv(a8=1 << 31) == _lib.ERANGE
    assert lib.fp4_gemv(None, 1, None, None, None, None, 1, 0, 8, 64, None) == _lib.OK


def test_clip_validation(lib):
    ptrs, numels, dtypes = array.array("Q", [P, P]), array.array("q", [5, 6]), array.array("i", [0, 1])
    at = lambda a: a.buffer_info()[0]  # noqa: E731

    def call(p=ptrs, o=ptrs, n=numels, d=dtypes, count=2, max_norm=1.0, eps=0.0, norm=P, ws=P, size=BIG):
        return lib.fp8bsq_clip_grad_norm(at(p) if p else None, at(o) if o else None, at(n), at(d), count, max_norm, eps,
                                         norm, ws, size, None)
    assert call(p=None) == _lib.EINVAL
    assert call(count=-1) == _lib.EINVAL
    assert call(max_norm=-1.0) == _lib.EINVAL and call(max_norm=float("nan")) == _lib.EINVAL
    assert call(eps=-1.0) == _lib.EINVAL
    assert call(norm=None) == _lib.EINVAL and call(ws=None) == _lib.EINVAL
    assert call(n=array.array("q", [5, -1])) == _lib.EINVAL
    assert call(d=array.array("i", [0, 2])) == _lib.EINVAL
    assert call(p=array.array("Q", [P, 0])) == _lib.EINVAL and call(o=array.array("Q", [0, P])) == _lib.EINVAL
    assert call(p=array.array("Q", [P + 2, P])) == _lib.EALIGN and call(o=array.array("Q", [P, P + 1])) == _lib.EALIGN
    assert call(norm=P + 2) == _lib.EALIGN and call(ws=P + 8) == _lib.EALIGN
    assert call(n=array.array("q", [5, 1 << 50])) == _lib.ERANGE
    assert call(size=8) == _lib.ESCRATCH


def test_python_functions_refuse_cpu_tensors_and_wrong_arguments():
    """No fallback: everything below raises before the library is called."""
    bf = torch.bfloat16
    x, w, s = torch.zeros(2, 128, dtype=bf), torch.zeros(128, 128, dtype=torch.uint8), torch.ones(1, 1)
    with pytest.raises(ValueError):
        fb.gated_ffn(x, w, s, w, s)
    with pytest.raises(ValueError):
        fb.gated_ffn_backward(x, x, x, x, w, s, w, s)
    with pytest.raises(ValueError):
        fb.fp4_weight_quant(torch.zeros(4, 64))
    with pytest.raises(ValueError):
        fb.fp4_gemv(torch.zeros(1, 64), torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(ValueError):
        fb.clip_grad_norm([torch.zeros(3)], 1.0)
    with pytest.raises(ValueError):
        fb.clip_grad_norm([], 1.0)
    with pytest.raises(ValueError):
        fb.clip_grad_norm([torch.zeros(3)], -1.0)
    with pytest.raises(TypeError):
        fb.gated_ffn(x, w.float(), s, w, s)
    with pytest.raises(ValueError):
        fb.GatedFFN(100, 128)
    with pytest.raises(ValueError):
        fb.GatedFFN(128, 100)
    assert [tuple(p.shape) for p in fb.GatedFFN(128, 256).parameters()] == [(256, 128)] * 2
