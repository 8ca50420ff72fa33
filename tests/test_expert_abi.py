"""C-ABI checks of the expert operators that need no GPU: bad arguments come back
with the documented status before HIP is touched (the pointers passed are never
dereferenced), and the Python functions refuse what they do not take."""

import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from fp8_block_scaled_quant_amd import _ffn_lib, _lib

P = 4096   # never dereferenced
BIG = 1 << 62


@pytest.fixture(scope="module")
def lib():
    return _ffn_lib.load_library()


def _call(fn, ok):
    """fn with some of the arguments changed: call(a3=0)."""
    def call(**changed):
        args = list(ok)
        for name, v in changed.items():
            args[int(name[1:])] = v
        return fn(*args)
    return call


def test_sort_validation(lib):
    #                                    ids ib n     E   off rows cho ws size stream
    call = _call(lib.fp8bsq_expert_sort, (P, 8, 9000, 64, P, P, P, P, BIG, None))
    for bad in (dict(a0=None), dict(a4=None), dict(a5=None), dict(a6=None), dict(a7=None), dict(a1=2), dict(a1=0), dict(a2=-1), dict(a3=0), dict(a3=-4)):
        assert call(**bad) == _lib.EINVAL, bad
    for bad in (dict(a0=P + 4), dict(a1=4, a0=P + 2), dict(a4=P + 2), dict(a5=P + 1), dict(a6=P + 2), dict(a7=P + 64)):
        assert call(**bad) == _lib.EALIGN, bad
    for bad in (dict(a3=1025), dict(a2=1 << 31), dict(a2=1 << 60)):
        assert call(**bad) == _lib.ERANGE, bad
    need = lib.fp8bsq_expert_sort_workspace(9000, 64)
    assert need > 0 and call(a8=need - 1) == _lib.ESCRATCH
    assert lib.fp8bsq_expert_sort_workspace(8, 64) == 0 and lib.fp8bsq_expert_sort_workspace(0, 64) == 0
    for sizes in ((-1, 64), (8, 0), (8, 1025), (1 << 31, 64)):
        assert lib.fp8bsq_expert_sort_workspace(*sizes) == 0


def test_dispatch_validation(lib):
    #                                        x  dt rows T  k  h   y  stream
    call = _call(lib.fp8bsq_expert_dispatch, (P, 1, P, 4, 2, 70, P, None))
    for bad in (dict(a0=None), dict(a2=None), dict(a6=None), dict(a1=2), dict(a3=-1), dict(a4=0), dict(a4=-1), dict(a5=-1)):
        assert call(**bad) == _lib.EINVAL, bad
    for bad in (dict(a0=P + 1), dict(a6=P + 1), dict(a2=P + 2), dict(a1=0, a0=P + 2)):
        assert call(**bad) == _lib.EALIGN, bad
    for bad in (dict(a3=1 << 30), dict(a3=1 << 40, a4=1 << 40), dict(a4=1 << 62), dict(a5=(1 << 21) + 1)):
        assert call(**bad) == _lib.ERANGE, bad
    assert call(a3=0, a0=None, a2=None, a6=None) == _lib.OK and call(a5=0, a0=None, a2=None, a6=None) == _lib.OK


def test_dispatch_quant_validation(lib):
    #                                           x  dt fmt rows T  k  h   y  s  stream
    call = _call(lib.fp8_expert_dispatch_quant, (P, 1, 0, P, 4, 2, 256, P, P, None))
    for bad in (dict(a0=None), dict(a3=None), dict(a7=None), dict(a8=None), dict(a1=-1), dict(a2=2), dict(a4=-1), dict(a5=0), dict(a6=-128)):
        assert call(**bad) == _lib.EINVAL, bad
    assert call(a6=200) == _lib.ESHAPE
    for bad in (dict(a0=P + 8), dict(a7=P + 8), dict(a8=P + 2), dict(a3=P + 2)):
        assert call(**bad) == _lib.EALIGN, bad
    for bad in (dict(a4=1 << 30), dict(a6=(1 << 21) + 128)):
        assert call(**bad) == _lib.ERANGE, bad
    assert call(a4=0, a0=None, a3=None, a7=None, a8=None) == _lib.OK and call(a6=0, a0=None) == _lib.OK


def test_combine_validation(lib):
    #                                       y  dt rows w  wd T  k  h   out stream
    call = _call(lib.fp8bsq_expert_combine, (P, 1, P, P, 0, 4, 2, 70, P, None))
    for bad in (dict(a0=None), dict(a2=None), dict(a8=None), dict(a1=2), dict(a4=2), dict(a5=-1), dict(a6=0), dict(a7=-1)):
        assert call(**bad) == _lib.EINVAL, bad
    for bad in (dict(a0=P + 1), dict(a8=P + 1), dict(a2=P + 2), dict(a3=P + 2), dict(a3=P + 1, a4=1)):
        assert call(**bad) == _lib.EALIGN, bad
    for bad in (dict(a5=1 << 30), dict(a6=1 << 62), dict(a7=(1 << 21) + 1)):
        assert call(**bad) == _lib.ERANGE, bad
    assert call(a5=0, a0=None, a2=None, a8=None) == _lib.OK and call(a7=0, a0=None, a8=None) == _lib.OK


def test_combine_backward_validation(lib):
    #                                                d  y  dt rows w  wd T  k  h   dy dw stream
    call = _call(lib.fp8bsq_expert_combine_backward, (P, P, 1, P, P, 0, 4, 2, 70, P, P, None))
    for bad in (dict(a0=None), dict(a1=None), dict(a3=None), dict(a2=2), dict(a5=2), dict(a6=-1), dict(a7=0), dict(a8=-1)):
        assert call(**bad) == _lib.EINVAL, bad
    for bad in (dict(a0=P + 1), dict(a1=P + 1), dict(a3=P + 2), dict(a4=P + 2), dict(a9=P + 1), dict(a10=P + 2)):
        assert call(**bad) == _lib.EALIGN, bad
    for bad in (dict(a6=1 << 30), dict(a8=(1 << 21) + 1)):
        assert call(**bad) == _lib.ERANGE, bad
    assert call(a9=None, a10=None) == _lib.OK and call(a6=0, a0=None, a3=None) == _lib.OK   # nothing asked for; no tokens
    assert call(a8=0, a10=None, a0=None, a1=None, a3=None) == _lib.OK                        # rows of no length


@pytest.mark.parametrize("gated", [False, True])
def test_product_validation(lib, gated):
    weights = (P, P, P, P) if gated else (P, P)
    c = 3 + len(weights)
    #                    a  as off weights  out dt R  E  f   k    stream
    call = _call(lib.fp8_expert_gated_ffn if gated else lib.fp8_expert_gemm, (P, P, P, *weights, P, 1, 9, 3, 70, 256, None))
    for i in range(c + 1):
        assert call(**{f"a{i}": None}) == _lib.EINVAL, i
    for bad in ({f"a{c + 1}": 2}, {f"a{c + 2}": -1}, {f"a{c + 3}": 0}, {f"a{c + 3}": -1}, {f"a{c + 4}": -1}, {f"a{c + 5}": 0}, {f"a{c + 5}": -128}):
        assert call(**bad) == _lib.EINVAL, bad
    assert call(**{f"a{c + 5}": 200}) == _lib.ESHAPE
    for bad in (dict(a0=P + 8), dict(a1=P + 2), dict(a2=P + 2), dict(a3=P + 8), dict(a4=P + 2), {f"a{c}": P + 1}):
        assert call(**bad) == _lib.EALIGN, bad
    for bad in ({f"a{c + 2}": 65535 * 16 + 1}, {f"a{c + 3}": 1025}, {f"a{c + 4}": (1 << 21) + 1}, {f"a{c + 5}": (1 << 21) + 128}):
        assert call(**bad) == _lib.ERANGE, bad
    assert call(**{f"a{c + 2}": 0, "a0": None}) == _lib.OK and call(**{f"a{c + 4}": 0, "a3": None}) == _lib.OK


def test_python_functions_refuse_cpu_tensors_and_wrong_arguments():
    """No fallback: everything below raises before the library is called."""
    rows, x, y = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 128), torch.zeros(8, 128)
    a, a_s, offsets = torch.zeros(8, 128, dtype=torch.uint8), torch.ones(8, 1), torch.zeros(4, dtype=torch.int32)
    w, w_s = torch.zeros(3, 128, 128, dtype=torch.uint8), torch.ones(3, 1, 1)
    for call in (lambda: fb.expert_sort(rows, 4), lambda: fb.expert_dispatch(x, rows), lambda: fb.expert_dispatch_quant(x, rows),
                 lambda: fb.expert_combine(y, rows), lambda: fb.expert_combine_backward(x, y, rows), lambda: fb.expert_gemm(a, a_s, offsets, w, w_s),
                 lambda: fb.expert_gated_ffn(a, a_s, offsets, w, w_s, w, w_s), lambda: fb.expert_dispatch_quant(x, rows, "e8"),
                 lambda: fb.Experts(0, 128, 128), lambda: fb.Experts(1025, 128, 128), lambda: fb.Experts(4, 100, 128), lambda: fb.Experts(4, 128, 100),
                 lambda: fb.Experts(4, 128, 128, torch.half), lambda: fb.Experts(4, 128, 128, scale_fmt="e8")):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: fb.expert_gemm(a.float(), a_s, offsets, w, w_s), lambda: fb.expert_gemm(a, a_s, offsets, w, w_s, torch.half)):
        with pytest.raises(TypeError):
            call()
    layer = fb.Experts(3, 128, 256)
    assert [tuple(p.shape) for p in layer.parameters()] == [(3, 256, 128), (3, 2, 1)] * 2 + [(3, 128, 256), (3, 1, 2)]
    assert not any(p.requires_grad for p in layer.parameters())
    with pytest.raises(ValueError):
        layer(torch.zeros(4, 256), rows, torch.ones(4, 2))
    with pytest.raises(ValueError):
        fb.Experts.from_weights(torch.zeros(3, 256, 128), torch.zeros(3, 128, 128), torch.zeros(3, 128, 256))
