"""The backward pass of the gated feed-forward block on every combination of the
ways its two products are launched, together and alone, sampled outputs against
the float64 oracle.

Bounds per element: 1e-3 sum |a b| for an E4M3 product (the block GEMM's bound),
half an ulp of the output type, and two E4M3 roundings among the element's terms
that the FP32 and the float64 value of a gradient take to different sides, each
an eighth of its term at most (a few in 10^6 values lie that near to a boundary).
"""

import numpy as np
import pytest
import torch

import fp8_block_scaled_quant_amd as fb
from oracle import ffn
from tests import ffn_util as U
from tests import gpu_util as G
from tests.test_gpu_gated_ffn_backward import _inputs, _run

pytestmark = pytest.mark.gpu

# (m, f, k): how dx goes, and dW: 256 x 256 tiles ("big"), 128 x 128 ("mid"), or
# those with the contraction in parts ("split"); on 256 compute units
TOGETHER = {(129, 256, 640): ("mid", "mid"), (1199, 1280, 1664): ("mid", "big"), (1504, 128, 128): ("mid", "split"),
            (3000, 256, 256): ("mid", "split"), (65, 1024, 896): ("split", "mid"), (3, 5120, 3968): ("split", "big"),
            (1533, 1280, 128): ("split", "split"), (690, 128, 6016): ("big", "mid"), (1686, 128, 2688): ("big", "split"),
            (1037, 384, 6912): ("big", "big")}
# a dW of few tokens that joins dx's launch, in 128 x 128 tiles, where alone it takes 256 x 256
JOINED = {(1, 640, 4736): ("mid", "mid"), (70, 1792, 3456): ("split", "mid")}
LARGE = (131077, 32768, 256)   # m f = 4.3e9, both products in 256 x 256 tiles


def _near(got, a, b, out):
    """got against a @ b, element by element and in the 2-norm."""
    want, terms = a @ b, np.abs(a) @ np.abs(b)
    top = np.stack([(np.abs(row)[:, None] * np.abs(b)).max(0) for row in a])
    tol = 1e-3 * terms + top / 4 + np.abs(want) * (2.0 ** -8 if out == "bf16" else 2.0 ** -23)
    assert np.all(np.abs(got - want) <= tol)
    assert U.rel_error(got, want) <= U.REL[out] + 3 / 8 / np.sqrt(a.size)


def _check(acts, wg, wu, got, out):
    dh, x, g, u = (t.float().double().numpy() for t in acts)
    (m, f), k = dh.shape, x.shape[1]
    rng = np.random.default_rng(0)
    pick = lambda n, count: np.unique(np.r_[0, n - 1, rng.integers(n, size=count)])  # noqa: E731
    dx, *dw = got
    cols = pick(k, 400)
    if dx is not None:
        assert dx.dtype == U.TYPES[out]
        rows = pick(m, 24)
        d = np.concatenate([ffn.quantize_rows(v) for v in ffn.activation_grads(dh[rows], g[rows], u[rows])], 1)
        _near(U.values(dx)[np.ix_(rows, cols)], d, np.concatenate([ffn.weight(*wg), ffn.weight(*wu)])[:, cols], out)
    feats = pick(f, 24)
    xq = ffn.quantize_tokens(x[:, cols])
    for have, v in zip(dw, ffn.activation_grads(dh[:, feats], g[:, feats], u[:, feats])):
        if have is not None:
            assert have.dtype == U.TYPES[out]
            _near(U.values(have)[np.ix_(feats, cols)], ffn.quantize_tokens(v).T, xq, out)


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("m,f,k", [*TOGETHER, *JOINED])
def test_every_launch(m, f, k, dtype, out):
    """Both products at once, and each alone: dx with frozen weights, dW of a first layer."""
    G.announce(f"gated_ffn_backward m={m} f={f} k={k} {dtype} -> {out}")
    acts, wg, wu = _inputs(m, f, k, dtype)
    both = _run(acts, wg, wu, out_dtype=U.TYPES[out])
    _check(acts, wg, wu, both, out)
    assert all(torch.equal(p, q) for p, q in zip(both, _run(acts, wg, wu, out_dtype=U.TYPES[out])))
    G.announce("dx alone")
    dx, *none = _run(acts, wg, wu, out_dtype=U.TYPES[out], weight_grad=False)
    assert none == [None, None] and torch.equal(dx, both[0])
    G.announce("dW alone")
    none, *dw = _run(acts, wg, wu, out_dtype=U.TYPES[out], input_grad=False)
    assert none is None
    _check(acts, wg, wu, (None, *dw), out)


def test_large_tiles_past_32_bits():
    m, f, k = LARGE
    G.announce(f"gated_ffn_backward {m} x {f} x {k}")
    gen = torch.Generator(G.device()).manual_seed(1)
    normal = lambda *shape: torch.randn(*shape, generator=gen, device=G.device(), dtype=torch.bfloat16)  # noqa: E731
    dh, g, u, x = normal(m, f), normal(m, f), normal(m, f), normal(m, k)
    wg, wu = U.weight(3, f, k), U.weight(4, f, k)
    dx, *dw = fb.gated_ffn_backward(dh, x, g, u, *[U.gpu(v) for v in (*wg, *wu)])
    rows = np.unique([0, 1, 2 ** 31 // f, 2 ** 31 // f + 1, 2 ** 32 // f, 2 ** 32 // f + 1, m - 2, m - 1])
    d = np.concatenate([ffn.quantize_rows(v) for v in ffn.activation_grads(*[U.values(t[rows]) for t in (dh, g, u)])], 1)
    _near(U.values(dx[rows]), d, np.concatenate([ffn.weight(*wg), ffn.weight(*wu)]), "bf16")
    feats = np.array([0, 127, 128, 16400, f - 1])
    xq = ffn.quantize_tokens(U.values(x))
    for have, v in zip(dw, ffn.activation_grads(*[U.values(t[:, feats]) for t in (dh, g, u)])):
        _near(U.values(have[feats]), ffn.quantize_tokens(v).T, xq, "bf16")
    torch.cuda.empty_cache()
