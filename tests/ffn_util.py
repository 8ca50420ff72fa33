"""Inputs and bounds shared by the feed-forward GPU tests."""

import numpy as np
import torch

import oracle
from inputs import gen
from tests import gpu_util as G

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# Relative error in the 2-norm.  Rounding to bf16 (8 significant bits) moves an
# element by at most 2^-8 of it; the E4M3 matrix product is within 1e-3 sum |a b|
# per element (the block GEMM's bound: the instruction drops low bits of
# products it aligns to the largest one).
REL = {"bf16": 2.0 ** -8 + 1e-3, "f32": 1e-3}


def weight(seed, n, k):
    """Codes and scales of spread 0.02, as tensors and numpy."""
    rng = np.random.default_rng(seed)
    w = rng.standard_normal((n, k)) * 100
    codes = oracle.e4m3.encode(np.clip(w, -448, 448))
    scales = gen.log_uniform_scales(rng, gen.scale_grid(n, k), -1, 1) * np.float32(2e-4)
    return codes, scales


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(G.device())


def values(t):
    return t.float().double().cpu().numpy()


def rel_error(got, want):
    norm = np.linalg.norm(want)
    return np.linalg.norm(got - want) / norm if norm else np.linalg.norm(got)


def guarded_like(shape, dtype):
    """A GPU tensor of that shape inside canary bytes, and the check of those."""
    size = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
    buf = G.Guarded(size)
    return buf.payload().view(dtype).view(shape), buf
