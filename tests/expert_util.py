"""Inputs shared by the tests of the expert operators."""

import numpy as np
import torch

from tests import ffn_util as U

TYPES = U.TYPES
STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}   # half a step, relative to the value
LEAST = {"bf16": 2.0 ** -134, "f32": 2.0 ** -150}   # half a step below the normal values


def choices(seed, tokens, top_k, experts, drop=0.0, skew=0.7):
    """[tokens, top_k] int64: a router's choices, different ones for a token where
    there are enough experts; a share `drop` of them is -1 or past the last expert."""
    rng = np.random.default_rng(seed)
    score = rng.standard_normal((tokens, experts)) + skew * rng.standard_normal(experts)
    if top_k <= experts:
        ids = np.argsort(-score, axis=1)[:, :top_k]
    else:
        ids = rng.integers(0, experts, (tokens, top_k))
    out = rng.random(ids.shape) < drop
    return np.where(out, np.where(rng.random(ids.shape) < 0.5, -1, experts), ids).astype(np.int64)


def sort(ids, experts):
    """The stable sort by numpy's: (offsets, rows, choices)."""
    flat = ids.reshape(-1)
    key = np.where((flat >= 0) & (flat < experts), flat, experts)
    order = np.argsort(key, kind="stable")
    offsets = np.searchsorted(key[order], np.arange(experts + 1))
    rows = np.empty(flat.size, np.int64)
    rows[order] = np.arange(flat.size)
    rows = np.where(key < experts, rows, ~rows)
    return offsets.astype(np.int32), rows.reshape(ids.shape).astype(np.int32), order.astype(np.int32)


def normal(seed, shape, kind, scale=1.0):
    """A CPU tensor of N(0, scale^2)."""
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape) * scale).to(TYPES[kind])


def weights(seed, experts, n, k):
    """Codes [E, N, K] and scales of all experts, numpy."""
    pairs = [U.weight(1000 * seed + e, n, k) for e in range(experts)]
    return np.stack([c for c, _ in pairs]), np.stack([s for _, s in pairs])


def within(got, want, bound):
    """Whether got (a tensor) is within bound of want everywhere."""
    got = U.values(got)
    assert got.shape == want.shape
    off = np.abs(got - want)
    assert np.all(off <= bound), f"{int((~(off <= bound)).sum())} of {off.size} off, the worst {np.nanmax(off - bound)} over its bound"
