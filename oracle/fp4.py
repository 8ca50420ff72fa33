"""4-bit weights (oracle; test infrastructure only).

E2M1: a sign bit, two exponent bits with bias 1, one mantissa bit; exponent 0
holds 0 and 0.5.  One scale 2^(e - 127) per 32 consecutive weights of a row, the
smallest power of two with max |w| <= 6 * scale (max |w| taken as at least
2^-100).  Codes round w / scale to nearest, ties to the even code, the sign kept
on zero.  Two codes to a byte, the even weight in the low half.
"""

import numpy as np

from .ffn import pow2_scale

GROUP = 32


def _decode_one(code):
    e, man = (code >> 1) & 3, code & 1
    v = man * 0.5 if e == 0 else (1 + man * 0.5) * 2.0 ** (e - 1)
    return -v if code & 8 else v


DECODE = np.array([_decode_one(c) for c in range(16)])


def encode(v):
    """float64 -> codes, by the distance to every magnitude."""
    v = np.asarray(v, dtype=np.float64)
    dist = np.abs(np.abs(v)[..., None] - DECODE[:8])
    best = dist.min(-1, keepdims=True)
    near = dist == best                                # one code, or a tie of two neighbours
    even = near & (np.arange(8) % 2 == 0)
    pick = np.where(near.sum(-1) > 1, even.argmax(-1), near.argmax(-1))
    return (pick + 8 * np.signbit(v)).astype(np.uint8)


def weight_quant(w):
    """(q uint8 [n, k/2], s uint8 [n, k/32]) of a float32 [n, k] weight."""
    n, k = w.shape
    b = w.astype(np.float64).reshape(n, k // GROUP, GROUP)
    scale = pow2_scale(np.abs(b).max(-1), 6.0)
    codes = encode(b / scale[..., None]).reshape(n, k // 2, 2)
    return codes[..., 0] | (codes[..., 1] << 4), (np.log2(scale) + 127).astype(np.uint8)


def dequant(q, s):
    n = q.shape[0]
    w = np.stack([DECODE[q & 15], DECODE[q >> 4]], -1).reshape(n, -1, GROUP)
    return (w * np.ldexp(1.0, s.astype(np.int64) - 127)[..., None]).reshape(n, -1)
