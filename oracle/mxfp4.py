"""MXFP4 quantiser of the oracle (test infrastructure only; see the package docstring).

MXFP4 is the 4-bit element type of the OCP Microscaling formats: E2M1 values with one shared
power-of-two scale per 32 consecutive values of a row, stored as UE8M0.  Scale rule, as for
this oracle's MXFP8: X = 2^e with e the smallest integer >= -127 such that amax <= 6 * 2^e, so
that nothing saturates.  Element rule: q_i = E2M1(v_i / X), round-to-nearest-even (v_i / X is
exact).  Value: e2m1(q_i) * 2^(S - 127) for scale code S.  A block with a NaN or an infinity
has scale code 255 (NaN) and zero codes.
"""

from __future__ import annotations

import numpy as np

from .mxfp8 import UE8M0_BIAS, ue8m0_decode
from .nvfp4 import e2m1_decode, e2m1_encode, pack_nibbles, unpack_nibbles

MX_BLOCK = 32


def scale_exponent(amax) -> np.ndarray:
    """e = smallest integer >= -127 with amax <= 6 * 2^e, for finite amax >= 0.

    With amax = f * 2^p, f in [0.5, 1), and 6 * 2^e = 0.75 * 2^(e + 3): e = p - 3 when
    f <= 0.75, else p - 2."""
    f, p = np.frexp(np.asarray(amax, np.float64))
    e = np.where(f <= 0.75, p - 3, p - 2).astype(np.int64)
    return np.maximum(np.where(np.asarray(amax) == 0, -UE8M0_BIAS, e), -UE8M0_BIAS)


def quantize_mxfp4(v):
    """v: array [..., K], K a multiple of 32 -> (packed codes [..., K/2], scale codes [..., K/32])."""
    v = np.asarray(v, np.float64)
    blocks = v.reshape(*v.shape[:-1], -1, MX_BLOCK)
    finite = np.isfinite(blocks).all(-1)
    safe = np.where(finite[..., None], blocks, 0.0)
    e = scale_exponent(np.abs(safe).max(-1))
    codes = e2m1_encode(np.ldexp(safe, -e[..., None]).astype(np.float32))
    scales = np.where(finite, e + UE8M0_BIAS, 255).astype(np.uint8)
    return pack_nibbles(codes.reshape(v.shape)), scales


def dequantize_mxfp4(packed, scodes) -> np.ndarray:
    q = e2m1_decode(unpack_nibbles(packed))
    blocks = q.reshape(*q.shape[:-1], -1, MX_BLOCK)
    return (blocks * ue8m0_decode(scodes)[..., None]).reshape(q.shape)
