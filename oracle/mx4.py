"""Plain definitions of microscaled 4-bit floating point (MX4), in numpy.

TEST INFRASTRUCTURE ONLY, like the rest of this package. Written from the
format: a block of 32 values, codes of a sign, two exponent bits and one mantissa
bit, a scale that is a power of two. Everything is float64, in which float32
inputs, scales and codes are exact.
"""

from __future__ import annotations

import math
from typing import Tuple

import numpy as np

BLOCK = 32
VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantise(x: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """Codes uint8 [M][K] (one each, not packed) and scale bytes [M][K/32] of
    float32 rows: one block at a time, each value against the format's eight."""
    M, K = x.shape
    codes = np.zeros((M, K), np.uint8)
    scales = np.zeros((M, K // BLOCK), np.uint8)
    for m in range(M):
        for b in range(K // BLOCK):
            v = x[m, b * BLOCK:(b + 1) * BLOCK].astype(np.float64)
            if not np.isfinite(v).all():
                scales[m, b] = 255
                continue
            top = np.abs(v).max()
            power = -127 if top == 0 else max(-127, math.frexp(top)[1] - 1 - 2)
            scales[m, b] = power + 127
            for i, t in enumerate(v):
                r = abs(math.ldexp(t, -power))
                off = np.abs(VALUES - r)
                near = np.flatnonzero(off == off.min())
                c = int(near[0]) if len(near) == 1 else int(near[near % 2 == 0][0])
                codes[m, b * BLOCK + i] = c + (8 if math.copysign(1.0, t) < 0 else 0)
    return codes, scales


def pack(codes: np.ndarray) -> np.ndarray:
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(packed: np.ndarray) -> np.ndarray:
    out = np.empty((packed.shape[0], 2 * packed.shape[1]), np.uint8)
    out[:, 0::2], out[:, 1::2] = packed & 15, packed >> 4
    return out


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 values of unpacked codes and scale bytes (255: NaN)."""
    v = VALUES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.ldexp(1.0, scales.astype(np.int32) - 127)
    s[scales == 255] = np.nan
    return v * np.repeat(s, BLOCK, axis=1)


def act(name: str, g: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """An activation and its derivative."""
    from scipy.special import ndtr
    g = g.astype(np.float64)
    if name == "silu":
        s = np.where(g < 0, np.exp(np.minimum(g, 0)), 1.0) / (1.0 + np.exp(-np.abs(g)))
        return g * s, s + g * s * (1 - s)
    if name == "gelu":
        c = ndtr(g)
        return g * c, c + g * np.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    z = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    # (1 + tanh z) / 2 without the cancellation at z << 0
    s = np.where(z < 0, np.exp(2 * np.minimum(z, 0)), 1.0) / (1.0 + np.exp(-2 * np.abs(z)))
    dz = math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g)
    return g * s, s + 2 * g * s * (1 - s) * dz
