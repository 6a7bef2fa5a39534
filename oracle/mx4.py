"""Plain NumPy oracle of the MX4 format (MXFP4 of the OCP Microscaling Formats
specification v1.0): block-wise quantization, the values that codes stand for, packing.

TEST INFRASTRUCTURE ONLY. Only the test suite may import this module; the library never
does, and it shares no code or table with the HIP path.

A block of 32 consecutive values of a row has one scale 2^(e - 127) and 4-bit codes: sign,
two exponent bits (bias 1), one mantissa bit. Conversion (the specification's section on
converting to MX): e - 127 = floor(log2 max|v|) - 2 (2 is the exponent of the largest
code, 6), clamped to what the scale byte and a later read in float32 allow, [-127, 125];
then each v / 2^(e - 127) to the nearest code, ties to the even mantissa, larger ones to
6. Readings: a block of zeros takes e = 0, a block with a NaN or an infinity takes e = 255
(NaN) and codes 0.
"""
from __future__ import annotations

import math
from typing import Tuple

import numpy as np

BLOCK = 32


def magnitude(code: int) -> float:
    """The magnitude of a code's low three bits."""
    exp, man = code >> 1 & 3, code & 1
    return man / 2 if exp == 0 else (1 + man / 2) * 2.0 ** (exp - 1)


MAGNITUDES = np.array([magnitude(c) for c in range(8)])


def quantize(x: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """[rows][cols] float64 -> codes int [rows][32 * blocks], scale bytes int [rows][blocks]."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    v = np.zeros((rows, nb * BLOCK))
    v[:, :cols] = x
    v = v.reshape(rows, nb, BLOCK)
    amax = np.max(np.abs(v), axis=2) if v.size else np.zeros((rows, nb))
    bad = ~np.isfinite(amax)
    safe = np.where(bad | (amax == 0), 1.0, amax)
    _, ex = np.frexp(safe)  # amax = f 2^ex, f in [0.5, 1)
    e = np.clip(ex - 1 - 2, -127, 125)
    e = np.where(amax == 0, -127, e)
    with np.errstate(invalid="ignore"):
        a = np.abs(v) * np.exp2(-e.astype(np.float64))[:, :, None]
    # nearest of the eight magnitudes; on a tie the even code
    dist = np.abs(np.where(bad[:, :, None], 0.0, a)[..., None] - MAGNITUDES)
    best = dist.min(axis=-1, keepdims=True)
    cand = dist == best
    even = cand & (np.arange(8) % 2 == 0)
    code = np.where(even.any(axis=-1), even.argmax(axis=-1), cand.argmax(axis=-1))
    code = np.where(np.signbit(v), code + 8, code)
    code = np.where(bad[:, :, None], 0, code)
    return code.reshape(rows, nb * BLOCK), np.where(bad, 255, e + 127)


def values(codes: np.ndarray, scales: np.ndarray, cols: int) -> np.ndarray:
    """float64 [rows][cols] that codes and scale bytes stand for."""
    rows, nb = scales.shape
    mag = MAGNITUDES[codes & 7] * np.where(codes >= 8, -1.0, 1.0)
    s = np.where(scales == 255, math.nan, np.exp2(scales.astype(np.float64) - 127))
    return (mag.reshape(rows, nb, BLOCK) * s[:, :, None]).reshape(rows, nb * BLOCK)[:, :cols]


def pack(codes: np.ndarray) -> np.ndarray:
    """uint8 [rows][16 * blocks]: value 2i in the low half of byte i."""
    return (codes[:, 0::2] | codes[:, 1::2] << 4).astype(np.uint8)


def unpack(packed: np.ndarray) -> np.ndarray:
    p = np.asarray(packed).astype(np.int64)
    return np.stack([p & 15, p >> 4], axis=2).reshape(p.shape[0], -1)


def rounded(x: np.ndarray) -> np.ndarray:
    """x through quantize and values."""
    c, s = quantize(x)
    return values(c, s, np.asarray(x).shape[1])
