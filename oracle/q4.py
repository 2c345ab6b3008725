"""The 4-bit block format and its products in float64.

Values are E2M1 codes with one power-of-two scale 2^e per block of 32 elements
along the direction that a product sums over.  e is the smallest integer with
max|block| <= 6 * 2^e, clamped to [-125, 126]; scale bytes hold e + 127.  A block
with a NaN or an infinity has the scale byte 255 and zero codes, and stands for
NaN.
"""

from __future__ import annotations

import numpy as np

BLOCK, PAD, SCALE_ROW = 32, 256, 16
MIN_EXP, MAX_EXP = -125, 126
NAN_BYTE = 255
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def up(n: int, a: int) -> int:
    return -(-n // a) * a


def exponent(amax: np.ndarray) -> np.ndarray:
    """The smallest e in range with amax <= 6 * 2^e."""
    amax = np.asarray(amax, np.float64)
    _, p = np.frexp(amax)
    e = p - 4  # 6 * 2^(p - 4) < 2^(p - 1) <= amax
    for _ in range(3):
        e = np.where(amax > np.ldexp(6.0, e), e + 1, e)
    return np.clip(np.where(amax > 0, e, MIN_EXP), MIN_EXP, MAX_EXP)


def round_e2m1(v: np.ndarray, random=None) -> np.ndarray:
    """Codes (bit 3 the sign) of |v| <= 6: to nearest, ties to the even code, or
    up iff 256 times the part of the step that is left is at least 255.5 - random."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    low = np.clip(np.searchsorted(MAGNITUDES, a, side="right") - 1, 0, 6)
    part = (a - MAGNITUDES[low]) / (MAGNITUDES[low + 1] - MAGNITUDES[low])
    if random is None:
        up_ = (part > 0.5) | ((part == 0.5) & (low % 2 == 1))
    else:
        up_ = 256.0 * part >= 255.5 - np.asarray(random, np.float64)
    return ((low + up_) | np.where(np.signbit(v), 8, 0)).astype(np.uint8)


def code_values(codes: np.ndarray) -> np.ndarray:
    return MAGNITUDES[codes & 7] * np.where(codes & 8, -1.0, 1.0)


def quantize(x: np.ndarray, random=None):
    """(codes, one a byte [R, Cp], scale bytes [Cp / 32, R16]) of x [R, C]."""
    r, c = x.shape
    cp = up(c, PAD)
    v = np.zeros((r, cp))
    v[:, :c] = x
    v = v.reshape(r, cp // BLOCK, BLOCK)
    bad = ~np.isfinite(v).all(axis=2)
    v = np.where(bad[:, :, None], 0.0, v)
    e = exponent(np.abs(v).max(axis=2)) if r else np.zeros((0, cp // BLOCK), int)
    if random is not None:
        n = np.zeros((r, cp))
        n[:, :c] = random
        random = n.reshape(v.shape)
    codes = round_e2m1(v * np.ldexp(1.0, -e)[:, :, None], random).reshape(r, cp)
    scales = np.full((cp // BLOCK, up(r, SCALE_ROW)), MIN_EXP + 127, np.uint8)
    scales[:, :r] = np.where(bad, NAN_BYTE, e + 127).T
    return codes, scales


def pack(codes: np.ndarray) -> np.ndarray:
    """Two codes to a byte, the first in the low four bits."""
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """The values [R, Cp] that codes and scale bytes stand for."""
    r, cp = codes.shape
    byte = scales[:, :r].T
    s = np.where(byte == NAN_BYTE, np.nan, np.ldexp(1.0, byte.astype(int) - 127))
    return (code_values(codes).reshape(r, cp // BLOCK, BLOCK) * s[:, :, None]).reshape(r, cp)


def quantized(x: np.ndarray, random=None) -> np.ndarray:
    """The values that x's codes stand for, [R, C]."""
    return values(*quantize(x, random))[:, :x.shape[1]]


def matmul(a: np.ndarray, b: np.ndarray, base=None):
    """(base + a b^T, |base| + |a| |b|^T) of operand values; the second bounds rounding."""
    g, m = a @ b.T, np.abs(a) @ np.abs(b).T
    return (g, m) if base is None else (base + g, np.abs(base) + m)
