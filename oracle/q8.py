"""The 8-bit block format and its products in float64.

Values are E4M3 codes with one power-of-two scale 2^e per block of 128
elements (rows: 1 x 128; weights: 128 x 128).  e is the smallest integer with
max|block| <= 448 * 2^e over the block's finite elements, clamped to
[-117, 120]; scale bytes hold e + 127.
"""

from __future__ import annotations

import numpy as np

BLOCK = 128
MIN_EXP, MAX_EXP = -117, 120


def up(n: int, a: int) -> int:
    return -(-n // a) * a


def exponent(amax: float) -> int:
    """The smallest e in range with amax <= 448 * 2^e."""
    e = MIN_EXP
    while e < MAX_EXP and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def round_e4m3(v: np.ndarray) -> np.ndarray:
    """Nearest E4M3 value, ties to even; |v| <= 448.  NaN and infinities give NaN."""
    v = np.asarray(v, np.float64)
    finite = np.isfinite(v)
    a = np.where(finite, v, 0.0)
    _, p = np.frexp(np.maximum(np.abs(a), 2.0 ** -6))
    step = np.ldexp(1.0, p - 4)
    return np.where(finite, np.rint(a / step) * step, np.nan)


def _finite_max(x: np.ndarray) -> float:
    x = np.abs(x[np.isfinite(x)])
    return float(x.max()) if x.size else 0.0


def quantize_rows(x: np.ndarray):
    """(code values [T, Kp], scale bytes [Kp / 128, T4]) of x [T, K]."""
    t, k = x.shape
    kp, t4 = up(k, BLOCK), up(t, 4)
    v = np.zeros((t, kp))
    v[:, :k] = x
    codes = np.zeros((t, kp))
    scales = np.full((kp // BLOCK, t4), MIN_EXP + 127, np.uint8)
    for b in range(kp // BLOCK):
        cols = slice(b * BLOCK, (b + 1) * BLOCK)
        for r in range(t):
            e = exponent(_finite_max(v[r, cols]))
            scales[b, r] = e + 127
            codes[r, cols] = round_e4m3(v[r, cols] * 2.0 ** -e)
    return codes, scales


def quantize_weight(w: np.ndarray):
    """(code values [N, Kp], scale bytes [Np / 128, Kp / 128], and both
    transposed: [K, Np], [Kp / 128, Np / 128]) of w [N, K]."""
    n, k = w.shape
    np_, kp = up(n, BLOCK), up(k, BLOCK)
    v = np.zeros((np_, kp))
    v[:n, :k] = w
    codes = np.zeros((np_, kp))
    scales = np.zeros((np_ // BLOCK, kp // BLOCK), np.uint8)
    for i in range(np_ // BLOCK):
        for j in range(kp // BLOCK):
            at = (slice(i * BLOCK, (i + 1) * BLOCK), slice(j * BLOCK, (j + 1) * BLOCK))
            e = exponent(_finite_max(v[at]))
            scales[i, j] = e + 127
            codes[at] = round_e4m3(v[at] * 2.0 ** -e)
    return codes[:n], scales, codes.T[:k].copy(), scales.T.copy()


def row_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """The values that rows' codes and scale bytes stand for."""
    t = codes.shape[0]
    s = 2.0 ** (scales[:, :t].T.astype(np.float64) - 127)
    return codes * np.repeat(s, BLOCK, axis=1)


def weight_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """The values that a weight's (or its transpose's) codes stand for."""
    s = 2.0 ** (scales.astype(np.float64) - 127)
    return codes * np.repeat(np.repeat(s, BLOCK, axis=0)[:codes.shape[0]], BLOCK, axis=1)


def matmul(a: np.ndarray, b: np.ndarray):
    """(a b^T, |a| |b|^T) of operand values; the second bounds rounding."""
    return a @ b.T, np.abs(a) @ np.abs(b).T


def weight_grad(dy: np.ndarray, x: np.ndarray, base=None):
    """(base + dy^T x, |base| + |dy|^T |x|)."""
    g, m = dy.T @ x, np.abs(dy).T @ np.abs(x)
    return (g, m) if base is None else (base + g, np.abs(base) + m)
