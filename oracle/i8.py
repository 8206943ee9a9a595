"""The 8-bit row format, its products and the norm that writes it, in fp64
(numpy, no code shared with the library).

A row with the largest magnitude a has the fp32 scale s = a / 127 and codes
rint(127 v / a), ties to even; a value is s times its code.  A row with a NaN
or an infinity, or whose scale is not finite in fp32, has s = NaN and codes 0.
"""

from __future__ import annotations

from fractions import Fraction

import numpy as np


def padded(K: int) -> int:
    return -(-K // 128) * 128


def nearest_code(v, a) -> int:
    """rint(127 v / a) by exact rationals (one value)."""
    x = 127 * Fraction(float(v)) / Fraction(float(a))
    return round(x)                                   # Python rounds halves to even


def encode(v, times=1.0):
    """Rows [R, K] fp64 -> (codes int8 [R, K], scales fp32 [R]); ``times`` is
    a factor of the scales that the codes do not have.

    The fp64 quotient of inputs of up to 24 bits is a half only where the exact
    one is, so rint decides every border as the exact quotient does."""
    v = np.asarray(v, dtype=np.float64)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        a = np.abs(v).max(-1)
        s = (a * times / 127.0).astype(np.float32)
        ok = np.isfinite(v).all(-1) & np.isfinite(s)
        q = np.rint(127.0 * v / a[..., None])
        c = np.where((ok & (a > 0))[..., None], q, 0.0).astype(np.int8)
    return c, np.where(ok, s, np.float32(np.nan)).astype(np.float32)


def decode(c, s):
    return np.asarray(c, dtype=np.float64) * np.asarray(s, dtype=np.float64)[..., None]


def pad(c):
    """Codes [R, K] -> [R, Kp] with zeros."""
    out = np.zeros((c.shape[0], padded(c.shape[1])), dtype=np.int8)
    out[:, :c.shape[1]] = c
    return out


def tile(c):
    """Codes [N, K] -> the weight's tiles, byte by byte as the header says."""
    N, K = c.shape
    Kp = padded(K)
    out = np.zeros(-(-N // 16) * 16 * Kp, dtype=np.int8)
    n, k = np.meshgrid(np.arange(N), np.arange(K), indexing="ij")
    at = ((n // 16) * (Kp // 64) + k // 64) * 1024 + (k % 64) // 16 * 256 + (n % 16) * 16 + k % 16
    out[at] = c
    return out.reshape(-1, Kp // 64, 4, 16, 16)


def sums(cx, cw):
    """Exact integer sums [M, N] of the codes' products (below 2^53 in fp64
    whatever the order)."""
    return (np.asarray(cx, dtype=np.float64) @ np.asarray(cw, dtype=np.float64).T).astype(np.int64)


def product(cx, sx, cw, sw):
    """[M, N] fp64."""
    with np.errstate(invalid="ignore"):
        return sums(cx, cw) * np.asarray(sw, np.float64) * np.asarray(sx, np.float64)[:, None]


def activation(g, act):
    g = np.asarray(g, dtype=np.float64)
    with np.errstate(over="ignore"):
        if act == "silu":
            return g / (1.0 + np.exp(-g))
        return 0.5 * g * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (g + 0.044715 * g ** 3)))


def norm(h, weight, eps):
    """The rows h (what is stored of x + residual) -> (codes, scales)."""
    h = np.asarray(h, dtype=np.float64)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        root = np.sqrt((h * h).mean(-1) + eps)
        return encode(h * np.asarray(weight, dtype=np.float64), 1.0 / root)
