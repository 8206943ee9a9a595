"""The 4-bit group format, the few-token product, the paged cache and the
attention over it, in fp64 (numpy, no code shared with the library).

A group of G values holds a code c in 0..15 each and a pair (s, m) of bf16;
a value is m + s c.  m is the minimum rounded down to bf16, s is (maximum -
m) / 15 rounded up to bf16, c = rint((v - m) / s), ties to even.  A group
with a NaN or an infinity, or whose m or s is not finite in bf16, is NaN.
"""

from __future__ import annotations

import numpy as np

NAN_BITS = 0x7FC0


def _f32_towards(x: np.ndarray, up: bool) -> np.ndarray:
    with np.errstate(over="ignore"):
        f = x.astype(np.float32)
    wrong = (f.astype(np.float64) < x) if up else (f.astype(np.float64) > x)
    return np.where(wrong, np.nextafter(f, np.float32(np.inf if up else -np.inf)), f)


def bf16_towards(x, up: bool) -> np.ndarray:
    """fp64 -> bf16 bits (uint16) rounded towards +inf or -inf."""
    f = _f32_towards(np.atleast_1d(np.asarray(x, dtype=np.float64)), up)
    b = f.view(np.uint32)
    cut = (b & 0xFFFF) != 0
    away = cut & ((b >> 31) == (0 if up else 1))     # magnitude grows
    return ((b >> 16) + away).astype(np.uint16)


def bits_value(b: np.ndarray) -> np.ndarray:
    return (np.asarray(b, dtype=np.uint32) << 16).view(np.float32).astype(np.float64)


def encode(v: np.ndarray):
    """[..., G] -> codes uint8 [..., G], pairs uint16 [..., 2] (s, m)."""
    v = np.asarray(v, dtype=np.float64)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        m = bf16_towards(v.min(-1), False).reshape(v.shape[:-1])
        s = bf16_towards((v.max(-1) - bits_value(m)) / 15.0, True).reshape(v.shape[:-1])
        sv, mv = bits_value(s), bits_value(m)
        ok = np.isfinite(v).all(-1) & np.isfinite(sv) & np.isfinite(mv)
        q = np.rint((v - mv[..., None]) / sv[..., None])
        c = np.where((ok & (sv > 0))[..., None], q, 0.0).astype(np.uint8)
    pairs = np.stack([np.where(ok, s, NAN_BITS), np.where(ok, m, NAN_BITS)], -1).astype(np.uint16)
    return c, pairs


def pack(c: np.ndarray) -> np.ndarray:
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)


def unpack(p: np.ndarray) -> np.ndarray:
    return np.stack([p & 15, p >> 4], -1).reshape(*p.shape[:-1], 2 * p.shape[-1])


def decode(packed: np.ndarray, pairs: np.ndarray) -> np.ndarray:
    """Packed codes [..., G/2] and pairs [..., 2] -> values [..., G] fp64."""
    return (bits_value(pairs[..., 1])[..., None]
            + bits_value(pairs[..., 0])[..., None] * unpack(packed))


def quantize_weight(w: np.ndarray, group: int):
    N, K = w.shape
    c, pairs = encode(w.reshape(N, K // group, group))
    return pack(c).reshape(N, K // 2), pairs


def weight_values(codes: np.ndarray, pairs: np.ndarray) -> np.ndarray:
    N, groups, _ = pairs.shape
    return decode(codes.reshape(N, groups, -1), pairs).reshape(N, -1)


def rotate(x: np.ndarray, cos_sin, pos: np.ndarray, interleaved: bool) -> np.ndarray:
    """x [T, H, D] fp64 rotated by rows ``pos`` of the table [P, rot]."""
    y = np.array(x, dtype=np.float64)
    if cos_sin is None:
        return y
    rot = cos_sin.shape[1]
    h = rot // 2
    c = cos_sin[pos, :h].astype(np.float64)[:, None]
    s = cos_sin[pos, h:].astype(np.float64)[:, None]
    ia = np.arange(0, rot, 2) if interleaved else np.arange(h)
    ib = ia + (1 if interleaved else h)
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, pos: int, length: int, scale: float,
           causal: bool, window: int, there=None):
    """One query row q [D] at position pos over k, v [L, D]: (out [D], lse,
    weights [L]).  ``there`` marks the tokens that have a page."""
    j = np.arange(k.shape[0])
    see = j < length
    if there is not None:
        see &= there
    if causal:
        see &= j <= pos
    if window:
        see &= j > pos - window
    w = np.zeros(k.shape[0])
    if not see.any():
        return np.zeros(v.shape[1]), -np.inf, w
    z = scale * (k[see] @ q)
    top = z.max()
    e = np.exp(z - top)
    w[see] = e / e.sum()
    return w[see] @ v[see], top + np.log(e.sum()), w
