"""Pins for the oracle's 4-bit group format, rotation and attention (CPU
only): hand-worked groups, the directed roundings against exact rationals,
the error bound, ties, degenerate groups, and attention against a direct
sum."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import u4


def test_hand_worked_group():
    # minimum -1 (exact in bf16); (14 + 1) / 15 = 1 exactly: s = 1, c = v + 1
    v = np.arange(-1.0, 15.0)
    c, p = u4.encode(v[None])
    assert p.tolist() == [[0x3F80, 0xBF80]]
    assert c.tolist() == [list(range(16))]
    assert np.array_equal(u4.decode(u4.pack(c), p)[0], v)
    assert u4.pack(c)[0, 0] == 0x10 and u4.pack(c)[0, 7] == 0xFE


def test_ties_go_to_the_even_code():
    v = np.array([0.0, 0.5, 1.5, 2.5, 13.5, 14.5, 15.0, 7.0])
    c, p = u4.encode(v[None])
    assert p.tolist() == [[0x3F80, 0x0000]]
    assert c[0].tolist() == [0, 0, 2, 2, 14, 14, 15, 7]


@pytest.mark.parametrize("up", [False, True])
def test_directed_rounding_is_the_nearest_bf16_on_its_side(up):
    rng = np.random.default_rng(3)
    x = rng.standard_normal(4000) * 10.0 ** rng.uniform(-30, 30, 4000)
    b = u4.bf16_towards(x, up)
    val = u4.bits_value(b)
    assert np.all(val >= x) if up else np.all(val <= x)
    # the neighbour towards x is on the other side of it
    toward = np.where((val > 0) == up, b.astype(np.int64) - 1, b.astype(np.int64) + 1)
    other = u4.bits_value(toward.astype(np.uint16))
    assert np.all((other < x) if up else (other > x))
    exact = u4.bits_value(np.array([0x3F80, 0xBF81, 0x0000], np.uint16))
    assert u4.bf16_towards(exact, up).tolist() == [0x3F80, 0xBF81, 0x0000]


@pytest.mark.parametrize("G", [32, 64, 128, 256])
@pytest.mark.parametrize("offset", [0.0, 40.0, -1000.0])
def test_error_is_at_most_half_a_step_and_nothing_is_clipped(G, offset):
    v = np.random.default_rng(G).standard_normal((200, G)) + offset
    c, p = u4.encode(v)
    s, m = u4.bits_value(p[:, 0]), u4.bits_value(p[:, 1])
    q = (v - m[:, None]) / s[:, None]
    assert q.min() >= 0 and q.max() <= 15
    err = np.abs(u4.decode(u4.pack(c), p) - v)
    assert np.all(err <= s[:, None] / 2 * (1 + 1e-12))
    # m and s are the tightest: the range is at most one bf16 step of each wider
    for r in range(5):
        lo, hi = Fraction(v[r].min()), Fraction(v[r].max())
        assert Fraction(m[r]) <= lo and Fraction(s[r]) * 15 >= hi - Fraction(m[r])
        assert lo - Fraction(m[r]) <= abs(Fraction(m[r])) / 64
        assert Fraction(s[r]) * 15 - (hi - Fraction(m[r])) <= 15 * Fraction(s[r]) / 64


def test_degenerate_groups():
    big = 3.4e38                                    # past bf16's largest value
    v = np.zeros((6, 32))
    v[1] = 2.5
    v[2, 5] = np.nan
    v[3, 7] = -np.inf
    v[4] = 1.0 + 2.0 ** -20                         # constant, not a bf16 value
    v[5, 0] = -big
    c, p = u4.encode(v)
    assert p[0].tolist() == [0, 0] and not c[0].any()
    assert p[1].tolist() == [0, 0x4020] and not c[1].any()
    for r in (2, 3, 5):
        assert p[r].tolist() == [u4.NAN_BITS] * 2 and not c[r].any()
    assert np.all(np.abs(u4.decode(u4.pack(c), p)[4] - v[4]) <= u4.bits_value(p[4, 0]) / 2)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [8, 16, 32])
def test_rotation_is_a_complex_product(inter, rot):
    rng = np.random.default_rng(5)
    T, H, D = 5, 3, 32
    x = rng.standard_normal((T, H, D))
    ang = rng.uniform(-7, 7, (9, rot // 2))
    table = np.concatenate([np.cos(ang), np.sin(ang)], -1).astype(np.float32)
    pos = np.array([0, 8, 3, 3, 1])
    y = u4.rotate(x, table, pos, inter)
    for t in range(T):
        z = table[pos[t], :rot // 2].astype(np.float64) + 1j * table[pos[t], rot // 2:]
        for h in range(H):
            for i in range(rot // 2):
                a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
                w = (x[t, h, a] + 1j * x[t, h, b]) * z[i]
                assert abs(w - (y[t, h, a] + 1j * y[t, h, b])) < 1e-12
    assert np.array_equal(y[..., rot:], x[..., rot:])


def test_attention_against_a_direct_sum():
    rng = np.random.default_rng(6)
    L, D = 9, 4
    q, k, v = rng.standard_normal(D), rng.standard_normal((L, D)), rng.standard_normal((L, D))
    there = np.ones(L, bool)
    there[2] = False
    o, lse, w = u4.attend(q, k, v, 6, 8, 0.3, True, 5, there)
    see = [3, 4, 5, 6]                               # 6 - 5 < j <= 6
    e = [np.exp(0.3 * float(np.dot(q, k[j]))) for j in see]
    assert np.allclose(o, sum(x * v[j] for x, j in zip(e, see)) / sum(e), atol=1e-13)
    assert abs(lse - np.log(sum(e))) < 1e-13 and np.flatnonzero(w).tolist() == see
    o, lse, w = u4.attend(q, k, v, -1, 8, 0.3, True, 0)
    assert not o.any() and lse == -np.inf and not w.any()
