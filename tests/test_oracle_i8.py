"""The 8-bit row format's oracle against exact rationals and plain loops."""

import numpy as np
import pytest

from oracle import i8


def halves(rng, rows, K, scale):
    """Rows whose quotients are often k + 1/2: a = 127 / 2^j, steps of half a code."""
    v = rng.integers(-254, 255, (rows, K)) * 0.5
    v[:, 0] = 127.0
    return (v * scale).astype(np.float32)


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -130, 2.0 ** 120, 0.37])
def test_codes_are_the_exact_quotients(scale):
    rng = np.random.default_rng(3)
    w = np.concatenate([halves(rng, 6, 40, scale), (rng.standard_normal((6, 40)) * scale).astype(np.float32)])
    c, s = i8.encode(w)
    for r in range(w.shape[0]):
        a = np.abs(w[r]).max()
        assert [i8.nearest_code(v, a) for v in w[r]] == c[r].tolist()
        assert s[r] == np.float32(np.float64(a) / 127.0)
    assert np.abs(c.astype(int)).max() == 127
    if scale == 1.0:
        assert np.any((127 * w[:6].astype(np.float64) / 127.0) % 1 == 0.5)


def test_products_of_two_16_bit_floats_are_decided_exactly():
    rng = np.random.default_rng(4)
    h = (rng.integers(1, 2 ** 11, (4, 300)) * 2.0 ** rng.integers(-12, 3, (4, 300)))
    w = rng.integers(1, 2 ** 11, 300) * 2.0 ** -10
    c, _ = i8.encode(h * w)
    for r in range(4):
        a = (h[r] * w).max()
        assert [i8.nearest_code(v, a) for v in h[r] * w] == c[r].tolist()


def test_error_zero_rows_and_rows_that_are_none():
    rng = np.random.default_rng(5)
    w = rng.standard_normal((7, 33)).astype(np.float32)
    w[1] = 0.0
    w[2, 5], w[3, 0], w[4, 32] = np.nan, np.inf, -np.inf
    c, s = i8.encode(w)
    assert s[1] == 0 and not c[1].any()
    assert np.isnan(s[2:5]).all() and not c[2:5].any()
    good = [0, 5, 6]
    a = np.abs(w[good]).max(-1, keepdims=True).astype(np.float64)
    off = np.abs(i8.decode(c[good], s[good]) - w[good])
    # half a step, and 127 codes times the scale's rounding
    assert np.all(off <= a / 254 + 127 * s[good].astype(np.float64)[:, None] * 2.0 ** -24)
    # a scale that fp32 does not hold
    c, s = i8.encode(np.full((1, 4), 1e30), times=1e20)
    assert np.isnan(s[0]) and not c.any()


@pytest.mark.parametrize("N,K", [(1, 1), (16, 64), (17, 129), (35, 200)])
def test_tiles_hold_every_code_once(N, K):
    rng = np.random.default_rng(N * K)
    c = rng.integers(-127, 128, (N, K)).astype(np.int8)
    t = i8.tile(c)
    assert t.shape == ((N + 15) // 16, i8.padded(K) // 64, 4, 16, 16)
    for n in range(N):
        for k in range(K):
            assert t[n // 16, k // 64, k % 64 // 16, n % 16, k % 16] == c[n, k]
    assert np.count_nonzero(t) == np.count_nonzero(c)


def test_product_and_norm_against_loops():
    rng = np.random.default_rng(6)
    cx, cw = (rng.integers(-127, 128, s).astype(np.int8) for s in ((3, 50), (4, 50)))
    sx, sw = rng.random(3).astype(np.float32), rng.random(4).astype(np.float32)
    y = i8.product(cx, sx, cw, sw)
    for m in range(3):
        for n in range(4):
            t = sum(int(cx[m, k]) * int(cw[n, k]) for k in range(50))
            assert y[m, n] == pytest.approx(t * float(sx[m]) * float(sw[n]), rel=1e-15)
    h, w = rng.standard_normal((3, 50)), 1 + 0.1 * rng.standard_normal(50)
    c, s = i8.norm(h, w, 1e-3)
    for m in range(3):
        r = (sum(float(v) ** 2 for v in h[m]) / 50 + 1e-3) ** -0.5
        a = max(abs(float(v) * float(u)) for v, u in zip(h[m], w))
        assert s[m] == pytest.approx(a * r / 127, rel=2.0 ** -23)
        want = [float(v) * float(u) * r for v, u in zip(h[m], w)]
        assert np.all(np.abs(i8.decode(c, s)[m] - want) <= a * r / 254 * (1 + 2.0 ** -15))


def test_activations():
    g = np.linspace(-12, 12, 97)
    import math
    for v, a, b in zip(g, i8.activation(g, "silu"), i8.activation(g, "gelu")):
        assert a == pytest.approx(v / (1 + math.exp(-v)), rel=1e-14)
        # the tanh form is within 5e-4 of gelu itself
        assert abs(b - v * 0.5 * (1 + math.erf(v / 2 ** 0.5))) < 5e-4


# planted mistakes: each differs from the oracle on these inputs
def test_mistakes_are_seen():
    rng = np.random.default_rng(7)
    w = halves(rng, 4, 64, 1.0).astype(np.float64)
    c, s = i8.encode(w)
    a = np.abs(w).max(-1, keepdims=True)
    away = np.sign(w) * np.floor(np.abs(127 * w / a) + 0.5)         # halves away from zero
    cut = np.trunc(127 * w / a)
    wide = np.clip(np.rint(128 * w / a), -128, 127)
    for wrong in (away, cut, wide):
        assert not np.array_equal(wrong, c)
    t = i8.tile(c)
    assert not np.array_equal(t, i8.tile(c[:, ::-1]))
    assert not np.array_equal(t.transpose(0, 1, 3, 2, 4).reshape(t.shape), t)
