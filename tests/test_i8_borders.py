"""Quotients 127 v / a that come as close to a half as such inputs let them:
their codes are the exact quotients' (oracle on the CPU, kernels on the GPU).

A quotient that is no half differs from h / 2, h odd, by |254 v - h a| / (h a)
of it.  With v = V 2^e and a = A 2^f the difference is a multiple of 2^min(e, f):
where that is 2^f, or e = f, it is at least 1 / (h A) of h / 2; where e < f it is
even, so at least 2 2^e / (h a), and h a is 254 v but for that: 1 / (127 V).
With A, V < 2^24 and h <= 253 both are above 2^-32, with 22 bits above 2^-30."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import i8


def pairs(top):
    """(V, A, h): 254 V = h A -+ 1, with the largest A below ``top``."""
    out = []
    for h in range(1, 254, 2):
        if h == 127:
            continue                                     # 254 V = 127 A -+ 1 has no solution
        for sign in (1, -1):
            A = sign * pow(h, -1, 254) % 254
            A += (top - 1 - A) // 254 * 254
            V, rest = divmod(h * A - sign, 254)
            assert rest == 0
            out.append((V, A, h))
    return out


def distance(v, a, h):
    """of 127 v / a from h / 2, of the latter."""
    half = Fraction(h, 2)
    return abs(127 * Fraction(v) / Fraction(a) - half) / half


def weight_rows(scale):
    """[R, 140] fp32, a row for each pair: its largest value, the close one and
    its negative; and the pair that is close to 1 / 2 from the other side."""
    p = pairs(1 << 24) + [(16777215, 16646143 * 256, 1)]
    w = np.zeros((len(p), 140))
    for r, (V, A, _) in enumerate(p):
        w[r, r % 140], w[r, (r + 1) % 140], w[r, (r + 70) % 140] = A, V, -V
    return (w * scale).astype(np.float32), p


def test_how_close_they_are():
    p = pairs(1 << 24)
    near = [distance(V, A, h) for V, A, h in p]
    assert len(p) == 252 and all(d == Fraction(1, h * A) for d, (V, A, h) in zip(near, p))
    assert Fraction(1, 2 ** 32) < min(near) < Fraction(1, 2 ** 31)
    d = distance((2 ** 24 - 1) / 256, 16646143, 1)
    assert Fraction(1, 2 ** 32) < d < Fraction(1, 2 ** 30)


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -140, 2.0 ** 90])
def test_oracle(scale):
    w, p = weight_rows(scale)
    c, _ = i8.encode(w)
    for r in range(len(p)):
        a = np.abs(w[r]).max()
        at = np.flatnonzero(w[r])
        assert [i8.nearest_code(w[r, k], a) for k in at] == c[r, at].tolist()
    if scale == 1.0:
        # fp32 takes the quotient for the half, whose code is the even one
        q32 = np.rint(np.float32(127) * w / np.abs(w).max(-1, keepdims=True))
        assert q32.dtype == np.float32 and not np.array_equal(q32, c)


def product_rows():
    """Values p q of two fp16 numbers of 11 bits, close to a half of their
    row's largest: rows [R, K] and a weight [K]."""
    rng = np.random.default_rng(11)
    bits11 = np.arange(1024, 2048)
    found = []
    while len(found) < 64:
        h = int(rng.integers(0, 127)) * 2 + 1
        if h == 127:
            continue
        s, t = (int(v) for v in rng.integers(1024, 2048, 2))
        for sign in (1, -1):
            V, rest = divmod(h * s * t - sign, 254)
            if rest == 0 and V > 0:
                by = bits11[V % bits11 == 0]
                if by.size and V // by[0] < 2048:
                    found.append((s, t, int(V // by[0]), int(by[0]), h))
    x, w = np.zeros((64, 128)), np.zeros(128)
    found = found[:64]
    for r, (s, t, u, v, h) in enumerate(found):
        x[r, 2 * r], w[2 * r], x[r, 2 * r + 1], w[2 * r + 1] = s, t, u, v
        assert Fraction(1, 2 ** 30) < distance(u * v, s * t, h) == Fraction(1, h * s * t)
    return x, w / 1024.0


def test_oracle_of_products():
    x, w = product_rows()
    c, _ = i8.encode(x * w)
    for r in range(x.shape[0]):
        assert c[r, 2 * r] == 127
        assert c[r, 2 * r + 1] == i8.nearest_code(x[r, 2 * r + 1] * w[2 * r + 1], x[r, 2 * r] * w[2 * r])


@pytest.mark.gpu
@pytest.mark.parametrize("K", [140, 5000, 12000, 30000, 40000])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -140, 2.0 ** 90])
def test_weight(cuda, scale, K):
    """In each of the quantiser's forms."""
    import bit_quantized_lora_03_amd as q
    import torch
    w, _ = weight_rows(scale)
    wide = np.zeros((w.shape[0], K), dtype=np.float32)
    wide[:, K - 140:] = w
    c, s = i8.encode(wide)
    iw = q.quantize_i8(torch.from_numpy(wide).cuda())
    assert np.array_equal(iw.tiles.cpu().numpy(), i8.tile(c))
    assert np.array_equal(iw.scales.cpu().numpy(), s)


@pytest.mark.gpu
@pytest.mark.parametrize("K", [128, 1500, 6000, 11008, 40000, 130944])
def test_norm(cuda, K):
    """In rows of one wave to sixteen."""
    import bit_quantized_lora_03_amd as q
    import torch
    x, w = (np.concatenate([np.zeros(v.shape[:-1] + (K - 128,)), v], -1) for v in product_rows())
    c, _ = i8.encode(x * w)
    xt, wt = (torch.from_numpy(v).to(torch.float16).cuda() for v in (x, w))
    assert np.array_equal(xt.double().cpu().numpy(), x)
    assert np.array_equal(wt.double().cpu().numpy(), w)
    t, _ = q.rms_norm_i8(xt, wt, 1e-5)
    assert np.array_equal(t.codes.cpu().numpy(), i8.pad(c))
