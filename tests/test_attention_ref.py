"""The bars that the GPU's attention is held to have force: an output as the
kernel may round it passes, and zeros, a lost or doubly weighted share of the
keys, weights in too few bits and exchanged rows do not (CPU only)."""

import numpy as np
import pytest

from tests import attention_ref as ref

CASES = [("bf16", 64, 1500, 2, 0), ("bf16", 128, 2500, 4, 0), ("f16", 128, 2500, 4, 700),
         ("bf16", 256, 1500, 2, 0), ("f16", 256, 1500, 1, 0)]


def case(dtype, D, L, Hq, window):
    pool = ref.HostPool([L, 40], 1, D, seed=D, values=ref.by_position)
    qv = ref.round16(np.random.default_rng(1).standard_normal((3, Hq, D)), dtype)
    return pool, qv, [2, 1], float(np.float32(D ** -0.5)), window


def bits_kept(x, n):
    m, e = np.frexp(x)
    return np.ldexp(np.rint(np.ldexp(m, n)), e - n)


def result(pool, qv, new, scale, window, dtype, change=None, weight_bits=11):
    """Outputs as the kernel forms them: the weights p s rounded, the middle
    code's share exact, one rounding at the end.  ``change`` alters the weights
    [R, L] without a word to the log sums."""
    o, lse = ref.outputs(pool, qv, new, scale, True, window)
    for t in ref.tiles(pool, qv, new, scale, True, window):
        w = t["w"] if change is None else change(t["w"])
        ps = bits_kept(w * t["vs"], weight_bits)
        o[t["at"]] = ps @ (t["vc"] - 8) + (w @ (8 * t["vs"] + t["vm"]))[:, None]
    return ref.round16(o, dtype), lse


@pytest.mark.parametrize("dtype,D,L,Hq,window", CASES)
def test_bars(dtype, D, L, Hq, window):
    pool, qv, new, scale, _ = c = case(dtype, D, L, Hq, window)

    def run(o, lse):
        ref.check_rows(pool, qv, o, lse, new, dtype, scale, True, window)

    good = 11 if dtype == "bf16" else 20
    o, lse = result(*c, dtype, weight_bits=good)
    run(o, lse)

    def fails(o2, lse2):
        with pytest.raises(AssertionError):
            run(o2, lse2)

    fails(np.zeros_like(o), lse)
    fails(o[:, ::-1] if Hq > 1 else o[::-1], lse)
    for lo, hi in ((0, 256) if not window else (L - 256, L - 100), (L - 256, L)):
        def lost(w):
            w = w.copy()
            if w.shape[1] == L:
                w[:, lo:hi] = 0
            return w

        def twice(w):
            w = w.copy()
            if w.shape[1] == L:
                w[:, lo:hi] *= 2
            return w / w.sum(1, keepdims=True)
        fails(*result(*c, dtype, lost, good))
        fails(*result(*c, dtype, twice, good))
    fails(*result(*c, dtype, weight_bits=4))
    fails(o, lse + 2e-2)


def test_rows_without_keys_and_with_nan():
    pool = ref.HostPool([0, 20], 1, 64, seed=2)
    qv = np.random.default_rng(3).standard_normal((2, 1, 64))
    scale = 0.125
    o, lse = ref.outputs(pool, qv, [1, 1], scale)
    assert not o[0].any() and lse[0, 0] == -np.inf
    ref.check_rows(pool, qv, ref.round16(o, "bf16"), lse, [1, 1], "bf16", scale)
    for bad in (np.nan, 1.0):
        o2 = ref.round16(o, "bf16")
        o2[0] = bad
        with pytest.raises(AssertionError):
            ref.check_rows(pool, qv, o2, lse, [1, 1], "bf16", scale)
    pool._of["k", 1][1][7] = 0x7FC0                  # a visible NaN
    with pytest.raises(AssertionError):
        ref.check_rows(pool, qv, ref.round16(o, "bf16"), lse, [1, 1], "bf16", scale)
    o[1], lse[1] = np.nan, np.nan
    ref.check_rows(pool, qv, o, lse, [1, 1], "bf16", scale)
