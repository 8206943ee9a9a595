"""Attention whose axis of keys is cut into many chunks, with several KV heads
and sequences: every form of the join, at every head size, with bars that a
lost chunk does not pass."""

import numpy as np
import pytest

import bit_quantized_lora_03_amd as q
from oracle import u4
from tests import attention_ref as ref
from tests.test_gpu_kv4 import Pool
from tests.test_gpu_kv4_precision import attend

pytestmark = pytest.mark.gpu


def filled(lens, page, Hkv, D, seed):
    pool = Pool(lens, page, Hkv, D, seed=seed).fill()
    for b, n in enumerate(lens):
        n = max(n, 0)
        c, p = u4.encode(ref.by_position(pool.rng.standard_normal((n, Hkv, D)),
                                         np.arange(n)[:, None, None]))
        for t in range(n):
            at = pool.table[b, t // page], slice(None), t % page
            pool.codes["v"][at], pool.pairs["v"][at] = u4.pack(c[t]), p[t]
    return pool


def chunks(pool, new, Hq, max_len, window=0):
    """How many chunks the longest sequence may have in the call's plan."""
    B, Hkv, D, rows = len(new), pool.Hkv, pool.D, max(new) * (Hq // pool.Hkv)
    tile = 32 if D == 128 and rows >= 64 else 16
    need = q.kv4_attention_workspace_bytes(B, max(new), max_len, Hq, Hkv, D, window)
    return need // (B * Hkv * -(-rows // tile) * tile * (D + 2) * 4)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,Hq,Hkv,new,lens,window,least", [
    # more than eight chunks: 16, 8 and 4 shares a row, some with several chunks
    (64, 4, 2, [1, 1, 1, 2], [256 * 33 + 5, 0, 700, 5000], 0, 33),
    (128, 6, 3, [1, 2, 1], [256 * 17 + 3, 2600, 31], 0, 17),
    (256, 4, 2, [1, 1, 2], [256 * 9 + 40, 1300, 0], 0, 10),
    (64, 2, 2, [1, 3], [9000, 6000], 5000, 9), (256, 3, 3, [2, 1], [4000, 2500], 3000, 9),
    # tiles of 32 rows
    (128, 16, 2, [9, 1], [256 * 17 + 100, 3000], 0, 9),
    # up to eight chunks, several heads
    (64, 6, 3, [1, 2, 1], [1500, 800, 2000], 0, 2), (128, 8, 4, [3, 1], [1024, 900], 0, 2),
    (256, 4, 4, [1, 5], [1030, 700], 0, 2), (128, 16, 2, [10, 4], [1500, 1100], 1000, 2)])
def test_join(cuda, dtype, D, Hq, Hkv, new, lens, window, least):
    pool = filled(lens, 16, Hkv, D, seed=D + Hq)
    n = chunks(pool, new, Hq, max(lens), window)
    assert n >= least and (least > 8 or n <= 8), n
    for max_len in (max(lens), 100000):
        qv, o, lse = attend(pool, new, Hq, dtype, window=window, max_len=max_len)
        ref.check_rows(pool, qv, o, lse, new, dtype, float(np.float32(D ** -0.5)), window=window,
                       name=f"{dtype} D{D} {Hq}/{Hkv} lens{lens} window{window} max_len{max_len}")


@pytest.mark.parametrize("D,L", [(64, 9000), (128, 4500), (256, 2600), (64, 1200), (128, 1200), (256, 1200)])
@pytest.mark.parametrize("name", ["k", "v"])
def test_nan_in_one_chunk(cuda, D, L, name):
    """A NaN in one chunk makes the rows that see it NaN, beside a sequence
    without tokens and ones without NaN."""
    lens, new = [L, 0, L, 300], [1, 1, 1, 1]
    pool = filled(lens, 32, 2, D, seed=D)
    pg, r = pool.table[0, (L // 2) // 32], L // 2 % 32
    pool.pairs[name][pg, 1, r] = u4.NAN_BITS         # head 1 of sequence 0
    qv, o, lse = attend(pool, new, 4, "bf16")
    bad = np.zeros((4, 4), bool)
    bad[0, 2:] = True
    assert np.array_equal(np.isnan(o).all(-1), bad) and np.array_equal(np.isnan(o).any(-1), bad)
    assert np.array_equal(np.isnan(lse), bad if name == "k" else np.zeros_like(bad))
    assert (o[1] == 0).all() and (lse[1] == -np.inf).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_rows(cuda, dtype, D):
    """Many rows of several heads on a long context, in one chunk and in more."""
    lens, new = [1300, 700, 90], [70, 33, 90]
    pool = filled(lens, 16, 2, D, seed=D + 1)
    for window in (0, 200):
        qv, o, lse = attend(pool, new, 4, dtype, window=window)
        ref.check_rows(pool, qv, o, lse, new, dtype, float(np.float32(D ** -0.5)), window=window,
                       name=f"{dtype} D{D} window{window}")
