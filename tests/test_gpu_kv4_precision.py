"""How exact the attention's outputs are: next to nothing is lost beside the
output's own rounding, whatever the steps of the values' groups are.

Bar.  With r = the norm of (rounded exact result - exact result) and e that of
what the kernel loses before it rounds, the outputs are sqrt(r^2 + e^2) off.
The weights p s enter the product with the values' codes with half a step of
2^-11 (fp16 results: of about 2^-22), where a bf16 result's own half step is
2^-8.  A sum over many keys has the relative error of its terms, times
|c - 8| s over the spread of the values, which is about one; so e is about r / 8
for bf16 and the outputs are sqrt(1 + 1/64) r = 1.008 r off.  fp32 sums add less
than a tenth of r for either type (2^-24 times 72 s per step of 128 keys,
against results of 4 s / sqrt(keys)).  1.05 r leaves room for both:
sqrt(1 + 1/64 + 1/100) = 1.013.  With weights in bf16, e is r and more."""

import numpy as np
import pytest

import bit_quantized_lora_03_amd as q
from oracle import u4
from tests import attention_ref as ref
from tests.gpu_util import Guarded
from tests.test_gpu_kv4 import Pool, strided
from tests.test_gpu_u4 import f64, tdtype

pytestmark = pytest.mark.gpu

SCALE = {D: float(np.float32(D ** -0.5)) for D in (64, 128, 256)}


def attend(pool, new, Hq, dtype, causal=True, window=0, max_len=None, seed=1):
    import torch
    qq = strided(sum(new), Hq, pool.D, tdtype(dtype), np.random.default_rng(seed), 8)
    out, lse = Guarded(qq.shape, tdtype(dtype)), Guarded(qq.shape[:2], torch.float32)
    q.kv4_attention(pool.cache(), qq, *pool.ints(new), max(new),
                    max(max(pool.lens), 0) if max_len is None else max_len, causal=causal,
                    window=window, out=out.t, lse=lse.t)
    out.check("out")
    lse.check("lse")
    return f64(qq), f64(out.t), f64(lse.t)


def check_norm(name, got, exact, dtype):
    assert np.all(np.isfinite(got)), name
    r = np.linalg.norm(ref.round16(exact, dtype) - exact)
    off = np.linalg.norm(got - exact)
    print(f"  {name}: {off / np.linalg.norm(exact):.2e} off, "
          f"{r / np.linalg.norm(exact):.2e} by rounding alone", flush=True)
    assert off <= 1.05 * r, (name, off / r)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,Hq,Hkv,new,lens", [
    (64, 4, 2, [1, 1, 2], [777, 40, 3000]), (128, 8, 2, [1, 3], [4000, 900]),
    (128, 8, 1, [9, 20], [1500, 700]), (256, 2, 1, [1, 12], [2000, 600])])
def test_outputs_are_off_by_their_rounding(cuda, dtype, D, Hq, Hkv, new, lens):
    pool = Pool(lens, 16, Hkv, D, seed=D + Hq).fill()
    qv, o, lse = attend(pool, new, Hq, dtype)
    ro, _ = ref.outputs(pool, qv, new, SCALE[D])
    check_norm(f"{dtype} D{D} lens{lens}", o, ro, dtype)
    ref.check_lse(pool, qv, lse, new, SCALE[D])


def steps_pool(scale_of, lens, D, seed=3):
    """Values of token t scaled by scale_of(t)."""
    pool = Pool(lens, 16, 1, D, seed=seed).fill()
    for b, n in enumerate(lens):
        x = pool.rng.standard_normal((n, 1, D)) * scale_of(np.arange(n))[:, None, None]
        c, p = u4.encode(x)
        for t in range(n):
            at = pool.table[b, t // 16], slice(None), t % 16
            pool.codes["v"][at], pool.pairs["v"][at] = u4.pack(c[t]), p[t]
    return pool


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", ["rising", "falling", "tiny", "large", "one"])
def test_steps_of_every_size(cuda, D, kind):
    """Steps that rise or fall by 2^110 along the axis, all near 2^-50, all
    near 2^90, and one token far above the others."""
    n = 1100
    scale_of = {"rising": lambda t: 2.0 ** (-40 + t / 10.0), "falling": lambda t: 2.0 ** (70 - t / 10.0),
                "tiny": lambda t: np.full(t.shape, 2.0 ** -50), "large": lambda t: np.full(t.shape, 2.0 ** 90),
                "one": lambda t: np.where(t == 517, 2.0 ** 40, 1.0)}[kind]
    pool = steps_pool(scale_of, [n, 33], D)
    for max_len in (n, 100000):
        qv, o, lse = attend(pool, [2, 1], 4, "bf16", max_len=max_len)
        ro, _ = ref.outputs(pool, qv, [2, 1], SCALE[D])
        for b, rows in ((0, slice(0, 2)), (1, slice(2, 3))):
            check_norm(f"{kind} D{D} {b}", o[rows], ro[rows], "bf16")
        ref.check_lse(pool, qv, lse, [2, 1], SCALE[D])


def test_constant_values_come_back(cuda):
    """Groups without a spread (s = 0): the result is their value."""
    pool = Pool([300, 5], 16, 1, 64, seed=4).fill()
    pool.pairs["v"][..., 0] = 0
    pool.pairs["v"][..., 1] = 0x4040                 # 3.0
    _, o, _ = attend(pool, [1, 1], 2, "bf16")
    assert (o == 3.0).all()


def test_large_steps_out_of_a_rows_window(cuda):
    """Rows of one tile of which some see tokens 2^60 above the others'."""
    pool = steps_pool(lambda t: np.where(t < 100, 2.0 ** 60, 1.0), [150], 128)
    new, window = [12], 46                           # rows 138 - 45 = 93 .. 149 - 45 = 104
    qv, o, lse = attend(pool, new, 2, "bf16", window=window)
    ro, _ = ref.outputs(pool, qv, new, SCALE[128], window=window)
    for i in range(12):
        check_norm(f"row {i}", o[i], ro[i], "bf16")
    ref.check_lse(pool, qv, lse, new, SCALE[128], window=window)


def test_steps_behind_the_length_have_no_effect(cuda):
    pool = Pool([128], 16, 1, 128, seed=5).fill()
    pool.lens = [101]
    first = attend(pool, [3], 4, "bf16")[1:]
    for t in range(101, 128):                        # steps of 2^120 and infinite ones
        pool.pairs["v"][pool.table[0, t // 16], :, t % 16] = (0x7B80, 0x7F80) if t % 2 else (0x7F80, 0)
    again = attend(pool, [3], 4, "bf16")[1:]
    for a, b in zip(first, again):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("at,score,size", [
    (0, -70.0, 40), (300, -70.0, 40), (517, -30.0, 30), (3, 0.0, 0), (1000, -120.0, 90)])
def test_large_values_without_weight(cuda, D, dtype, at, score, size):
    """One visible token whose values are 2^size larger but whose score leaves
    it next to no weight: the others' values lose nothing.  Before the first
    token with weight, among them and last."""
    import torch
    n, L = 1, 1100
    pool = steps_pool(lambda t: np.where(t == at, 2.0 ** size, 1.0), [L], D)
    qq = strided(n, 1, D, tdtype(dtype), np.random.default_rng(9), 8)
    x = f64(qq)[0, 0]
    if score:
        k = x * (score * D ** 0.5 / (x @ x))
        c, p = u4.encode(k[None])
        where = pool.table[0, at // 16], 0, at % 16
        pool.codes["k"][where], pool.pairs["k"][where] = u4.pack(c[0]), p[0]
    for max_len in (L, 100000):
        out, lse = Guarded(qq.shape, tdtype(dtype)), Guarded(qq.shape[:2], torch.float32)
        q.kv4_attention(pool.cache(), qq, *pool.ints([n]), 1, max_len, out=out.t, lse=lse.t)
        ro, _ = ref.outputs(pool, f64(qq), [n], SCALE[D])
        assert np.abs(ro).max() < 4                  # the token is not in the result
        check_norm(f"{dtype} D{D} {at} {score} 2^{size}", f64(out.t), ro, dtype)
        ref.check_lse(pool, f64(qq), f64(lse.t), [n], SCALE[D])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_scores_and_steps_against_each_other(cuda, D):
    """Scores that rise by 2^200 along the axis while the steps fall by 2^100,
    and the other way round."""
    import torch
    L = 900
    for sign in (1.0, -1.0):
        pool = steps_pool(lambda t: 2.0 ** (-sign * (t - 450) / 9.0), [L], D)
        qq = strided(1, 1, D, torch.bfloat16, np.random.default_rng(9), 8)
        x = f64(qq)[0, 0]
        scores = sign * np.linspace(-70, 70, L)
        c, p = u4.encode(x[None] * (scores[:, None] * D ** 0.5 / (x @ x)))
        for t in range(L):
            where = pool.table[0, t // 16], 0, t % 16
            pool.codes["k"][where], pool.pairs["k"][where] = u4.pack(c[t]), p[t]
        for max_len in (L, 100000):
            out, lse = Guarded(qq.shape, torch.bfloat16), Guarded(qq.shape[:2], torch.float32)
            q.kv4_attention(pool.cache(), qq, *pool.ints([1]), 1, max_len, out=out.t, lse=lse.t)
            ro, _ = ref.outputs(pool, f64(qq), [1], SCALE[D])
            check_norm(f"D{D} {sign}", f64(out.t), ro, "bf16")
            ref.check_lse(pool, f64(qq), f64(lse.t), [1], SCALE[D])


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("at", [0, 150, 700, 1099])
@pytest.mark.parametrize("size", [20, 60, 95])
def test_large_values_among_constant_ones(cuda, D, at, size):
    """Tokens without a spread (s = 0, values 0 or 1) and one whose values are
    2^size: it is weighted as the others are."""
    for rest in (0.0, 1.0):
        pool = steps_pool(lambda t: np.where(t == at, 2.0 ** size, 0.0), [1100], D)
        x = np.full((1100, 1, D), rest)
        x[at] = pool.rng.standard_normal((1, D)) * 2.0 ** size
        c, p = u4.encode(x)
        for t in range(1100):
            where = pool.table[0, t // 16], slice(None), t % 16
            pool.codes["v"][where], pool.pairs["v"][where] = u4.pack(c[t]), p[t]
        for max_len in (1100, 0):              # chunks of 256, and one
            qv, o, lse = attend(pool, [2], 2, "bf16", causal=False, max_len=max_len)
            ro, _ = ref.outputs(pool, qv, [2], SCALE[D], causal=False)
            check_norm(f"D{D} {at} 2^{size} {rest}", o, ro, "bf16")
            ref.check_lse(pool, qv, lse, [2], SCALE[D], causal=False)
