"""GPU parity of the 4-bit group format and its few-token product against the
fp64 oracle.

Bars.  Codes and pairs are compared bit for bit: the kernel decides borders
in fp64, as the oracle does.  A decoded value is m + s c rounded to fp32 and
once more to 16 bits (u = 2^-8 bf16, 2^-11 fp16; half a step at the fp16
subnormals, 2^-25).  The product: with a group's sums d = sum x (OFF + c) and
X = sum x, each fp32 sum of at most G terms (and the scaled sums over
groups, waves) is off by at most (terms + 2) 2^-24 of the sum of its terms'
magnitudes, so
  |y - ref| <= u |ref| + 2^-24 sum_g (G + groups + 40) sum|x| (s (2 OFF + 15) + |m - OFF s|)
(OFF = 128 for bf16, 16 for fp16; 40 covers the join of the waves and the
roundings of s d, m - OFF s and the scale)."""

import numpy as np
import pytest

import bit_quantized_lora_03_amd as q
from oracle import u4
from tests.gpu_util import Guarded

pytestmark = pytest.mark.gpu

TYPES = {"bf16": (2.0 ** -8, 128.0), "f16": (2.0 ** -11, 16.0)}


def tdtype(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16}[name]


def bits(t):
    import torch
    return t.detach().view(torch.int16).cpu().numpy().view(np.uint16)


def f64(t):
    return t.detach().double().cpu().numpy()


def to_dev(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def pairs_dev(p):
    import torch
    return to_dev(p.astype(np.uint16).view(np.int16)).view(torch.bfloat16)


def weight(N, K, G, seed=0, offset=0.0):
    w = (np.random.default_rng(seed).standard_normal((N, K)) * 0.05 + offset).astype(np.float32)
    return w, u4.quantize_weight(w, G)


# ---------------------------------------------------------------------------
# quantiser
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("N,groups", [(1, 1), (1, 3), (3, 5), (17, 31), (64, 16), (129, 77)])
def test_quantize_is_bit_exact(cuda, G, N, groups):
    w, (codes, pairs) = weight(N, G * groups, G, seed=N + groups)
    w[0, :G] = 0.25                                  # constant, exact in bf16
    w[-1, -G:] = 0.1                                 # constant, not exact
    codes, pairs = u4.quantize_weight(w, G)
    uw = q.quantize_u4(to_dev(w), G)
    assert np.array_equal(bits(uw.pairs), pairs)
    assert np.array_equal(uw.codes.cpu().numpy(), codes)
    assert (uw.N, uw.K, uw.group) == (N, G * groups, G)


@pytest.mark.parametrize("G", [32, 64, 128])
def test_quantize_ties_scales_and_special_groups(cuda, G):
    rng = np.random.default_rng(G)
    # values on the borders: bf16 inputs whose quotients are often k + 1/2
    t = rng.integers(-64, 65, (64, G)).astype(np.float32) * np.float32(0.125)
    rows = [t]
    for e in (-140, -126, -110, -101, -99, -60, 60, 100, 126):
        rows.append(np.ldexp(rng.standard_normal((8, G)), e).astype(np.float32))
    rows.append((rng.standard_normal((32, G)) + 1e4).astype(np.float32))  # range far below the offset
    s = rng.standard_normal((8, G)).astype(np.float32)
    s[0, 3], s[1, G - 1], s[2, 0], s[3] = np.nan, np.inf, -np.inf, np.nan
    s[4, 7], s[5, 7] = 3.4e38, -3.4e38
    rows.append(s)
    w = np.concatenate(rows)
    codes, pairs = u4.quantize_weight(w, G)
    uw = q.quantize_u4(to_dev(w), G)
    assert np.array_equal(bits(uw.pairs), pairs)
    assert np.array_equal(uw.codes.cpu().numpy(), codes)


def test_quantize_writes_nothing_else(cuda):
    import torch
    n, G = 64 * 37, 64
    w = torch.randn(1, n, device="cuda")
    codes, pairs = Guarded((n // 2,), torch.uint8), Guarded((n // G, 2), torch.int16)
    q.lib().qlora_quantize_u4(w.data_ptr(), n, G, codes.t.data_ptr(), pairs.t.data_ptr(),
                              torch.cuda.current_stream().cuda_stream)
    codes.check("codes")
    pairs.check("pairs")
    c, p = u4.quantize_weight(w.cpu().numpy(), G)
    assert np.array_equal(codes.t.cpu().numpy(), c[0])
    assert np.array_equal(bits(pairs.t), p[0])


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("N,groups", [(1, 1), (5, 7), (64, 33)])
def test_dequantize(cuda, dtype, G, N, groups):
    _, (codes, pairs) = weight(N, G * groups, G, seed=9)
    pairs[0, 0] = u4.NAN_BITS
    got = f64(q.dequantize_u4(q.U4Weight(to_dev(codes), pairs_dev(pairs)), tdtype(dtype)))
    ref = u4.weight_values(codes, pairs)
    assert np.isnan(got[0, :G]).all()
    got, ref = got.reshape(-1)[G:], ref.reshape(-1)[G:]
    u = TYPES[dtype][0]
    # once to fp32 (2^-24), once to 16 bits
    assert np.all(np.abs(got - ref) <= np.maximum((u + 2.0 ** -23) * np.abs(ref), 2.0 ** -25))


# ---------------------------------------------------------------------------
# product
# ---------------------------------------------------------------------------

def check_linear(name, got, x, codes, pairs, dtype):
    u, off = TYPES[dtype]
    x, N, groups = f64(x), codes.shape[0], pairs.shape[1]
    G = 2 * codes.shape[1] // groups
    ref = x @ u4.weight_values(codes, pairs).T
    s, m = u4.bits_value(pairs[..., 0]), u4.bits_value(pairs[..., 1])
    ax = np.abs(x).reshape(x.shape[0], groups, G).sum(-1)
    mag = ax @ (s * (2 * off + 15) + np.abs(m - off * s)).T
    tol = u * np.abs(ref) + 2.0 ** -24 * (G + groups + 40) * mag
    if dtype == "f16":
        tol = np.maximum(tol, 2.0 ** -25)
    err = np.abs(f64(got) - ref)
    assert np.all(np.isfinite(f64(got))), name
    print(f"  {name}: worst err / bar {np.max(err / np.maximum(tol, 1e-300)):.3f}", flush=True)
    assert np.all(err <= tol), name


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("M,N,groups", [
    (1, 1, 1), (1, 16, 2), (2, 17, 3), (1, 1000, 16), (5, 64, 7), (16, 250, 40), (17, 33, 9),
    (31, 100, 17), (33, 48, 5), (48, 129, 64), (64, 300, 21), (65, 40, 18), (130, 70, 3)])
def test_linear(cuda, dtype, G, M, N, groups):
    import torch
    K = G * groups
    _, (codes, pairs) = weight(N, K, G, seed=M + N)
    x = to_dev(np.random.default_rng(M).standard_normal((M, K)).astype(np.float32)).to(tdtype(dtype))
    y = Guarded((M, N), tdtype(dtype))
    uw = q.U4Weight(to_dev(codes), pairs_dev(pairs))
    assert q.linear_u4_fwd(uw, x, y=y.t) is y.t
    y.check("y")
    check_linear(f"{dtype} G{G} {M}x{N}x{K}", y.t, x, codes, pairs, dtype)
    again = q.linear_u4_fwd(uw, x)
    assert torch.equal(again.view(torch.int16), y.t.view(torch.int16))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K,G", [(1, 4096, 4096, 64), (16, 1111, 8192, 128), (40, 2048, 4096, 32)])
def test_linear_larger(cuda, dtype, M, N, K, G):
    _, (codes, pairs) = weight(N, K, G, seed=7, offset=0.01)
    x = to_dev(np.random.default_rng(8).standard_normal((M, K)).astype(np.float32)).to(tdtype(dtype))
    y = q.linear_u4_fwd(q.U4Weight(to_dev(codes), pairs_dev(pairs)), x)
    check_linear(f"{dtype} {M}x{N}x{K}", y, x, codes, pairs, dtype)


@pytest.mark.parametrize("dtype,M,N,K,G", [
    # several row tiles per block, with 16, 8 and 4 waves, and a K whose last
    # unit is partial; each token-tile variant
    ("bf16", 1, 8203, 4160, 64), ("f16", 4, 9001, 4224, 128), ("bf16", 1, 20000, 2112, 64),
    ("f16", 3, 17000, 2080, 32), ("bf16", 2, 70000, 384, 128), ("bf16", 16, 9000, 1056, 32),
    ("f16", 9, 40011, 320, 64), ("bf16", 20, 9000, 640, 64), ("f16", 50, 9000, 1152, 128),
    ("bf16", 70, 9000, 160, 32)])
def test_linear_many_rows(cuda, dtype, M, N, K, G):
    _, (codes, pairs) = weight(N, K, G, seed=11)
    x = to_dev(np.random.default_rng(12).standard_normal((M, K)).astype(np.float32)).to(tdtype(dtype))
    y = Guarded((M, N), tdtype(dtype))
    q.linear_u4_fwd(q.U4Weight(to_dev(codes), pairs_dev(pairs)), x, y=y.t)
    y.check("y")
    check_linear(f"{dtype} {M}x{N}x{K}", y.t, x, codes, pairs, dtype)


@pytest.mark.parametrize("M,K,G", [(1, 96, 32), (4, 192, 64), (13, 416, 32), (33, 160, 32), (60, 384, 128)])
def test_linear_what_lies_between_the_rows_of_x(cuda, M, K, G):
    """NaN beside x in its wider tensor, before the first and behind the last
    row and between the rows, stays out of y."""
    import torch
    _, (codes, pairs) = weight(70, K, G)
    wide = torch.full((M + 2, K + 64), float("nan"), device="cuda", dtype=torch.bfloat16)
    x = wide[1:M + 1, 16:16 + K]
    x.copy_(torch.randn(M, K, device="cuda"))
    y = q.linear_u4_fwd(q.U4Weight(to_dev(codes), pairs_dev(pairs)), x)
    check_linear(f"{M}x{K}", y, x, codes, pairs, "bf16")


@pytest.mark.parametrize("M", [1, 7, 40])
def test_linear_strided_rows(cuda, M):
    import torch
    N, K, G = 90, 192, 64
    _, (codes, pairs) = weight(N, K, G)
    wide = torch.randn(M, K + 72, device="cuda").to(torch.bfloat16)
    x = wide[:, 8:8 + K]
    out = torch.full((M, N + 13), 7.0, device="cuda", dtype=torch.bfloat16)
    y = out[:, 3:3 + N]                              # odd: rows need no alignment
    q.linear_u4_fwd(q.U4Weight(to_dev(codes), pairs_dev(pairs)), x, y=y)
    check_linear("strided", y, x, codes, pairs, "bf16")
    assert (out[:, :3] == 7).all() and (out[:, 3 + N:] == 7).all()


def test_linear_keeps_non_finite_values_in_their_row_and_column(cuda):
    import torch
    M, N, K, G = 20, 40, 256, 64
    _, (codes, pairs) = weight(N, K, G)
    pairs[5, 2] = u4.NAN_BITS
    x = torch.randn(M, K, device="cuda").to(torch.bfloat16)
    x[3, 100] = float("inf")
    x[19, 0] = float("nan")
    y = f64(q.linear_u4_fwd(q.U4Weight(to_dev(codes), pairs_dev(pairs)), x))
    bad = ~np.isfinite(y)
    want = np.zeros((M, N), bool)
    want[[3, 19]] = True
    want[:, 5] = True
    assert np.array_equal(bad, want)


def test_linear_no_tokens_and_refusals(cuda):
    import torch
    _, (codes, pairs) = weight(32, 128, 64)
    uw = q.U4Weight(to_dev(codes), pairs_dev(pairs))
    x = torch.zeros(0, 128, device="cuda", dtype=torch.bfloat16)
    assert q.linear_u4_fwd(uw, x).shape == (0, 32)
    good = torch.zeros(4, 128, device="cuda", dtype=torch.bfloat16)
    for bad in (good.float(), good[:, :64], good.cpu(), good[0], good.t().contiguous().t()):
        with pytest.raises(ValueError):
            q.linear_u4_fwd(uw, bad)
    with pytest.raises(ValueError):
        q.linear_u4_fwd(uw, good, y=torch.zeros(4, 31, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        q.linear_u4_fwd(uw, good, y=torch.zeros(4, 32, device="cuda", dtype=torch.float16))
    with pytest.raises(q.QloraError):                # rows 132 elements apart: not 16-byte aligned
        q.linear_u4_fwd(uw, torch.zeros(4, 132, device="cuda", dtype=torch.bfloat16)[:, :128])
    w = torch.zeros(4, 96, device="cuda")
    for g in (64, 48, 0):
        with pytest.raises(ValueError):
            q.quantize_u4(w, g)
    with pytest.raises(ValueError):
        q.quantize_u4(w.half(), 32)
    with pytest.raises(ValueError):
        q.dequantize_u4(uw, torch.float32)
    with pytest.raises(ValueError):
        q.U4Weight(uw.codes[:16], uw.pairs)
    with pytest.raises(ValueError):
        q.U4Weight(uw.codes, uw.pairs[:, :1].contiguous()[:, :, :1])


def test_merged_adapter_to_the_group_format(cuda):
    """Merge, quantise again, serve: the served product is the merged layer's
    within the format's half steps."""
    import torch
    from bit_quantized_lora_03_amd import workloads
    L = workloads.layer(4, 128, 256, 8, 16.0, seed=3)
    dev = lambda a: to_dev(a.view(np.int16) if a.dtype == np.uint16 else a)  # noqa: E731
    f, _, _ = q.merge_adapter(dev(L.w), dev(L.A_bits), dev(L.B_bits), L.alpha)
    f2, _, uw = q.merge_adapter(dev(L.w), dev(L.A_bits), dev(L.B_bits), L.alpha, requantize="u4")
    assert torch.equal(f, f2) and isinstance(uw, q.U4Weight) and uw.group == 64
    codes, pairs = u4.quantize_weight(f.cpu().numpy(), 64)
    assert np.array_equal(uw.codes.cpu().numpy(), codes) and np.array_equal(bits(uw.pairs), pairs)
    x = dev(L.x_bits).view(torch.bfloat16)
    y = f64(q.linear_u4_fwd(uw, x))
    ref = f64(x) @ f64(f).T
    half = np.abs(f64(x)).reshape(4, 4, 64).sum(-1) @ (u4.bits_value(pairs[..., 0]) / 2).T
    assert np.all(np.abs(y - ref) <= half + 2.0 ** -7 * (np.abs(ref) + half))
    with pytest.raises(ValueError):
        q.merge_adapter(dev(L.w), dev(L.A_bits), dev(L.B_bits), L.alpha, requantize="other")
