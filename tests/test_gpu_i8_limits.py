"""The 8-bit calls with as many tokens and rows as they take, over more rows
than one launch has, and several at once on streams of their own.

A row's result does not depend on the others, so rows are compared bit for bit
with the same ones alone, and products' last columns with torch's in fp64 (sums
of K products of two codes are exact in it and round to fp32 as the library's)."""

import pytest

import bit_quantized_lora_03_amd as q
from tests.test_gpu_i8_extremes import random_codes

pytestmark = pytest.mark.gpu


def tokens(M, K):
    import torch
    codes = random_codes(M, 128)
    codes[:, K:] = 0
    return q.I8Tokens(codes, torch.rand(M, device="cuda") + 0.5, K)


def weight(N, K):
    """Random codes [N, K], N a multiple of 16 and K 64 or 128."""
    import torch
    tiles = random_codes(N // 16, 2, 4, 16, 16)
    tiles[:, K // 64:] = 0
    return q.I8Weight(tiles, (torch.rand(N, device="cuda") + 0.5) / 5000, N, K)


def parts(n, size):
    """A few runs of ``size`` neighbouring rows of n."""
    return [slice(a, a + size) for a in sorted({max(0, v) for v in (0, n // 2, n - size)})]


@pytest.mark.parametrize("M,N,K", [((1 << 28) - 64, 16, 64), ((1 << 27) - 64, 64, 128),
                                   (1, (1 << 23) - 64, 128), (500, (1 << 23) - 64, 64)])
def test_most_tokens_and_most_rows(cuda, M, N, K):
    import torch
    torch.manual_seed(0)
    gate, up, t = weight(N, K), weight(N, K), tokens(M, K)
    last = gate.tiles[-1].permute(2, 0, 1, 3).reshape(16, 128).double()
    for gated in (False, True):
        f = (lambda x: q.gated_i8_fwd(gate, up, x)) if gated else (lambda x: q.linear_i8_fwd(gate, x))
        y = f(t)
        for p in parts(M, min(M, 16)):
            some = q.I8Tokens(t.codes[p], t.scales[p], K)
            assert torch.equal(f(some), y[p])
            if not gated:
                sums = (some.codes.double() @ last.t().contiguous()).float()
                want = (sums * gate.scales[-16:] * some.scales[:, None]).to(y.dtype)
                assert torch.equal(y[p, -16:], want)
        del y


@pytest.mark.parametrize("M,K", [((1 << 21) + 5, 600), ((1 << 21) + 5, 3000), ((1 << 23) + 9, 1)])
def test_rows_of_several_launches(cuda, M, K):
    import torch
    torch.manual_seed(1)
    x, r = (torch.randn(M, K, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w = (1 + 0.1 * torch.randn(K, device="cuda")).to(torch.bfloat16)
    t, h = q.rms_norm_i8(x, w, 1e-5, residual=r)
    s = q.quantize_tokens_i8(x)
    v = q.dequantize_tokens_i8(s)
    for p in parts(M, 9) + [slice((1 << 21) - 4, (1 << 21) + 5)]:
        one, hp = q.rms_norm_i8(x[p], w, 1e-5, residual=r[p])
        assert torch.equal(hp, h[p]) and torch.equal(hp, (x[p].float() + r[p].float()).to(x.dtype))
        assert torch.equal(one.codes, t.codes[p]) and torch.equal(one.scales, t.scales[p])
        one = q.quantize_tokens_i8(x[p])
        assert torch.equal(one.codes, s.codes[p]) and torch.equal(one.scales, s.scales[p])
        assert torch.equal(q.dequantize_tokens_i8(one), v[p])


def test_weight_of_most_rows(cuda):
    import torch
    torch.manual_seed(2)
    N, K = (1 << 23) - 64, 64
    w = torch.randn(N, K, device="cuda")
    iw = q.quantize_i8(w)
    v = q.dequantize_i8(iw)
    for first in (0, N // 32 * 16, N - 48):
        part = q.quantize_i8(w[first:first + 48])
        assert torch.equal(part.tiles, iw.tiles[first // 16:first // 16 + 3])
        assert torch.equal(part.scales, iw.scales[first:first + 48])
        assert torch.equal(q.dequantize_i8(part), v[first:first + 48])


def test_one_weight_twice_and_several_streams(cuda):
    """The same tokens and weights in calls that run together; the two halves
    of a gated call may be one weight."""
    import torch
    torch.manual_seed(3)
    w = q.quantize_i8(torch.randn(5001, 2500, device="cuda") * 0.02)
    x = torch.randn(700, 2500, device="cuda").to(torch.bfloat16)
    t = q.quantize_tokens_i8(x)
    want = q.gated_i8_fwd(w, w, t), q.linear_i8_fwd(w, t), t.codes.clone()
    g = q.linear_i8_fwd(w, t, dtype=torch.float16).double()
    plain = torch.nn.functional.silu(g) * g
    # g's rounding to fp16 (2^-11) in both factors, the slope of silu below 1.13
    off = (want[0].double() - plain).abs()
    assert bool((off <= 2.0 ** -8 * plain.abs() + 2.2 * 2.0 ** -11 * g * g + 1e-6).all())
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for i in range(12):
        with torch.cuda.stream(streams[i % 3]):
            got.append((q.gated_i8_fwd(w, w, t), q.linear_i8_fwd(w, t), q.quantize_tokens_i8(x).codes))
    torch.cuda.synchronize()
    for some in got:
        assert all(torch.equal(a, b) for a, b in zip(some, want))
