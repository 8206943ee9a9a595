"""The 8-bit serving calls at the ends of their ranges: weights, tokens and
outputs past 32 bits of address, more rows than one launch has.

Rows are compared bit for bit with the same rows worked out alone: a row's
result does not depend on the others."""

import numpy as np
import pytest

import bit_quantized_lora_03_amd as q
from tests.gpu_util import Guarded  # noqa: F401
from tests.test_gpu_i8 import bits, f64, round16, scaled
from oracle import i8

pytestmark = pytest.mark.gpu


def random_codes(*shape):
    """Codes of any value, made a GiB at a time."""
    import torch
    out = torch.empty(shape, dtype=torch.int8, device="cuda")
    for part in out.view(-1).split(1 << 30):
        part.random_(-127, 128)
    return out


@pytest.mark.parametrize("M", [3, 30, 70])
def test_weight_past_32_bits(cuda, M):
    import torch
    torch.manual_seed(M)
    K = 8192
    N = (1 << 32) // K + 1000
    tiles = random_codes((N + 15) // 16, K // 64, 4, 16, 16)
    iw = q.I8Weight(tiles, torch.rand(N, device="cuda") + 0.5, N, K)
    t = q.quantize_tokens_i8(torch.randn(M, K, device="cuda").to(torch.bfloat16))
    y = q.linear_i8_fwd(iw, t)
    cx, sx = t.codes.cpu().numpy(), t.scales.cpu().numpy()
    for first in (0, (1 << 31) // K // 16 * 16 - 16, (1 << 32) // K // 16 * 16 - 16, N // 16 * 16 - 16):
        n = min(48, N - first)
        part = tiles[first // 16:(first + n + 15) // 16].cpu().numpy()
        cw = part.transpose(0, 3, 1, 2, 4).reshape(-1, K)[:n]
        sw = iw.scales[first:first + n].cpu().numpy()
        assert np.array_equal(bits(y[:, first:first + n]), round16(scaled(i8.sums(cx, cw), sw, sx), "bf16"))
    if M == 3:
        v = q.dequantize_i8(iw)
        for n in (0, N // 2, N - 1):
            c = tiles[n // 16, :, :, n % 16].reshape(-1).cpu().numpy()
            s = iw.scales[n].cpu().numpy()
            assert np.array_equal(bits(v[n]), round16(c.astype(np.float32) * s, "bf16"))


def test_quantizer_past_32_bits(cuda):
    import torch
    torch.manual_seed(0)
    K = 4096
    N = (1 << 32) // K // 4 + 37                       # fp32 rows past 4 GiB
    w = torch.randn(N, K, device="cuda")
    iw = q.quantize_i8(w)
    for first in (0, N // 2 // 16 * 16, (N - 1) // 16 * 16):
        rows = w[first:first + 16].cpu().numpy()
        c, s = i8.encode(rows)
        assert np.array_equal(iw.tiles[first // 16:first // 16 + 1].cpu().numpy(), i8.tile(c))
        assert np.array_equal(iw.scales[first:first + 16].cpu().numpy(), s)


@pytest.mark.parametrize("N", [40, 300])
def test_tokens_past_32_bits(cuda, N):
    import torch
    torch.manual_seed(N)
    K = 8192
    M = (1 << 32) // K + 77
    t = q.I8Tokens(random_codes(M, K), torch.rand(M, device="cuda") + 0.5, K)
    iw = q.quantize_i8(torch.randn(N, K, device="cuda"))
    y = q.linear_i8_fwd(iw, t)
    for first in (0, (1 << 31) // K - 8, (1 << 32) // K - 8, M - 16):
        part = q.I8Tokens(t.codes[first:first + 16], t.scales[first:first + 16], K)
        assert torch.equal(q.linear_i8_fwd(iw, part), y[first:first + 16])
    if N == 40:
        v = q.dequantize_tokens_i8(t)
        part = q.I8Tokens(t.codes[M - 5:], t.scales[M - 5:], K)
        assert torch.equal(q.dequantize_tokens_i8(part), v[M - 5:])


@pytest.mark.parametrize("M,K", [((1 << 32) // 8192 // 2 + 77, 8192), ((1 << 21) + 5, 72)])
def test_norm_and_quantizer_of_many_rows(cuda, M, K):
    """Rows past 4 GiB, and more of them than one launch has."""
    import torch
    torch.manual_seed(1)
    x = torch.randn(M, K, dtype=torch.bfloat16, device="cuda")
    r = torch.randn(M, K, dtype=torch.bfloat16, device="cuda")
    w = (1 + 0.1 * torch.randn(K, device="cuda")).to(torch.bfloat16)
    plain = q.quantize_tokens_i8(x)
    parts = [slice(0, 9), slice(M // 2, M // 2 + 9), slice(min(M - 9, (1 << 21) - 4), min(M, (1 << 21) + 5)),
             slice(M - 9, M)]
    want = [((x[p].float() + r[p].float()).to(x.dtype), x[p].clone()) for p in parts]
    t, h = q.rms_norm_i8(x, w, 1e-5, residual=r, h=r)
    assert h is r
    for p, (s, v) in zip(parts, want):
        assert torch.equal(h[p], s)
        alone, _ = q.rms_norm_i8(s, w, 1e-5)
        assert torch.equal(alone.codes, t.codes[p]) and torch.equal(alone.scales, t.scales[p])
        alone = q.quantize_tokens_i8(v)
        assert torch.equal(alone.codes, plain.codes[p]) and torch.equal(alone.scales, plain.scales[p])


@pytest.mark.parametrize("strided", [False, True])
def test_outputs_past_32_bits(cuda, strided):
    import torch
    torch.manual_seed(2)
    M, N, K = (3000, 100, 256) if strided else (66000, 33000, 128)
    t = q.quantize_tokens_i8(torch.randn(M, K, device="cuda").to(torch.bfloat16))
    gate, up = (q.quantize_i8(torch.randn(N, K, device="cuda")) for _ in range(2))
    wide = torch.full((M, 1 << 20), 7.0, dtype=torch.bfloat16, device="cuda") if strided else None
    y = q.linear_i8_fwd(gate, t, y=wide[:, 8:8 + N] if strided else None)
    for first in (0, M // 2, M - 16):
        part = q.I8Tokens(t.codes[first:first + 16], t.scales[first:first + 16], K)
        assert torch.equal(q.linear_i8_fwd(gate, part), y[first:first + 16])
    if strided:
        assert (wide[:, :8] == 7).all() and (wide[:, 8 + N:] == 7).all()
        return
    del y
    y = q.gated_i8_fwd(gate, up, t)
    for first in (0, M // 2, M - 40):
        part = q.I8Tokens(t.codes[first:first + 40], t.scales[first:first + 40], K)
        assert torch.equal(q.gated_i8_fwd(gate, up, part), y[first:first + 40])


def test_longest_rows(cuda):
    """K = 2^17 - 128 through every call."""
    import torch
    torch.manual_seed(3)
    K = (1 << 17) - 128
    w = torch.randn(30, K, device="cuda")
    iw = q.quantize_i8(w)
    cw, sw = i8.encode(w.cpu().numpy())
    assert np.array_equal(iw.tiles.cpu().numpy(), i8.tile(cw))
    for M in (2, 50, 300):
        x = torch.randn(M, K, device="cuda").to(torch.float16)
        g = (1 + 0.1 * torch.randn(K, device="cuda")).to(torch.float16)
        t, _ = q.rms_norm_i8(x, g, 1e-5)
        c, _ = i8.norm(f64(x), f64(g), 1e-5)
        assert np.array_equal(t.codes.cpu().numpy(), c)
        y = q.linear_i8_fwd(iw, t, dtype=torch.float16)
        assert np.array_equal(bits(y), round16(scaled(i8.sums(c, cw), sw, t.scales.cpu().numpy()), "f16"))


@pytest.mark.parametrize("M,N", [(60, 4096), (60, 8191), (40, 11000), (150, 8192), (701, 4099), (2000, 8192)])
def test_longest_rows_in_every_tile(cuda, M, N):
    """K = 2^17 - 128 against enough rows for the larger tiles, 32 x 32 to 128 x
    256: codes of all values, and -128 throughout, whose sums are 2^31 - 2^21."""
    import torch
    torch.manual_seed(M)
    K = (1 << 17) - 128
    tiles, codes = random_codes((N + 15) // 16, K // 64, 4, 16, 16), random_codes(M, K)
    w = q.I8Weight(tiles, torch.rand(N, device="cuda") + 0.5, N, K)
    t = q.I8Tokens(codes, torch.rand(M, device="cuda") + 0.5, K)
    y = q.linear_i8_fwd(w, t)
    rows = [0, 1, M // 2, M - 1]
    cx, sx = codes[rows].cpu().numpy(), t.scales[rows].cpu().numpy()
    for first in (0, N // 32 * 16, (N - 1) // 16 * 16):
        n = min(16, N - first)
        cw = tiles[first // 16].cpu().numpy().transpose(2, 0, 1, 3).reshape(16, K)[:n]
        sw = w.scales[first:first + n].cpu().numpy()
        want = round16(scaled(i8.sums(cx, cw), sw, sx), "bf16")
        assert np.array_equal(bits(y[rows][:, first:first + n]), want)
    tiles.fill_(-128)
    codes.fill_(-128)
    w.scales.fill_(0.5)
    t.scales.fill_(1.0)
    assert (q.linear_i8_fwd(w, t) == float(np.float32(K << 14)) * 0.5).all()
