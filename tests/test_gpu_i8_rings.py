"""The 8-bit products in large tiles where K has many tiles: the ring of token
stages goes round, stages are filled again and the steady wait is what keeps
them apart.

Every output is compared bit for bit with the small tiles' (tokens sixteen at a
time, a kernel of its own that has no ring), and those of some tokens with the
oracle: the plain product bit for bit, the gated one within the bar that
``test_gpu_i8`` derives."""

import numpy as np
import pytest

import bit_quantized_lora_03_amd as q
from oracle import i8
from tests.test_gpu_i8 import U16, bits, f64, gated_ref, round16, scaled, tdtype
from tests.test_gpu_i8_extremes import random_codes

pytestmark = pytest.mark.gpu

LONGEST = (1 << 17) - 128

# 32 x 128, 64 x 128, 128 x 128, with odd and even numbers of K's tiles
GATED = [(61, 11008, 4096), (40, 11000, 4200), (128, 11008, 4097), (300, 11008, 2500),
         (1025, 4100, 2100), (2047, 5001, 2500)]
# these and 128 x 256
PLAIN = [(61, 11008, 4096), (40, 11000, 4200), (501, 4096, 4096), (501, 4091, 4200),
         (701, 4099, 2100), (2047, 5001, 2500), (1000, 8192, 2100), (2000, 8192, 2048)]
# the same tiles of the gated product, at the longest rows
GATED_LONGEST = [(40, 11000), (150, 8192), (701, 4099)]


def tokens(M, K):
    import torch
    codes = random_codes(M, i8.padded(K))
    codes[:, K:] = 0
    return q.I8Tokens(codes, torch.rand(M, device="cuda") + 0.5, K)


def weight(N, K):
    """Random codes of all values, with scales that make products of a few
    units (a code's root-mean-square is 73), and the codes in rows."""
    import torch
    Kp, P = i8.padded(K), -(-N // 16)
    rows = random_codes(16 * P, Kp)
    rows[:, K:] = 0
    tiles = rows.view(P, 16, Kp // 64, 4, 16).permute(0, 2, 3, 1, 4).contiguous()
    scales = (torch.rand(N, device="cuda") + 0.5) * (2 / 73 ** 2 / K ** 0.5)
    return q.I8Weight(tiles, scales, N, K), rows[:N, :K]


def some(M):
    """Tokens at the tiles' and the instructions' edges."""
    return sorted({m for m in (0, 1, 15, 16, 31, 32, 63, 64, 127, 128, M // 2, M - 1) if m < M})


def sixteen(f, t):
    """f over sixteen tokens at a time."""
    import torch
    return torch.cat([f(q.I8Tokens(c, s, t.K))
                      for c, s in zip(t.codes.split(16), t.scales.split(16))])


@pytest.mark.parametrize("M,N,K", PLAIN)
def test_product(cuda, M, N, K):
    import torch
    torch.manual_seed(M)
    (w, cw), t = weight(N, K), tokens(M, K)
    rows = some(M)
    sums = i8.sums(t.codes[rows, :K].cpu().numpy(), cw.cpu().numpy())
    want = scaled(sums, w.scales.cpu().numpy(), t.scales[rows].cpu().numpy())
    for dtype in ("bf16", "f16"):
        y = q.linear_i8_fwd(w, t, dtype=tdtype(dtype))
        assert np.array_equal(bits(y[rows]), round16(want, dtype))
        assert torch.equal(y, sixteen(lambda x: q.linear_i8_fwd(w, x, dtype=tdtype(dtype)), t))
        for _ in range(4):
            assert torch.equal(q.linear_i8_fwd(w, t, dtype=tdtype(dtype)), y)


@pytest.mark.parametrize("M,N,K", GATED)
def test_gated(cuda, M, N, K):
    import torch
    torch.manual_seed(M)
    (gate, cg), (up, cu), t = weight(N, K), weight(N, K), tokens(M, K)
    rows = some(M)
    cx, sx = t.codes[rows, :K].cpu().numpy(), t.scales[rows].cpu().numpy()
    sg, su = gate.scales.cpu().numpy(), up.scales.cpu().numpy()
    cg, cu = cg.cpu().numpy(), cu.cpu().numpy()
    for act in ("silu", "gelu"):
        ref, bar = gated_ref(cx, sx, cg, sg, cu, su, act)
        # a product of the wrong weights, or of none, is no answer
        other, _ = gated_ref(cx, sx, cu, su, cg, sg, act)
        for dtype in ("bf16", "f16"):
            f = lambda x: q.gated_i8_fwd(gate, up, x, act=act, dtype=tdtype(dtype))  # noqa: E731
            y = f(t)
            within = U16[dtype] * (np.abs(ref) + bar) + bar + 2.0 ** -25
            assert np.all(np.abs(f64(y[rows]) - ref) <= within)
            assert not np.any(np.all(np.abs(other - ref) <= within, -1))
            assert not np.any(np.all(np.abs(ref) <= within, -1))
            assert torch.equal(y, sixteen(f, t))
            for _ in range(4):
                assert torch.equal(f(t), y)


@pytest.mark.parametrize("M,N", GATED_LONGEST)
def test_gated_longest_rows(cuda, M, N):
    """K = 2^17 - 128: codes of all values, and those at the ends of their
    range throughout, whose sums are 2^31 - 2^21 and -2^31 + 2^24 + 2^21 - 2^14."""
    import torch
    torch.manual_seed(M)
    K = LONGEST
    t = tokens(M, K)
    gate, up = (q.I8Weight(random_codes((N + 15) // 16, K // 64, 4, 16, 16),
                           (torch.rand(N, device="cuda") + 0.5) * (2 / 73 ** 2 / K ** 0.5), N, K)
                for _ in range(2))
    y = {act: q.gated_i8_fwd(gate, up, t, act=act) for act in ("silu", "gelu")}
    rows = some(M)
    cx, sx = t.codes[rows].cpu().numpy(), t.scales[rows].cpu().numpy()
    for first in (0, N // 32 * 16, (N - 1) // 16 * 16):
        n = min(16, N - first)
        cg, cu = (w.tiles[first // 16].cpu().numpy().transpose(2, 0, 1, 3).reshape(16, K)[:n]
                  for w in (gate, up))
        sg, su = (w.scales[first:first + n].cpu().numpy() for w in (gate, up))
        for act, out in y.items():
            ref, bar = gated_ref(cx, sx, cg, sg, cu, su, act)
            off = np.abs(f64(out[rows][:, first:first + n]) - ref)
            assert np.all(off <= U16["bf16"] * (np.abs(ref) + bar) + bar + 2.0 ** -25)
    gate.tiles.fill_(-128)
    up.tiles.fill_(127)
    t.codes.fill_(-128)
    t.scales.fill_(1.0)
    gate.scales.fill_(2.0 ** -30)
    up.scales.fill_(2.0 ** -30)
    assert 128 * 128 * K == 2 ** 31 - 2 ** 21
    assert -128 * 127 * K == -2 ** 31 + 2 ** 24 + 2 ** 21 - 2 ** 14
    one = np.ones((1, 1))
    for act in y:
        ref, bar = gated_ref(-128 * one, one[0], -128 * one, one[0] * K * 2.0 ** -30, 127 * one,
                             one[0] * K * 2.0 ** -30, act)
        out = q.gated_i8_fwd(gate, up, t, act=act)
        assert (out == out[0, 0]).all()
        off = np.abs(f64(out[0, 0]) - ref)
        assert np.all(off <= U16["bf16"] * (np.abs(ref) + bar) + bar)
