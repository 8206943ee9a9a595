"""The 4-bit serving calls at the ends of their ranges: offsets past 32 bits in
weights and caches, the most sequences and the most tokens of a call."""

import numpy as np
import pytest

import bit_quantized_lora_03_amd as q
from oracle import u4
from tests.test_gpu_u4 import bits, check_linear, f64, pairs_dev, to_dev

pytestmark = pytest.mark.gpu


def test_quantise_past_32_bits(cuda):
    """2^31 + 2^14 weights: the last groups, and the sums of all codes of a
    weight that repeats."""
    import torch
    N, K, G = (1 << 15) + 1, 1 << 16, 128
    row = torch.randn(1, K, device="cuda")
    w = row.expand(N, K).contiguous()
    w[-1] = torch.randn(K, device="cuda")
    uw = q.quantize_u4(w, G)
    codes, pairs = u4.quantize_weight(row.cpu().numpy(), G)
    assert bool((uw.codes[:-1] == to_dev(codes)).all())
    assert bool((uw.pairs[:-1].view(torch.int16) == pairs_dev(pairs).view(torch.int16)).all())
    codes, pairs = u4.quantize_weight(w[-1:].cpu().numpy(), G)
    assert np.array_equal(uw.codes[-1:].cpu().numpy(), codes)
    assert np.array_equal(bits(uw.pairs[-1:]), pairs)
    del w
    back = q.dequantize_u4(uw)
    assert bool((back[:-1].view(torch.int16) == back[:1].view(torch.int16)).all())
    ref = u4.weight_values(codes, pairs)
    assert np.all(np.abs(f64(back[-1:]) - ref) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(ref))
    x = torch.randn(3, K, device="cuda").to(torch.bfloat16)
    y = q.linear_u4_fwd(uw, x)
    check_linear("last row", y[:, -1:], x, codes, pairs, "bf16")
    assert bool((y[:, :-1].view(torch.int16) == y[:, :1].view(torch.int16)).all())


def test_product_of_the_most_tokens(cuda):
    import torch
    M, N, K = 65535 * 16, 33, 32
    w = torch.randn(N, K, device="cuda")
    uw = q.quantize_u4(w, 32)
    x = torch.randn(64, K, device="cuda").to(torch.bfloat16)
    y = q.linear_u4_fwd(uw, x.repeat(M // 64 + 1, 1)[:M])
    want = q.linear_u4_fwd(uw, x).view(torch.int16)
    assert bool((y[: M // 64 * 64].view(torch.int16).view(-1, 64, N) == want).all())
    assert torch.equal(y[M // 64 * 64:].view(torch.int16), want[: M % 64])
    with pytest.raises(q.QloraError):
        q.linear_u4_fwd(uw, x[:1].expand(M + 1, K).contiguous())


def test_the_most_sequences(cuda):
    """65535 sequences of one token: each gets its own value back."""
    import torch
    B, D = 65535, 64
    cache = q.Kv4Cache.empty(B, 16, 1, D)
    k, v, qq = (torch.randn(B, 1, D, device="cuda").to(torch.bfloat16) for _ in range(3))
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    lens = torch.ones(B, dtype=torch.int32, device="cuda")
    table = torch.randperm(B, device="cuda").to(torch.int32).view(B, 1)
    q.kv4_append(cache, k, v, cu, lens, table, 1)
    rk, rv = q.kv4_read(cache, cu, lens, table, 1, B)
    o, lse = q.kv4_attention(cache, qq, cu, lens, table, 1, 1, return_lse=True)
    # one key: its weight is 1, so o is m + s c but for
    #   both roundings to bf16: 2^-8 of the value each
    #   p s as an fp16 operand, p = 2^(z - M) being no power of two: 2^-11 of
    #   s |c - 8|, which is at most 8 (2 big (1 + 2^-6)) / 15 < 1.1 big
    #   fp32 sums: 2^-21 of s (72 + 15) + |m|, below 2^-14 big
    big = np.abs(f64(v)).max(-1, keepdims=True)
    assert np.all(np.abs(f64(o) - f64(rv)) <= 2.0 ** -7 * np.abs(f64(rv))
                  + (1.1 * 2.0 ** -11 + 2.0 ** -14) * big)
    z = (f64(qq) * f64(rk)).sum(-1) * D ** -0.5
    # rk is rounded to bf16: 2^-8 of each product at most; the score's own sums
    # are far below
    aq = (np.abs(f64(qq) * f64(rk))).sum(-1) * D ** -0.5
    assert np.all(np.abs(f64(lse) - z) <= 2.0 ** -8 * aq + 2.0 ** -10)
    more = torch.zeros(B + 2, dtype=torch.int32, device="cuda")
    with pytest.raises(q.QloraError):
        q.kv4_read(cache, more, more[1:], table.new_zeros(B + 1, 1), 1, 1)


@pytest.mark.parametrize("D,Hkv", [(64, 2), (256, 1)])
def test_cache_past_32_bits(cuda, D, Hkv):
    """A pool of more than 2^32 bytes of keys: sequences in its last pages give
    what the same give in a small pool."""
    import torch
    page, n = 32, 200
    pages = (1 << 32) // (Hkv * page * D // 2) + 40
    used = -(-n // page)
    k, v = (torch.randn(2 * n, Hkv, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    qq = torch.randn(2 * n, 2 * Hkv, D, device="cuda").to(torch.bfloat16)
    i = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    got = []
    for total in (40, pages):
        cache = q.Kv4Cache.empty(total, page, Hkv, D)
        # the last pages, from the last on, and the first ones
        table = torch.stack([total - 1 - torch.arange(used), torch.arange(used)]).to(torch.int32).cuda()
        batch = i([0, n, 2 * n]), i([n, n]), table
        q.kv4_append(cache, k, v, *batch, n)
        got.append((q.kv4_attention(cache, qq, *batch, n, n),) + q.kv4_read(cache, *batch, n, 2 * n))
        del cache
    for a, b in zip(*got):
        assert torch.equal(a, b) and torch.isfinite(a).all()
    torch.cuda.empty_cache()


def test_two_graphs_share_a_workspace(cuda):
    """Attention of two batches, many chunks each, captured with one workspace
    and replayed in turn with eager calls between: each replay writes what it
    reads."""
    import torch
    from tests.test_gpu_kv4 import Pool
    calls, size = [], 0
    for seed, lens, new in ((1, [3000, 700], [1, 2]), (2, [2600, 0, 4500], [1, 1, 1])):
        pool = Pool(lens, 32, 2, 128, seed=seed).fill()
        qq = torch.randn(sum(new), 8, 128, device="cuda").to(torch.bfloat16)
        calls.append((pool.cache(), qq, *pool.ints(new), max(new), max(lens)))
        size = max(size, q.kv4_attention_workspace_bytes(len(lens), max(new), max(lens), 8, 2, 128))
    assert size > 0
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN throughout
    want = [q.kv4_attention(*c) for c in calls]
    torch.cuda.synchronize()
    graphs = []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = q.kv4_attention(*c, workspace=ws)
        graphs.append((g, o))
    for _ in range(3):
        for (g, o), w, c in zip(graphs, want, calls):
            o.fill_(7.0)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, w)
            assert torch.equal(q.kv4_attention(*c, workspace=ws), w)
            ws.fill_(0xFF)
