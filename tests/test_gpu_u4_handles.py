"""A 4-bit weight whose tensors were exchanged, and a cache that was moved,
through the calls."""

import pytest

import bit_quantized_lora_03_amd as q

pytestmark = pytest.mark.gpu


def test_calls_follow_the_tensors(cuda):
    import torch
    a, b = (q.quantize_u4(torch.randn(96, 128, device="cuda")) for _ in range(2))
    c = q.quantize_u4(torch.randn(32, 256, device="cuda"), 128)
    x, x2 = (torch.randn(3, k, device="cuda").to(torch.bfloat16) for k in (128, 256))
    want = q.linear_u4_fwd(b, x), q.dequantize_u4(b), q.linear_u4_fwd(c, x2)
    a.codes, a.pairs = b.codes, b.pairs
    assert torch.equal(q.linear_u4_fwd(a, x), want[0])
    a.codes.data, a.pairs.data = a.codes.clone(), a.pairs.clone()
    assert torch.equal(q.dequantize_u4(a), want[1])
    a.codes, a.pairs = c.codes, c.pairs
    assert torch.equal(q.linear_u4_fwd(a, x2), want[2])
    with pytest.raises(ValueError):
        q.linear_u4_fwd(a, x)
    a.codes = c.codes.cpu()
    with pytest.raises(ValueError):
        q.linear_u4_fwd(a, x2)


def test_a_cache_that_was_moved(cuda):
    import torch
    i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = q.Kv4Cache.empty(3, 16, 2, 64)
    k, v = (torch.randn(20, 2, 64, device="cuda").to(torch.bfloat16) for _ in range(2))
    qq = torch.randn(20, 4, 64, device="cuda").to(torch.bfloat16)
    batch = i([0, 20]), i([20]), i([[2, 0]])
    q.kv4_append(cache, k, v, *batch, 20)
    want, read = q.kv4_attention(cache, qq, *batch, 20, 20), q.kv4_read(cache, *batch, 20, 20)
    old = [getattr(cache, n) for n in ("k_codes", "k_pairs", "v_codes", "v_pairs")]
    for n in ("k_codes", "k_pairs", "v_codes", "v_pairs"):
        setattr(cache, n, getattr(cache, n).clone())
    for t in old:
        t.zero_()
    assert torch.equal(q.kv4_attention(cache, qq, *batch, 20, 20), want)
    for x, y in zip(q.kv4_read(cache, *batch, 20, 20), read):
        assert torch.equal(x, y)
    q.kv4_append(cache, k, v, *batch, 20)
    assert not any(t.any() for t in old)             # nothing written where it was
