"""Sizes at the ends of the 4-bit serving calls' ranges (CPU only: every
refusal comes before a HIP call)."""

import os

import pytest

import bit_quantized_lora_03_amd as q
from tests.test_u4_abi import ESHAPE, at, weight

pytestmark = pytest.mark.skipif(not os.path.exists(q.LIB_PATH), reason="libqlora.so not built")

TB = 1 << 40


@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize_past_a_launch(group):
    """256 threads for 4096 values: 2^36 values are 2^32 threads."""
    f = q.lib().qlora_quantize_u4
    most = ((1 << 24) - 1) * 4096
    for n in (most + group, 1 << 36, 1 << 42, (1 << 62) - 128):
        assert f(TB, n, group, 64 * TB, 96 * TB, None) == ESHAPE, n
    # up to there only the pointers are wrong
    assert f(TB + 4, most, group, 64 * TB, 96 * TB, None) == q.lib().qlora_quantize_u4(
        TB + 4, group, group, 64 * TB, 96 * TB, None)


@pytest.mark.parametrize("tail", ["", "_f16"])
def test_dequantize_past_a_launch(tail):
    """256 threads for 8192 values: 2^37 values are 2^32 threads."""
    f = getattr(q.lib(), "qlora_dequantize_u4" + tail)
    for N, K in ((1 << 17, 1 << 20), ((1 << 28) - 1, 1 << 23), ((1 << 14), 1 << 23),
                 ((1 << 24) - 1, 8192 + 32)):
        w = weight(N=N, K=K, group=32, codes=TB, pairs=64 * TB)
        assert f(w, 96 * TB, None) == ESHAPE, (N, K)
    w = weight(N=(1 << 24) - 1, K=8192, group=32, codes=TB, pairs=64 * TB)
    assert f(w, 96 * TB + 2, None) == -3             # refused for its alignment only


BIG = 1 << 32


def test_batches_past_32_bits_do_not_wrap():
    """Numbers of sequences and widths of the block table that do not fit the
    library's 32 bits are refused, not cut to what they are modulo 2^32."""
    torch = pytest.importorskip("torch")
    from types import SimpleNamespace
    from bit_quantized_lora_03_amd import u4
    pool = SimpleNamespace(index=-1)                 # tensors without memory

    def ints(*shape):
        return torch.empty(shape, dtype=torch.int32, device="meta")

    u4._batch(pool, ints(3), ints(2), ints(2, 5), 1, 2)
    for seqs, width in ((2, BIG), (2, BIG + 5), (2, 1 << 31), (BIG, 1), (BIG + 2, 3), (1 << 31, 1), (0, BIG)):
        with pytest.raises(ValueError):
            u4._batch(pool, ints(seqs + 1), ints(seqs), ints(seqs, width), 1, 2)


def test_rotation_tables_and_heads_past_32_bits_do_not_wrap(monkeypatch):
    torch = pytest.importorskip("torch")
    from types import SimpleNamespace
    from bit_quantized_lora_03_amd import u4
    monkeypatch.setattr(u4, "_dense", lambda *a: None)
    monkeypatch.setattr(u4, "_call", lambda *a: pytest.fail("the library was called"))
    pool = SimpleNamespace(index=-1, kv_heads=2, head_dim=64, now=lambda: None, device="meta")

    def new(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="meta")

    k = new(4, 2, 64)
    batch = (new(2, dtype=torch.int32), new(1, dtype=torch.int32), new(1, 1, dtype=torch.int32), 4)
    with pytest.raises(ValueError):
        u4.kv4_append(pool, k, k, *batch, cos_sin=new(9, BIG + 64, dtype=torch.float32))
    with pytest.raises(ValueError):
        u4.kv4_append(pool, k, k, *batch, q=new(4, BIG + 4, 64))
    with pytest.raises(ValueError):
        u4.kv4_attention(pool, new(4, BIG + 4, 64), *batch, 4)


@pytest.mark.parametrize("name,value", [("q_heads", BIG + 8), ("kv_heads", BIG + 8), ("head_dim", BIG + 64),
                                        ("window", BIG + 10), ("seqs", (1 << 64) + 1),
                                        ("max_q", (1 << 64) + 1), ("max_len", (1 << 64) + (1 << 17))])
def test_workspace_of_sizes_past_32_bits(name, value):
    args = dict(seqs=1, max_q=1, max_len=1 << 17, q_heads=8, kv_heads=8, head_dim=64, window=0)
    assert q.kv4_attention_workspace_bytes(**args) > 0
    with pytest.raises(ValueError):
        q.kv4_attention_workspace_bytes(**(args | {name: value}))
