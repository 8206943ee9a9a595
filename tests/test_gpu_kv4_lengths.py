"""Lengths far past the block table: the tokens that are not there are not
attended to, whatever the window leaves."""

import numpy as np
import pytest

import bit_quantized_lora_03_amd as q
from tests.gpu_util import Guarded
from tests.test_gpu_kv4 import Pool
from tests.test_gpu_u4 import to_dev

pytestmark = pytest.mark.gpu

TOP = 2 ** 31 - 1


def run(cache, qq, lens, table, new, window, max_len, causal=True):
    import torch
    cu = to_dev(np.concatenate([[0], np.cumsum(new)]).astype(np.int32))
    out, lse = Guarded(qq.shape, qq.dtype), Guarded(qq.shape[:2], torch.float32)
    q.kv4_attention(cache, qq, cu, to_dev(np.array(lens, np.int32)), table, max(new), max_len,
                    window=window, causal=causal, out=out.t, lse=lse.t)
    out.check("out")
    lse.check("lse")
    return out.t, lse.t


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("length", [TOP, TOP - 31, TOP - 300, 2 ** 30 + 17, 2 ** 30])
@pytest.mark.parametrize("max_len", [48, 2 ** 20, 2 ** 30])
def test_window_behind_the_table(cuda, D, length, max_len):
    import torch
    pool = Pool([48, 33, 48], 16, 2, D, seed=D).fill()
    cache, table, new = pool.cache(), to_dev(pool.table), [1, 1, 3]
    qq = torch.randn(5, 4, D, device="cuda").to(torch.bfloat16)
    for window in (1, 40, 4096):
        out, lse = run(cache, qq, [length, 33, length], table, new, window, max_len)
        for rows in (slice(0, 1), slice(2, 5)):
            assert (out[rows] == 0).all() and (lse[rows] == -float("inf")).all()
        want, wl = run(cache, qq, [0, 33, 0], table, new, window, max_len)
        assert torch.equal(out[1], want[1]) and torch.equal(lse[1], wl[1])


@pytest.mark.parametrize("causal", [True, False])
def test_all_of_the_table_of_a_longer_sequence(cuda, causal):
    """Without a window, or with one that reaches back to token 1."""
    import torch
    pool = Pool([48, 33], 16, 2, 128, seed=3).fill()
    cache, table = pool.cache(), to_dev(pool.table)
    qq = torch.randn(2, 4, 128, device="cuda").to(torch.bfloat16)
    for length, window, same in ((TOP, 0, 0), (2 ** 30 + 5, 0, 0), (TOP, TOP - 1, 47)):
        out, lse = run(cache, qq, [length, 33], table, [1, 1], window, 100, causal)
        want, wl = run(cache, qq, [48, 33], table, [1, 1], same, 100, causal)
        assert torch.equal(out[0], want[0]) and torch.equal(lse[0], wl[0]), (length, window)


@pytest.mark.parametrize("cu", [[TOP, 0, 0], [0, TOP, -TOP - 1], [-TOP - 1, TOP, 3], [5, 2, 0],
                                [TOP - 8, -TOP - 1, TOP], [5, 9, 5]])
@pytest.mark.parametrize("Hq,Hkv", [(16, 2), (8, 1), (3, 1)])
def test_rows_that_do_not_ascend(cuda, cu, Hq, Hkv):
    """Nothing outside the call's rows is read or written, and rows that no
    sequence has stay as they were."""
    import torch
    D, T = 64, 5
    pool = Pool([48, 48], 16, Hkv, D, seed=7).fill()
    cache, table = pool.cache(), to_dev(pool.table)
    qq, k = (torch.randn(T, h, D, device="cuda").to(torch.bfloat16) for h in (Hq, Hkv))
    out, lse = Guarded(qq.shape, qq.dtype), Guarded(qq.shape[:2], torch.float32)
    before = out.t.clone().view(torch.int16)
    batch = to_dev(np.array(cu, np.int32)), to_dev(np.array([48, 48], np.int32)), table
    for max_len in (48, 1 << 16):
        q.kv4_attention(cache, qq, *batch, 4, max_len, out=out.t, lse=lse.t)
    out.check("out")
    lse.check("lse")
    mine = np.zeros(T, bool)
    for a, b in zip(cu, cu[1:]):
        if a >= 0:
            mine[a:min(max(b, a), T, a + 4)] = True
    same = (out.t.view(torch.int16) == before).all(-1).all(-1).cpu().numpy()
    assert np.array_equal(same, ~mine)
    q.kv4_append(cache, k, k, *batch, 4, q=qq, q_out=out.t)
    q.kv4_read(cache, *batch, 4, T)
    out.check("q_out")
