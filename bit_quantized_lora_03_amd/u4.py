"""Torch-facing calls of the 4-bit group format and the 4-bit paged cache
(``qlora_*_u4*`` and ``qlora_kv4_*`` of include/qlora.h).

As in the rest of the binding these only check and marshal arguments; the
arithmetic is the library's.  Work goes to the current stream of the device
that the tensors are on.  Arguments that do not fit raise ``ValueError``
before the library is called; what the library itself refuses raises
:class:`QloraError`.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import Kv4BatchStruct, Kv4CacheStruct, QloraError, U4Struct, check

GROUPS = (32, 64, 128)
HEAD_DIMS = (64, 128, 256)
_16BIT = {torch.bfloat16: "", torch.float16: "_f16"}
_u8, _i32, _f32, _bf16 = torch.uint8, torch.int32, torch.float32, torch.bfloat16


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _dense(t, name: str, dtype, device=None) -> None:
    if t.dtype is not dtype:
        raise ValueError(f"{name}: {dtype} expected, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: a tensor on the GPU is needed")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, the others on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: has to be contiguous")


class _On:
    """Makes ``device`` the current one for a call if it is not already, and
    gives the raw handle of its current stream."""
    __slots__ = ("index", "was")

    def __init__(self, device):
        self.index = device.index

    def __enter__(self):
        self.was = torch.cuda.current_device()
        if self.index != self.was:
            torch.cuda.set_device(self.index)
        return torch._C._cuda_getCurrentRawStream(self.index)

    def __exit__(self, *exc):
        if self.index != self.was:
            torch.cuda.set_device(self.was)


# ---------------------------------------------------------------------------
# weights
# ---------------------------------------------------------------------------

class U4Weight:
    """A weight [N, K] in the 4-bit group format: ``codes`` uint8 [N, K/2]
    (even element in the low nibble) and ``pairs`` bf16 [N, K/group, 2] (s
    and m; a value is m + s * code)."""

    __slots__ = ("codes", "pairs", "N", "K", "group", "device", "struct")

    def __init__(self, codes, pairs):
        _dense(codes, "codes", _u8)
        _dense(pairs, "pairs", _bf16, codes.device)
        _need(codes.dim() == 2 and pairs.dim() == 3 and pairs.shape[0] == codes.shape[0]
              and pairs.shape[2] == 2 and pairs.shape[1] > 0,
              "codes [N, K/2] and pairs [N, K/group, 2] are needed")
        self.N, half = codes.shape
        self.K, self.group = 2 * half, 2 * half // pairs.shape[1]
        _need(self.group in GROUPS and self.group * pairs.shape[1] == self.K,
              f"groups of {GROUPS} values are supported")
        self.codes, self.pairs, self.device = codes, pairs, codes.device
        self.struct = U4Struct(codes.data_ptr(), pairs.data_ptr(), self.N, self.K, self.group)


def quantize_u4(w, group: int = 64) -> U4Weight:
    """fp32 [N, K] device weight -> U4Weight with groups of ``group`` (32, 64
    or 128) along K."""
    _need(w.dim() == 2 and w.dtype is _f32 and w.is_cuda, "an fp32 [N, K] tensor on the GPU is needed")
    _need(group in GROUPS, f"groups of {GROUPS} values are supported")
    N, K = w.shape
    _need(N > 0 and K > 0 and K % group == 0, f"K = {K} is not a positive multiple of {group}")
    w = w.contiguous()
    codes = torch.empty((N, K // 2), dtype=_u8, device=w.device)
    pairs = torch.empty((N, K // group, 2), dtype=_bf16, device=w.device)
    with _On(w.device) as s:
        check(_lib.lib().qlora_quantize_u4(w.data_ptr(), N * K, group, codes.data_ptr(),
                                           pairs.data_ptr(), s), "qlora_quantize_u4")
    return U4Weight(codes, pairs)


def dequantize_u4(uw: U4Weight, dtype=torch.bfloat16):
    """U4Weight -> its values [N, K] in bf16 or fp16."""
    _need(dtype in _16BIT, "bf16 or fp16 values")
    out = torch.empty((uw.N, uw.K), dtype=dtype, device=uw.device)
    name = "qlora_dequantize_u4" + _16BIT[dtype]
    with _On(uw.device) as s:
        check(getattr(_lib.lib(), name)(ctypes.byref(uw.struct), out.data_ptr(), s), name)
    return out


def linear_u4_fwd(uw: U4Weight, x, y=None):
    """y = x . W^T for few tokens: x [M, K] bf16 or fp16 (rows may be
    strided), y [M, N] of the same type (rows may be strided)."""
    tail = _16BIT.get(x.dtype)
    _need(tail is not None, "x has to be bf16 or fp16")
    _need(x.dim() == 2 and x.shape[1] == uw.K and x.device == uw.device and x.stride(1) == 1,
          f"x: [M, {uw.K}] on {uw.device} with unit stride along K is needed")
    M = x.shape[0]
    if y is None:
        y = torch.empty((M, uw.N), dtype=x.dtype, device=uw.device)
        ldy = uw.N
    else:
        _need(y.dtype is x.dtype and tuple(y.shape) == (M, uw.N) and y.device == uw.device
              and (y.stride(1) == 1 or uw.N == 1),
              f"y: [{M}, {uw.N}] like x, with unit stride along N, is needed")
        ldy = y.stride(0) if M > 1 else max(uw.N, y.stride(0))
    ldx = x.stride(0) if M > 1 else uw.K
    lib = _lib.lib()
    f = lib.qlora_linear_u4_fwd_f16 if tail else lib.qlora_linear_u4_fwd
    with _On(uw.device) as s:
        st = f(uw.struct, x.data_ptr(), ldx, M, y.data_ptr(), ldy, s)
    if st:
        raise QloraError(st, "qlora_linear_u4_fwd" + tail)
    return y


# ---------------------------------------------------------------------------
# the paged cache
# ---------------------------------------------------------------------------

class Kv4Cache:
    """Keys and values in the 4-bit group format, in pages: codes uint8
    [pages, kv_heads, page_size, head_dim / 2] and pairs bf16 [pages,
    kv_heads, page_size, 2], one pair per token and head."""

    __slots__ = ("k_codes", "k_pairs", "v_codes", "v_pairs", "pages", "kv_heads", "page_size",
                 "head_dim", "device", "struct")

    def __init__(self, k_codes, k_pairs, v_codes, v_pairs):
        self.device = k_codes.device
        for t, n, dt in ((k_codes, "k_codes", _u8), (k_pairs, "k_pairs", _bf16),
                         (v_codes, "v_codes", _u8), (v_pairs, "v_pairs", _bf16)):
            _dense(t, n, dt, self.device)
        _need(k_codes.dim() == 4, "codes [pages, kv_heads, page_size, head_dim / 2] are needed")
        self.pages, self.kv_heads, self.page_size, half = k_codes.shape
        self.head_dim = 2 * half
        pair = (self.pages, self.kv_heads, self.page_size, 2)
        _need(v_codes.shape == k_codes.shape and tuple(k_pairs.shape) == pair
              and tuple(v_pairs.shape) == pair, "codes and pairs of one cache differ in shape")
        _need(self.head_dim in HEAD_DIMS, f"head_dim {self.head_dim}: {HEAD_DIMS} are supported")
        _need(16 <= self.page_size <= 1024 and self.page_size & (self.page_size - 1) == 0,
              f"page_size {self.page_size}: a power of two from 16 to 1024 is needed")
        self.k_codes, self.k_pairs, self.v_codes, self.v_pairs = k_codes, k_pairs, v_codes, v_pairs
        self.struct = Kv4CacheStruct(k_codes.data_ptr(), k_pairs.data_ptr(), v_codes.data_ptr(),
                                     v_pairs.data_ptr(), self.pages, self.page_size,
                                     self.kv_heads, self.head_dim)

    @classmethod
    def empty(cls, pages: int, page_size: int, kv_heads: int, head_dim: int, device="cuda"):
        """A pool of ``pages`` pages, uninitialised."""
        def new(n, dt):
            return torch.empty((pages, kv_heads, page_size, n), dtype=dt, device=device)
        return cls(new(head_dim // 2, _u8), new(2, _bf16), new(head_dim // 2, _u8), new(2, _bf16))


def _batch(cache: Kv4Cache, cu_q, seq_lens, block_table, max_q: int, rows: int) -> Kv4BatchStruct:
    for t, n in ((cu_q, "cu_q"), (seq_lens, "seq_lens"), (block_table, "block_table")):
        if t.dtype is not _i32 or t.device != cache.device or not t.is_contiguous():
            raise ValueError(f"{n}: a contiguous int32 tensor on {cache.device} is needed")
    B = seq_lens.shape[0]
    if cu_q.dim() != 1 or cu_q.shape[0] != B + 1 or seq_lens.dim() != 1 or \
            block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("cu_q [B + 1], seq_lens [B] and block_table [B, width] are needed")
    if max_q < 0:
        raise ValueError("max_q is negative")
    return Kv4BatchStruct(cu_q.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(), rows, B,
                          block_table.shape[1], max_q)


def _rows(cache: Kv4Cache, t, name: str, dtype, rows: Optional[int], heads: Optional[int]):
    """Checks a [T, heads, head_dim] tensor; returns its (token, head) strides."""
    if t.dim() != 3 or t.shape[2] != cache.head_dim or t.dtype is not dtype or \
            t.device != cache.device or (rows is not None and t.shape[0] != rows) or \
            (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name}: [{'T' if rows is None else rows}, "
                         f"{'heads' if heads is None else heads}, {cache.head_dim}] of {dtype} on "
                         f"{cache.device} is needed, got {tuple(t.shape)} of {t.dtype} on {t.device}")
    ts, hs, ds = t.stride()
    if ds != 1:
        raise ValueError(f"{name}: unit stride along head_dim is needed")
    # the stride of an axis of length one says nothing
    return (ts if t.shape[0] > 1 else 0), (hs if t.shape[1] > 1 else 0)


def kv4_append(cache: Kv4Cache, k, v, cu_q, seq_lens, block_table, max_q: int, q=None,
               cos_sin=None, interleaved: bool = False, q_out=None):
    """Appends k, v [T, kv_heads, head_dim] (bf16 or fp16, strided rows
    allowed) to the cache, keys rotated by ``cos_sin`` fp32 [positions, rot]
    (cosines, then sines); returns the rotated queries [T, q_heads, head_dim]
    where ``q`` is given, else None.

    Rows cu_q[b] .. cu_q[b + 1] - 1 are the last tokens of sequence b, whose
    length with them is seq_lens[b]; block_table [B, width] names its pages;
    no sequence has more than ``max_q`` rows."""
    dt = k.dtype
    tail = _16BIT.get(dt)
    _need(tail is not None, "k, v and q have to be bf16 or fp16")
    T = k.shape[0] if k.dim() else 0
    kts, khs = _rows(cache, k, "k", dt, None, cache.kv_heads)
    vts, vhs = _rows(cache, v, "v", dt, T, cache.kv_heads)
    qp = op = None
    qts = qhs = heads = 0
    if q is not None:
        qts, qhs = _rows(cache, q, "q", dt, T, None)
        heads = q.shape[1]
        if q_out is None:
            q_out = torch.empty((T, heads, cache.head_dim), dtype=dt, device=cache.device)
        else:
            _need(q_out.shape == q.shape and q_out.dtype is dt and q_out.device == cache.device
                  and q_out.is_contiguous(), "q_out has to be contiguous and like q")
        qp, op = q.data_ptr(), q_out.data_ptr()
    else:
        _need(q_out is None, "q_out without q")
    rot = rows = 0
    tp = None
    if cos_sin is not None:
        _need(cos_sin.dim() == 2, "cos_sin: [positions, rot] is needed")
        _dense(cos_sin, "cos_sin", _f32, cache.device)
        rows, rot = cos_sin.shape
        tp = cos_sin.data_ptr()
    bt = _batch(cache, cu_q, seq_lens, block_table, max_q, T)
    lib = _lib.lib()
    f = lib.qlora_kv4_append_f16 if tail else lib.qlora_kv4_append
    with _On(cache.device) as s:
        st = f(cache.struct, bt, k.data_ptr(), kts, khs, v.data_ptr(), vts, vhs, qp, qts, qhs,
               heads, tp, rows, rot, 1 if interleaved else 0, op, s)
    if st:
        raise QloraError(st, "qlora_kv4_append" + tail)
    return q_out


def kv4_read(cache: Kv4Cache, cu_q, seq_lens, block_table, max_q: int, rows: int,
             dtype=torch.bfloat16) -> Tuple[object, object]:
    """The keys and values that the cache holds for the batch's ``rows`` rows,
    [rows, kv_heads, head_dim] each, in bf16 or fp16; rows behind
    cu_q[-1] are uninitialised."""
    tail = _16BIT.get(dtype)
    _need(tail is not None, "bf16 or fp16 values")
    _need(rows >= 0, "rows is negative")
    bt = _batch(cache, cu_q, seq_lens, block_table, max_q, rows)
    shape = (rows, cache.kv_heads, cache.head_dim)
    k = torch.empty(shape, dtype=dtype, device=cache.device)
    v = torch.empty(shape, dtype=dtype, device=cache.device)
    lib = _lib.lib()
    f = lib.qlora_kv4_read_f16 if tail else lib.qlora_kv4_read
    with _On(cache.device) as s:
        st = f(cache.struct, bt, k.data_ptr(), v.data_ptr(), s)
    if st:
        raise QloraError(st, "qlora_kv4_read" + tail)
    return k, v


def kv4_attention_workspace_bytes(seqs: int, max_q: int, max_len: int, q_heads: int,
                                  kv_heads: int, head_dim: int, window: int = 0) -> int:
    return int(_lib.lib().qlora_kv4_attention_workspace_bytes(seqs, max_q, max_len, q_heads,
                                                              kv_heads, head_dim, window))


def kv4_attention(cache: Kv4Cache, q, cu_q, seq_lens, block_table, max_q: int, max_len: int,
                  scale: Optional[float] = None, causal: bool = True, window: int = 0, out=None,
                  return_lse: bool = False, lse=None, workspace=None):
    """Attention of the batch's rows q [T, q_heads, head_dim] over the cache
    (after :func:`kv4_append` of the same batch); returns out, or (out, lse)
    with ``return_lse``.  ``scale`` defaults to head_dim ** -0.5; no sequence
    is longer than ``max_len``; a row at position p sees keys up to p
    (``causal``) and after p - window (``window`` > 0)."""
    dt = q.dtype
    tail = _16BIT.get(dt)
    _need(tail is not None, "q has to be bf16 or fp16")
    qts, qhs = _rows(cache, q, "q", dt, None, None)
    T, heads, D = q.shape
    bt = _batch(cache, cu_q, seq_lens, block_table, max_q, T)
    if out is None:
        out = torch.empty((T, heads, D), dtype=dt, device=cache.device)
    else:
        _need(out.shape == q.shape and out.dtype is dt and out.device == cache.device
              and out.is_contiguous(), "out has to be contiguous and like q")
    if lse is not None:
        _need(tuple(lse.shape) == (T, heads) and lse.dtype is _f32 and lse.is_contiguous()
              and lse.device == cache.device, f"lse: fp32 [{T}, {heads}] is needed")
    elif return_lse:
        lse = torch.empty((T, heads), dtype=_f32, device=cache.device)
    lib = _lib.lib()
    need = lib.qlora_kv4_attention_workspace_bytes(bt.seqs, max_q, max_len, heads, cache.kv_heads,
                                                   D, window)
    if workspace is None:
        if need:
            workspace = torch.empty(need, dtype=_u8, device=cache.device)
    else:
        _dense(workspace, "workspace", _u8, cache.device)
        need = workspace.numel()
    f = lib.qlora_kv4_attention_f16 if tail else lib.qlora_kv4_attention
    with _On(cache.device) as s:
        st = f(cache.struct, bt, q.data_ptr(), qts, qhs, heads,
               D ** -0.5 if scale is None else scale, 1 if causal else 0, window, max_len,
               out.data_ptr(), None if lse is None else lse.data_ptr(),
               None if workspace is None else workspace.data_ptr(), need, s)
    if st:
        raise QloraError(st, "qlora_kv4_attention" + tail)
    return (out, lse) if return_lse else out
