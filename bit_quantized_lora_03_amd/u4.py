"""Torch-facing calls of the 4-bit group format and the 4-bit paged cache
(``qlora_*_u4*`` and ``qlora_kv4_*`` of include/qlora.h).

As in the rest of the binding these only check and marshal arguments; the
arithmetic is the library's.  Work goes to the current stream of the device
that the tensors are on.  Arguments that do not fit raise ``ValueError``
before the library is called; what the library itself refuses raises
:class:`QloraError`.
"""

from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _lib
from ._lib import Kv4BatchStruct, Kv4CacheStruct, QloraError, U4Struct

GROUPS = (32, 64, 128)
HEAD_DIMS = (64, 128, 256)
_16BIT = {torch.bfloat16: "", torch.float16: "_f16"}
_u8, _i32, _f32, _bf16 = torch.uint8, torch.int32, torch.float32, torch.bfloat16
_current = torch._C._cuda_getDevice
_stream = torch._C._cuda_getCurrentRawStream
_entry = {}
_I32 = 2 ** 31  # ctypes would cut larger ones to their low bits


def _call(name: str, dtype, index: int, *args) -> None:
    """Calls the entry point (its fp16 form where ``dtype`` is fp16) with
    ``args`` and the current stream of GPU ``index``, which is the current
    device meanwhile."""
    f = _entry.get((name, dtype))
    if f is None:
        f = _entry[name, dtype] = getattr(_lib.lib(), name + _16BIT.get(dtype, ""))
    if _current() == index:
        st = f(*args, _stream(index))
    else:
        with torch.cuda.device(index):
            st = f(*args, _stream(index))
    if st:
        raise QloraError(st, name + _16BIT.get(dtype, ""))


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _dense(t, name: str, dtype, index: int = -1) -> None:
    at = t.get_device()
    if t.dtype is not dtype:
        raise ValueError(f"{name}: {dtype} expected, got {t.dtype}")
    if at < 0:
        raise ValueError(f"{name}: a tensor on the GPU is needed")
    if index >= 0 and at != index:
        raise ValueError(f"{name}: on {t.device}, the others on GPU {index}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: has to be contiguous")


# ---------------------------------------------------------------------------
# weights
# ---------------------------------------------------------------------------

class U4Weight:
    """A weight [N, K] in the 4-bit group format: ``codes`` uint8 [N, K/2]
    (even element in the low nibble) and ``pairs`` bf16 [N, K/group, 2] (s
    and m; a value is m + s * code)."""

    __slots__ = ("codes", "pairs", "N", "K", "group", "index", "struct", "at")

    def __init__(self, codes, pairs):
        _dense(codes, "codes", _u8)
        index = codes.get_device()
        _dense(pairs, "pairs", _bf16, index)
        cs, ps = codes.shape, pairs.shape
        if len(cs) != 2 or len(ps) != 3 or ps[0] != cs[0] or ps[2] != 2 or ps[1] == 0:
            raise ValueError("codes [N, K/2] and pairs [N, K/group, 2] are needed")
        N, K = cs[0], 2 * cs[1]
        group = K // ps[1]
        if group not in GROUPS or group * ps[1] != K:
            raise ValueError(f"groups of {GROUPS} values are supported")
        self.codes, self.pairs, self.index = codes, pairs, index
        self.N, self.K, self.group = N, K, group
        c, p = codes.data_ptr(), pairs.data_ptr()
        self.at = codes, c, pairs, p
        self.struct = U4Struct(c, p, N, K, group)

    def now(self) -> U4Struct:
        """The descriptor of the tensors as they are: checked and written anew
        where one was exchanged or has other memory since."""
        codes, c, pairs, p = self.at
        if self.codes is not codes or self.pairs is not pairs or codes.data_ptr() != c or \
                pairs.data_ptr() != p:
            self.__init__(self.codes, self.pairs)
        return self.struct

    @property
    def device(self):
        return self.codes.device


def quantize_u4(w, group: int = 64) -> U4Weight:
    """fp32 [N, K] device weight -> U4Weight with groups of ``group`` (32, 64
    or 128) along K."""
    _need(w.dim() == 2 and w.dtype is _f32 and w.is_cuda, "an fp32 [N, K] tensor on the GPU is needed")
    _need(group in GROUPS, f"groups of {GROUPS} values are supported")
    N, K = w.shape
    _need(N > 0 and K > 0 and K % group == 0, f"K = {K} is not a positive multiple of {group}")
    w = w.contiguous()
    device = w.device
    codes = torch.empty((N, K // 2), dtype=_u8, device=device)
    pairs = torch.empty((N, K // group, 2), dtype=_bf16, device=device)
    _call("qlora_quantize_u4", None, w.get_device(), w.data_ptr(), N * K, group, codes.data_ptr(),
          pairs.data_ptr())
    return U4Weight(codes, pairs)


def dequantize_u4(uw: U4Weight, dtype=torch.bfloat16):
    """U4Weight -> its values [N, K] in bf16 or fp16."""
    _need(dtype in _16BIT, "bf16 or fp16 values")
    w = uw.now()
    out = torch.empty((uw.N, uw.K), dtype=dtype, device=uw.device)
    _call("qlora_dequantize_u4", dtype, uw.index, w, out.data_ptr())
    return out


def linear_u4_fwd(uw: U4Weight, x, y=None):
    """y = x . W^T for few tokens: x [M, K] bf16 or fp16 (rows may be
    strided), y [M, N] of the same type (rows may be strided)."""
    w = uw.now()
    dt, shape, N, K, index = x.dtype, x.shape, uw.N, uw.K, uw.index
    if dt not in _16BIT:
        raise ValueError("x has to be bf16 or fp16")
    if len(shape) != 2 or shape[1] != K or x.get_device() != index or x.stride(1) != 1:
        raise ValueError(f"x: [M, {K}] on GPU {index} with unit stride along K is needed")
    M = shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=dt, device=x.device)
        ldy = N
    else:
        _need(y.dtype is dt and tuple(y.shape) == (M, N) and y.get_device() == index
              and (y.stride(1) == 1 or N == 1),
              f"y: [{M}, {N}] like x, with unit stride along N, is needed")
        ldy = y.stride(0) if M > 1 else N
    _call("qlora_linear_u4_fwd", dt, index, w, x.data_ptr(), x.stride(0) if M > 1 else K,
          M, y.data_ptr(), ldy)
    return y


# ---------------------------------------------------------------------------
# the paged cache
# ---------------------------------------------------------------------------

class Kv4Cache:
    """Keys and values in the 4-bit group format, in pages: codes uint8
    [pages, kv_heads, page_size, head_dim / 2] and pairs bf16 [pages,
    kv_heads, page_size, 2], one pair per token and head."""

    __slots__ = ("k_codes", "k_pairs", "v_codes", "v_pairs", "pages", "kv_heads", "page_size",
                 "head_dim", "index", "struct", "at")

    def __init__(self, k_codes, k_pairs, v_codes, v_pairs):
        _dense(k_codes, "k_codes", _u8)
        index = k_codes.get_device()
        _dense(k_pairs, "k_pairs", _bf16, index)
        _dense(v_codes, "v_codes", _u8, index)
        _dense(v_pairs, "v_pairs", _bf16, index)
        shape = k_codes.shape
        if len(shape) != 4:
            raise ValueError("codes [pages, kv_heads, page_size, head_dim / 2] are needed")
        pages, heads, size, half = shape
        pair = (pages, heads, size, 2)
        if v_codes.shape != shape or k_pairs.shape != pair or v_pairs.shape != pair:
            raise ValueError("codes and pairs of one cache differ in shape")
        if 2 * half not in HEAD_DIMS:
            raise ValueError(f"head_dim {2 * half}: {HEAD_DIMS} are supported")
        if not 16 <= size <= 1024 or size & (size - 1):
            raise ValueError(f"page_size {size}: a power of two from 16 to 1024 is needed")
        self.k_codes, self.k_pairs, self.v_codes, self.v_pairs = k_codes, k_pairs, v_codes, v_pairs
        self.pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, size, 2 * half
        self.index = index
        self.at = at = (k_codes, k_codes.data_ptr(), k_pairs, k_pairs.data_ptr(),
                        v_codes, v_codes.data_ptr(), v_pairs, v_pairs.data_ptr())
        self.struct = Kv4CacheStruct(*at[1::2], pages, size, heads, 2 * half)

    def now(self) -> Kv4CacheStruct:
        """The descriptor of the tensors as they are (as :meth:`U4Weight.now`)."""
        kc, kca, kp, kpa, vc, vca, vp, vpa = self.at
        if self.k_codes is not kc or self.k_pairs is not kp or self.v_codes is not vc or \
                self.v_pairs is not vp or kc.data_ptr() != kca or kp.data_ptr() != kpa or \
                vc.data_ptr() != vca or vp.data_ptr() != vpa:
            self.__init__(self.k_codes, self.k_pairs, self.v_codes, self.v_pairs)
        return self.struct

    @property
    def device(self):
        return self.k_codes.device

    @classmethod
    def empty(cls, pages: int, page_size: int, kv_heads: int, head_dim: int, device="cuda"):
        """A pool of ``pages`` pages, uninitialised."""
        def new(n, dt):
            return torch.empty((pages, kv_heads, page_size, n), dtype=dt, device=device)
        return cls(new(head_dim // 2, _u8), new(2, _bf16), new(head_dim // 2, _u8), new(2, _bf16))


def _batch(cache: Kv4Cache, cu_q, seq_lens, block_table, max_q: int, rows: int) -> Kv4BatchStruct:
    index = cache.index
    for t, n in ((cu_q, "cu_q"), (seq_lens, "seq_lens"), (block_table, "block_table")):
        if t.dtype is not _i32 or t.get_device() != index or not t.is_contiguous():
            raise ValueError(f"{n}: a contiguous int32 tensor on GPU {index} is needed")
    cs, ls, bs = cu_q.shape, seq_lens.shape, block_table.shape
    if len(ls) != 1 or len(cs) != 1 or len(bs) != 2 or cs[0] != ls[0] + 1 or bs[0] != ls[0]:
        raise ValueError("cu_q [B + 1], seq_lens [B] and block_table [B, width] are needed")
    if not 0 <= max_q < _I32:
        raise ValueError(f"max_q {max_q} is out of range")
    if ls[0] >= _I32 or bs[1] >= _I32:
        raise ValueError(f"block_table {tuple(bs)} is out of range")
    return Kv4BatchStruct(cu_q.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(), rows,
                          ls[0], bs[1], max_q)


def _rows(cache: Kv4Cache, t, name: str, dtype, rows: int, heads: int):
    """Checks a [rows, heads, head_dim] tensor (-1: any); returns its rows,
    heads and (token, head) strides."""
    shape = t.shape
    if len(shape) != 3 or shape[2] != cache.head_dim or t.dtype is not dtype or \
            t.get_device() != cache.index or (rows >= 0 and shape[0] != rows) or \
            (heads >= 0 and shape[1] != heads):
        raise ValueError(f"{name}: [{'T' if rows < 0 else rows}, "
                         f"{'heads' if heads < 0 else heads}, {cache.head_dim}] of {dtype} on "
                         f"{cache.device} is needed, got {tuple(shape)} of {t.dtype} on {t.device}")
    ts, hs, ds = t.stride()
    if shape[1] >= _I32:
        raise ValueError(f"{name}: {shape[1]} heads are out of range")
    if ds != 1:
        raise ValueError(f"{name}: unit stride along head_dim is needed")
    # the stride of an axis of length one says nothing
    T, H = shape[0], shape[1]
    return T, H, (ts if T > 1 else 0), (hs if H > 1 else 0)


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
    if dt not in _16BIT:
        raise ValueError("k, v and q have to be bf16 or fp16")
    pool = cache.now()
    T, _, kts, khs = _rows(cache, k, "k", dt, -1, cache.kv_heads)
    _, _, vts, vhs = _rows(cache, v, "v", dt, T, cache.kv_heads)
    qp = op = None
    qts = qhs = heads = 0
    if q is not None:
        _, heads, qts, qhs = _rows(cache, q, "q", dt, T, -1)
        if q_out is None:
            q_out = torch.empty((T, heads, cache.head_dim), dtype=dt, device=k.device)
        else:
            _need(q_out.shape == q.shape and q_out.dtype is dt and q_out.get_device() == cache.index
                  and q_out.is_contiguous(), "q_out has to be contiguous and like q")
        qp, op = q.data_ptr(), q_out.data_ptr()
    else:
        _need(q_out is None, "q_out without q")
    rot = rows = 0
    tp = None
    if cos_sin is not None:
        _need(cos_sin.dim() == 2, "cos_sin: [positions, rot] is needed")
        _dense(cos_sin, "cos_sin", _f32, cache.index)
        rows, rot = cos_sin.shape
        _need(rot < _I32, f"cos_sin: {rot} columns are out of range")
        tp = cos_sin.data_ptr()
    bt = _batch(cache, cu_q, seq_lens, block_table, max_q, T)
    _call("qlora_kv4_append", dt, cache.index, pool, bt, k.data_ptr(), kts, khs,
          v.data_ptr(), vts, vhs, qp, qts, qhs, heads, tp, rows, rot, 1 if interleaved else 0, op)
    return q_out


def kv4_read(cache: Kv4Cache, cu_q, seq_lens, block_table, max_q: int, rows: int,
             dtype=torch.bfloat16) -> Tuple[object, object]:
    """The keys and values that the cache holds for the batch's ``rows`` rows,
    [rows, kv_heads, head_dim] each, in bf16 or fp16; rows behind
    cu_q[-1] are uninitialised."""
    _need(dtype in _16BIT, "bf16 or fp16 values")
    _need(rows >= 0, "rows is negative")
    pool = cache.now()
    bt = _batch(cache, cu_q, seq_lens, block_table, max_q, rows)
    shape, device = (rows, cache.kv_heads, cache.head_dim), cu_q.device
    k = torch.empty(shape, dtype=dtype, device=device)
    v = torch.empty(shape, dtype=dtype, device=device)
    _call("qlora_kv4_read", dtype, cache.index, pool, bt, k.data_ptr(), v.data_ptr())
    return k, v


def kv4_attention_workspace_bytes(seqs: int, max_q: int, max_len: int, q_heads: int,
                                  kv_heads: int, head_dim: int, window: int = 0) -> int:
    # what is negative is the library's to refuse
    for n, v in (("q_heads", q_heads), ("kv_heads", kv_heads), ("head_dim", head_dim),
                 ("window", window)):
        _need(-_I32 <= v < _I32, f"{n} {v} is out of range")
    for n, v in (("seqs", seqs), ("max_q", max_q), ("max_len", max_len)):
        _need(-2 ** 63 <= v < 2 ** 63, f"{n} {v} is out of range")
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
    if dt not in _16BIT:
        raise ValueError("q has to be bf16 or fp16")
    pool = cache.now()
    T, heads, qts, qhs = _rows(cache, q, "q", dt, -1, -1)
    D, index, device = cache.head_dim, cache.index, q.device
    bt = _batch(cache, cu_q, seq_lens, block_table, max_q, T)
    if out is None:
        out = torch.empty((T, heads, D), dtype=dt, device=device)
    else:
        _need(out.shape == q.shape and out.dtype is dt and out.get_device() == index
              and out.is_contiguous(), "out has to be contiguous and like q")
    if lse is not None:
        _need(tuple(lse.shape) == (T, heads) and lse.dtype is _f32 and lse.is_contiguous()
              and lse.get_device() == index, f"lse: fp32 [{T}, {heads}] is needed")
    elif return_lse:
        lse = torch.empty((T, heads), dtype=_f32, device=device)
    # what is negative is the library's to refuse
    if not -_I32 <= window < _I32 or not -2 ** 63 <= max_len < 2 ** 63:
        raise ValueError(f"window {window} or max_len {max_len} is out of range")
    need = _lib.lib().qlora_kv4_attention_workspace_bytes(bt.seqs, max_q, max_len, heads,
                                                          cache.kv_heads, D, window)
    if workspace is None:
        if need:
            workspace = torch.empty(need, dtype=_u8, device=device)
    else:
        _dense(workspace, "workspace", _u8, index)
        need = workspace.numel()
    _call("qlora_kv4_attention", dt, index, pool, bt, q.data_ptr(), qts, qhs, heads,
          D ** -0.5 if scale is None else scale, 1 if causal else 0, window, max_len,
          out.data_ptr(), None if lse is None else lse.data_ptr(),
          None if workspace is None else workspace.data_ptr(), need)
    return (out, lse) if return_lse else out
