"""Torch-facing calls of the 8-bit row format (``qlora_*_i8*`` of
include/qlora.h): the quantisers of weights and tokens, the norm that writes
8-bit tokens, the product of the two and the gated half of an MLP.

As in the rest of the binding these only check and marshal arguments; the
arithmetic is the library's.  Work goes to the current stream of the device
that the tensors are on.  Arguments that do not fit raise ``ValueError``
before the library is called; what the library itself refuses raises
:class:`QloraError`.
"""

from __future__ import annotations

import torch

from ._lib import I8TokensStruct, I8WeightStruct
from .u4 import _16BIT, _call, _dense, _need

PAD = 128
ACTS = {"silu": 0, "gelu": 1}
_i8, _f32 = torch.int8, torch.float32
_empty = torch.empty  # (0.3 us less a call with the sizes as arguments than as a tuple)


def _padded(K: int) -> int:
    return (K + PAD - 1) // PAD * PAD


def _held(what, index, first, scales):
    """Refuses tensors that are not int8 and fp32, dense and on one GPU."""
    _dense(first, what, _i8)
    _dense(scales, "scales", _f32, index)


class I8Weight:
    """A weight [N, K] in the 8-bit row format: ``tiles`` int8
    [ceil(N / 16), Kp / 64, 4, 16, 16] with Kp = K rounded up to 128 (sixteen
    rows' first 16 columns, then their next) and ``scales`` fp32 [N]; a value
    is its row's scale times its code."""

    __slots__ = ("tiles", "scales", "N", "K", "index", "struct", "at")

    def __init__(self, tiles, scales, N: int, K: int):
        index = tiles.get_device()
        if tiles.dtype is not _i8 or scales.dtype is not _f32 or index < 0 or \
                scales.get_device() != index or not tiles.is_contiguous() or \
                not scales.is_contiguous():
            _held("tiles", index, tiles, scales)
        if N < 1 or K < 1 or scales.shape != (N,) or \
                tiles.shape != ((N + 15) // 16, (K + 127) // 128 * 2, 4, 16, 16):
            raise ValueError(f"tiles [{(N + 15) // 16}, {_padded(K) // 64}, 4, 16, 16] and scales "
                             f"[{N}] are needed for a weight [{N}, {K}]")
        self.tiles, self.scales, self.N, self.K, self.index = tiles, scales, N, K, index
        t, s = tiles.data_ptr(), scales.data_ptr()
        self.at = tiles, t, scales, s
        self.struct = I8WeightStruct(t, s, N, K)

    def now(self) -> I8WeightStruct:
        """The descriptor of the tensors as they are: checked and written anew
        where one was exchanged or has other memory since."""
        tiles, t, scales, s = self.at
        struct = self.struct
        if self.tiles is not tiles or self.scales is not scales or tiles.data_ptr() != t or \
                scales.data_ptr() != s or self.N != struct.N or self.K != struct.K:
            self.__init__(self.tiles, self.scales, self.N, self.K)
        return self.struct

    @property
    def device(self):
        return self.tiles.device


class I8Tokens:
    """Tokens [M, K] in the 8-bit row format: ``codes`` int8 [M, Kp], Kp = K
    rounded up to 128 (zeros from column K on), and ``scales`` fp32 [M]."""

    __slots__ = ("codes", "scales", "M", "K", "index", "struct", "at")

    def __init__(self, codes, scales, K: int):
        index = codes.get_device()
        if codes.dtype is not _i8 or scales.dtype is not _f32 or index < 0 or \
                scales.get_device() != index or not codes.is_contiguous() or \
                not scales.is_contiguous():
            _held("codes", index, codes, scales)
        shape = codes.shape
        if K < 1 or len(shape) != 2 or shape[1] != (K + 127) // 128 * 128 or \
                scales.shape != shape[:1]:
            raise ValueError(f"codes [M, {_padded(K)}] and scales [M] are needed for K = {K}")
        self.codes, self.scales, self.M, self.K, self.index = codes, scales, shape[0], K, index
        c, s = codes.data_ptr(), scales.data_ptr()
        self.at = codes, c, scales, s
        self.struct = I8TokensStruct(c, s, shape[0], K)

    def now(self) -> I8TokensStruct:
        """The descriptor of the tensors as they are (as :meth:`I8Weight.now`)."""
        codes, c, scales, s = self.at
        struct = self.struct
        if self.codes is not codes or self.scales is not scales or codes.data_ptr() != c or \
                scales.data_ptr() != s or self.M != struct.M or self.K != struct.K:
            self.__init__(self.codes, self.scales, self.K)
        return self.struct

    @property
    def device(self):
        return self.codes.device

    @classmethod
    def empty(cls, M: int, K: int, device="cuda"):
        """Room for ``M`` tokens, uninitialised."""
        if K < 1:
            raise ValueError(f"K = {K}: tokens have at least one value")
        codes = _empty(M, (K + 127) // 128 * 128, dtype=_i8, device=device)
        scales = _empty(M, dtype=_f32, device=device)
        index = codes.get_device()
        if index < 0:
            raise ValueError(f"tokens on the GPU are needed, not on {codes.device}")
        t = cls.__new__(cls)
        t.codes, t.scales, t.M, t.K, t.index = codes, scales, M, K, index
        c, s = codes.data_ptr(), scales.data_ptr()
        t.at = codes, c, scales, s
        t.struct = I8TokensStruct(c, s, M, K)
        return t


def _rows(t, name: str, dtype, M: int, K: int, index: int):
    """Checks a tensor of rows [M, K]; returns its row distance."""
    if t.dtype is not dtype or t.shape != (M, K) or t.get_device() != index or index < 0:
        raise ValueError(f"{name}: [{M}, {K}] of {dtype} on GPU {index} is needed, got "
                         f"{tuple(t.shape)} of {t.dtype} on {t.device}")
    ld, one = t.stride()
    if one != 1 and K != 1:
        raise ValueError(f"{name}: unit stride along its columns is needed")
    # the stride of an axis of length one says nothing
    return ld if M > 1 else K


def _tokens(out, M: int, K: int, x) -> I8Tokens:
    if out is None:
        return I8Tokens.empty(M, K, x.device)
    out.now()
    if out.M != M or out.K != K or out.index != x.get_device():
        raise ValueError(f"out: tokens [{M}, {K}] on {x.device} are needed")
    return out


# ---------------------------------------------------------------------------
# quantisers
# ---------------------------------------------------------------------------

def quantize_i8(w) -> I8Weight:
    """fp32 [N, K] device weight -> I8Weight, one scale per output channel."""
    _need(w.dim() == 2 and w.dtype is _f32 and w.is_cuda,
          "an fp32 [N, K] tensor on the GPU is needed")
    N, K = w.shape
    _need(N > 0 and K > 0, f"a weight [{N}, {K}] is empty")
    w = w.contiguous()
    tiles = torch.empty(((N + 15) // 16, _padded(K) // 64, 4, 16, 16), dtype=_i8, device=w.device)
    scales = torch.empty(N, dtype=_f32, device=w.device)
    _call("qlora_quantize_i8", None, w.get_device(), w.data_ptr(), N, K, tiles.data_ptr(),
          scales.data_ptr())
    return I8Weight(tiles, scales, N, K)


def dequantize_i8(iw: I8Weight, dtype=torch.bfloat16):
    """I8Weight -> its values [N, K] in bf16 or fp16."""
    _need(dtype in _16BIT, "bf16 or fp16 values")
    w = iw.now()
    out = _empty(iw.N, iw.K, dtype=dtype, device=iw.device)
    _call("qlora_dequantize_i8", dtype, iw.index, w, out.data_ptr())
    return out


def quantize_tokens_i8(x, out=None) -> I8Tokens:
    """x [M, K] bf16 or fp16 (rows may be strided) -> I8Tokens, one scale per
    token, into ``out`` where it is given."""
    dt = x.dtype
    shape = x.shape
    if dt not in _16BIT or len(shape) != 2 or shape[1] == 0:
        raise ValueError("x: [M, K] in bf16 or fp16 is needed")
    M, K = shape
    ld = _rows(x, "x", dt, M, K, x.get_device())
    out = _tokens(out, M, K, x)
    _call("qlora_quantize_tokens_i8", dt, out.index, x.data_ptr(), ld, M, K, out.codes.data_ptr(),
          out.scales.data_ptr())
    return out


def dequantize_tokens_i8(t: I8Tokens, dtype=torch.bfloat16):
    """I8Tokens -> their values [M, K] in bf16 or fp16."""
    _need(dtype in _16BIT, "bf16 or fp16 values")
    s = t.now()
    out = _empty(t.M, t.K, dtype=dtype, device=t.device)
    _call("qlora_dequantize_tokens_i8", dtype, t.index, s, out.data_ptr())
    return out


def rms_norm_i8(x, weight, eps: float, residual=None, h=None, out=None):
    """The root-mean-square norm of a residual stream, as 8-bit tokens: with
    h = x + residual (x itself without ``residual``), the tokens of
    h * weight / sqrt(mean(h^2) + eps).  x and residual [M, K] bf16 or fp16
    (rows may be strided), weight [K] of the same type.  Returns (tokens, h).

    The sum goes into ``h`` where it is given, which may be x or residual, and
    the tokens into ``out``."""
    dt = x.dtype
    shape = x.shape
    if dt not in _16BIT or len(shape) != 2 or shape[1] == 0:
        raise ValueError("x: [M, K] in bf16 or fp16 is needed")
    M, K = shape
    index = x.get_device()
    ldx = _rows(x, "x", dt, M, K, index)
    _dense(weight, "weight", dt, index)
    if weight.shape != (K,):
        raise ValueError(f"weight: [{K}] is needed")
    rp = hp = None
    ldr = ldh = 0
    if residual is not None:
        ldr = _rows(residual, "residual", dt, M, K, index)
        rp = residual.data_ptr()
        if h is None:
            h, ldh = _empty(M, K, dtype=dt, device=x.device), K
        else:
            ldh = _rows(h, "h", dt, M, K, index)
        hp = h.data_ptr()
    else:
        _need(h is None, "h without residual")
        h = x
    out = _tokens(out, M, K, x)
    _call("qlora_rms_norm_i8", dt, index, x.data_ptr(), ldx, rp, ldr, weight.data_ptr(), eps, M, K,
          hp, ldh, out.codes.data_ptr(), out.scales.data_ptr())
    return out, h


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

def _place(w: I8Weight, x: I8Tokens, y, dtype):
    """Checks the tokens and the output of a product; returns the output, its
    type and its row distance."""
    N, M = w.N, x.M
    if x.K != w.K or x.index != w.index:
        raise ValueError(f"tokens of {w.K} values on GPU {w.index} are needed, got {x.K} on "
                         f"{x.device}")
    if y is not None:
        if dtype is None:
            dtype = y.dtype
        ld = _rows(y, "y", dtype, M, N, w.index)
    elif dtype is None:
        dtype = torch.bfloat16
    if dtype not in _16BIT:
        raise ValueError("bf16 or fp16 outputs")
    if y is None:
        return _empty(M, N, dtype=dtype, device=x.device), dtype, N
    return y, dtype, ld


def linear_i8_fwd(iw: I8Weight, x: I8Tokens, y=None, dtype=None):
    """y = x . W^T of 8-bit tokens and an 8-bit weight, [M, N] in ``dtype``
    (bf16 or fp16; default: y's type, or bf16); y may have strided rows."""
    w, t = iw.now(), x.now()
    y, dtype, ld = _place(iw, x, y, dtype)
    _call("qlora_linear_i8_fwd", dtype, iw.index, w, t, y.data_ptr(), ld)
    return y


def gated_i8_fwd(gate: I8Weight, up: I8Weight, x: I8Tokens, act: str = "silu", y=None, dtype=None):
    """y = act(x . gate^T) * (x . up^T), [M, N], in one pass; ``act`` is
    "silu" or "gelu" (its tanh form).  Other arguments as
    :func:`linear_i8_fwd`."""
    if act not in ACTS:
        raise ValueError(f"act: one of {tuple(ACTS)} is needed, not {act!r}")
    g, u, t = gate.now(), up.now(), x.now()
    if up.N != gate.N or up.K != gate.K or up.index != gate.index:
        raise ValueError(f"up: [{gate.N}, {gate.K}] on GPU {gate.index} is needed, got "
                         f"[{up.N}, {up.K}] on {up.device}")
    y, dtype, ld = _place(gate, x, y, dtype)
    _call("qlora_gated_i8_fwd", dtype, gate.index, g, u, ACTS[act], t, y.data_ptr(), ld)
    return y
