"""ctypes binding of ``libqlora.so`` -- the C ABI declared in include/qlora.h.

The raw functions keep the C names and take integers for device pointers.
The torch-facing helpers below only marshal arguments (shapes, dtypes,
``data_ptr()``, the current stream) and call the raw functions; all
arithmetic happens in the library's HIP kernels.  If the library is
missing, loading raises -- there is no fallback path.
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqlora.so")

QLORA_OK = 0
STATUS_NAMES = {0: "QLORA_OK", -1: "QLORA_EINVAL", -2: "QLORA_ESHAPE", -3: "QLORA_EALIGN",
                -4: "QLORA_ENOTSUP", -5: "QLORA_EWORKSPACE", -6: "QLORA_EHIP",
                -7: "QLORA_ESCRATCH"}

EXPORTS = ("qlora_quantize_nf4", "qlora_double_quant", "qlora_quantize_nf4_dq",
           "qlora_dq_centred_workspace_bytes", "qlora_double_quant_centred",
           "qlora_quantize_nf4_dq_centred",
           "qlora_dequantize_nf4",
           "qlora_linear_fwd", "qlora_linear_bwd", "qlora_linear_workspace_bytes",
           "qlora_linear_fwd_dropout", "qlora_linear_bwd_dropout",
           "qlora_dequantize_nf4_f16", "qlora_linear_fwd_f16", "qlora_linear_bwd_f16",
           "qlora_linear_bf16_fwd", "qlora_linear_bf16_bwd",
           "qlora_dropout_keep_mask", "qlora_linear_fwd_dropout_rng",
           "qlora_linear_bwd_dropout_rng",
           "qlora_merge_adapter", "qlora_linear_fwd_noalloc", "qlora_nf4_levels",
           "qlora_nf4_thresholds", "qlora_status_string",
           "qlora_quantize_u4", "qlora_dequantize_u4", "qlora_dequantize_u4_f16",
           "qlora_linear_u4_fwd", "qlora_linear_u4_fwd_f16",
           "qlora_kv4_append", "qlora_kv4_append_f16", "qlora_kv4_read", "qlora_kv4_read_f16",
           "qlora_kv4_attention_workspace_bytes", "qlora_kv4_attention",
           "qlora_kv4_attention_f16",
           "qlora_quantize_i8", "qlora_dequantize_i8", "qlora_dequantize_i8_f16",
           "qlora_quantize_tokens_i8", "qlora_quantize_tokens_i8_f16",
           "qlora_dequantize_tokens_i8", "qlora_dequantize_tokens_i8_f16",
           "qlora_rms_norm_i8", "qlora_rms_norm_i8_f16",
           "qlora_linear_i8_fwd", "qlora_linear_i8_fwd_f16",
           "qlora_gated_i8_fwd", "qlora_gated_i8_fwd_f16")


class QloraError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)} "
                         f"({lib().qlora_status_string(status).decode()})")


class Nf4Weight(ctypes.Structure):
    """``qlora_nf4_weight``: device pointers to codes, qscale, dq_step; N, K;
    dq_mean (null for the unsigned scale format)."""
    _fields_ = [("codes", ctypes.c_void_p), ("qscale", ctypes.c_void_p),
                ("dq_step", ctypes.c_void_p), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("dq_mean", ctypes.c_void_p)]


class U4Struct(ctypes.Structure):
    """``qlora_u4_weight``."""
    _fields_ = [("codes", ctypes.c_void_p), ("pairs", ctypes.c_void_p), ("N", ctypes.c_int64),
                ("K", ctypes.c_int64), ("group", ctypes.c_int32)]


class Kv4CacheStruct(ctypes.Structure):
    """``qlora_kv4_cache``."""
    _fields_ = [("k_codes", ctypes.c_void_p), ("k_pairs", ctypes.c_void_p),
                ("v_codes", ctypes.c_void_p), ("v_pairs", ctypes.c_void_p),
                ("pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class Kv4BatchStruct(ctypes.Structure):
    """``qlora_kv4_batch``."""
    _fields_ = [("cu_q", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("seqs", ctypes.c_int32), ("table_width", ctypes.c_int32),
                ("max_q", ctypes.c_int32)]


class I8WeightStruct(ctypes.Structure):
    """``qlora_i8_weight``."""
    _fields_ = [("tiles", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("N", ctypes.c_int64),
                ("K", ctypes.c_int64)]


class I8TokensStruct(ctypes.Structure):
    """``qlora_i8_tokens``."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("M", ctypes.c_int64),
                ("K", ctypes.c_int64)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load the library once; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing; build it with "
                          "`python -m bit_quantized_lora_03_amd.csrc.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, f32, sz, u64 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32,
                                  ctypes.c_float, ctypes.c_size_t, ctypes.c_uint64)
    wp = ctypes.POINTER(Nf4Weight)
    up, cp, bp = (ctypes.POINTER(U4Struct), ctypes.POINTER(Kv4CacheStruct),
                  ctypes.POINTER(Kv4BatchStruct))
    append = [cp, bp, vp, i64, i64, vp, i64, i64, vp, i64, i64, i32, vp, i64, i32, i32, vp, vp]
    iw, it, f64 = (ctypes.POINTER(I8WeightStruct), ctypes.POINTER(I8TokensStruct),
                   ctypes.c_double)
    tokens = [vp, i64, i64, i64, vp, vp, vp]
    norm = [vp, i64, vp, i64, vp, f64, i64, i64, vp, i64, vp, vp, vp]
    product = [iw, it, vp, i64, vp]
    gated = [iw, iw, i32, it, vp, i64, vp]
    attend = [cp, bp, vp, i64, i64, i32, f32, i32, i32, i64, vp, vp, vp, sz, vp]
    sig = {
        "qlora_quantize_nf4": ([vp, i64, i32, vp, vp, vp], ctypes.c_int),
        "qlora_double_quant": ([vp, i64, i32, vp, vp, vp], ctypes.c_int),
        "qlora_quantize_nf4_dq": ([vp, i64, vp, vp, vp, vp, vp], ctypes.c_int),
        "qlora_dq_centred_workspace_bytes": ([i64], sz),
        "qlora_double_quant_centred": ([vp, i64, vp, vp, vp, vp, sz, vp], ctypes.c_int),
        "qlora_quantize_nf4_dq_centred": ([vp, i64, vp, vp, vp, vp, vp, vp, sz, vp],
                                          ctypes.c_int),
        "qlora_dequantize_nf4": ([wp, vp, vp], ctypes.c_int),
        "qlora_linear_fwd": ([wp, vp, i64, vp, vp, i32, f32, vp, vp, sz, vp], ctypes.c_int),
        "qlora_linear_bwd": ([wp, vp, vp, i64, vp, vp, i32, f32, vp, vp, vp, i32, vp, sz, vp],
                             ctypes.c_int),
        "qlora_linear_workspace_bytes": ([i32, i64, i64, i64, i32], sz),
        "qlora_merge_adapter": ([wp, vp, i64, i64, vp, vp, i32, f32, vp, vp, vp], ctypes.c_int),
        "qlora_dequantize_nf4_f16": ([wp, vp, vp], ctypes.c_int),
        "qlora_linear_fwd_f16": ([wp, vp, i64, vp, vp, i32, f32, vp, vp, sz, vp], ctypes.c_int),
        "qlora_linear_bwd_f16": ([wp, vp, vp, i64, vp, vp, i32, f32, vp, vp, vp, i32, vp, sz, vp],
                                 ctypes.c_int),
        "qlora_linear_fwd_dropout": ([wp, vp, i64, vp, vp, i32, f32, vp, f32, vp, vp, sz, vp],
                                     ctypes.c_int),
        "qlora_linear_bwd_dropout": ([wp, vp, vp, i64, vp, vp, i32, f32, vp, f32, vp, vp, vp, i32,
                                      vp, sz, vp], ctypes.c_int),
        "qlora_linear_bf16_fwd": ([vp, i64, i64, vp, i64, vp, vp, i32, f32, vp, vp, sz, vp],
                                  ctypes.c_int),
        "qlora_linear_bf16_bwd": ([vp, i64, i64, vp, vp, i64, vp, vp, i32, f32, vp, vp, vp, i32,
                                   vp, sz, vp], ctypes.c_int),
        "qlora_linear_fwd_noalloc": ([wp, vp, i64, vp, vp, i32, f32, vp, vp], ctypes.c_int),
        "qlora_dropout_keep_mask": ([i64, i64, f32, u64, u64, vp, vp], ctypes.c_int),
        "qlora_linear_fwd_dropout_rng": ([wp, vp, i64, vp, vp, i32, f32, f32, u64, u64, vp, vp,
                                          sz, vp], ctypes.c_int),
        "qlora_linear_bwd_dropout_rng": ([wp, vp, vp, i64, vp, vp, i32, f32, f32, u64, u64, vp,
                                          vp, vp, i32, vp, sz, vp], ctypes.c_int),
        "qlora_nf4_levels": ([vp], ctypes.c_int),
        "qlora_nf4_thresholds": ([vp], ctypes.c_int),
        "qlora_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "qlora_quantize_u4": ([vp, i64, i32, vp, vp, vp], ctypes.c_int),
        "qlora_dequantize_u4": ([up, vp, vp], ctypes.c_int),
        "qlora_dequantize_u4_f16": ([up, vp, vp], ctypes.c_int),
        "qlora_linear_u4_fwd": ([up, vp, i64, i64, vp, i64, vp], ctypes.c_int),
        "qlora_linear_u4_fwd_f16": ([up, vp, i64, i64, vp, i64, vp], ctypes.c_int),
        "qlora_kv4_append": (append, ctypes.c_int),
        "qlora_kv4_append_f16": (append, ctypes.c_int),
        "qlora_kv4_read": ([cp, bp, vp, vp, vp], ctypes.c_int),
        "qlora_kv4_read_f16": ([cp, bp, vp, vp, vp], ctypes.c_int),
        "qlora_kv4_attention_workspace_bytes": ([i64, i64, i64, i32, i32, i32, i32], sz),
        "qlora_kv4_attention": (attend, ctypes.c_int),
        "qlora_kv4_attention_f16": (attend, ctypes.c_int),
        "qlora_quantize_i8": ([vp, i64, i64, vp, vp, vp], ctypes.c_int),
        "qlora_dequantize_i8": ([iw, vp, vp], ctypes.c_int),
        "qlora_dequantize_i8_f16": ([iw, vp, vp], ctypes.c_int),
        "qlora_quantize_tokens_i8": (tokens, ctypes.c_int),
        "qlora_quantize_tokens_i8_f16": (tokens, ctypes.c_int),
        "qlora_dequantize_tokens_i8": ([it, vp, vp], ctypes.c_int),
        "qlora_dequantize_tokens_i8_f16": ([it, vp, vp], ctypes.c_int),
        "qlora_rms_norm_i8": (norm, ctypes.c_int),
        "qlora_rms_norm_i8_f16": (norm, ctypes.c_int),
        "qlora_linear_i8_fwd": (product, ctypes.c_int),
        "qlora_linear_i8_fwd_f16": (product, ctypes.c_int),
        "qlora_gated_i8_fwd": (gated, ctypes.c_int),
        "qlora_gated_i8_fwd_f16": (gated, ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _lib = L
    return L


def check(status: int, what: str) -> None:
    if status != QLORA_OK:
        raise QloraError(status, what)


# ---------------------------------------------------------------------------
# host-only helpers
# ---------------------------------------------------------------------------

def nf4_levels():
    """The library's own fp32 NF4 levels and thresholds (numpy arrays)."""
    import numpy as np
    lv = np.zeros(16, dtype=np.float32)
    th = np.zeros(15, dtype=np.float32)
    check(lib().qlora_nf4_levels(lv.ctypes.data), "qlora_nf4_levels")
    check(lib().qlora_nf4_thresholds(th.ctypes.data), "qlora_nf4_thresholds")
    return lv, th


def workspace_bytes(op: int, M: int, N: int, K: int, r: int) -> int:
    return int(lib().qlora_linear_workspace_bytes(op, M, N, K, r))


# ---------------------------------------------------------------------------
# torch-facing marshalling (device tensors in, device tensors out)
# ---------------------------------------------------------------------------

def _torch():
    import torch
    return torch


def _stream_ptr() -> int:
    torch = _torch()
    return torch.cuda.current_stream().cuda_stream


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


class PackedWeight:
    """A frozen NF4 base weight living in device memory; ``dq_mean`` (an fp32
    device tensor of one element) marks the mean-centred scale format."""

    def __init__(self, codes, qscale, dq_step, N: int, K: int, dq_mean=None):
        self.codes, self.qscale, self.dq_step = codes, qscale, dq_step
        self.dq_mean = dq_mean
        self.N, self.K = int(N), int(K)

    def struct(self) -> Nf4Weight:
        return Nf4Weight(self.codes.data_ptr(), self.qscale.data_ptr(),
                         self.dq_step.data_ptr(), self.N, self.K, _ptr(self.dq_mean))


def quantize_nf4(w) -> Tuple[object, object]:
    """fp32 device tensor -> (packed codes uint8 [ceil(n/2)], absmax fp32 [ceil(n/64)])."""
    torch = _torch()
    assert w.dtype == torch.float32 and w.is_cuda and w.is_contiguous()
    n = w.numel()
    codes = torch.empty((n + 1) // 2, dtype=torch.uint8, device=w.device)
    absmax = torch.empty((n + 63) // 64, dtype=torch.float32, device=w.device)
    check(lib().qlora_quantize_nf4(_ptr(w), n, 64, _ptr(codes), _ptr(absmax), _stream_ptr()),
          "qlora_quantize_nf4")
    return codes, absmax


def double_quant(absmax) -> Tuple[object, object]:
    """fp32 block scales -> (qscale uint8 [nb], dq_step fp32 [ceil(nb/256)])."""
    torch = _torch()
    assert absmax.dtype == torch.float32 and absmax.is_cuda and absmax.is_contiguous()
    nb = absmax.numel()
    q = torch.empty(nb, dtype=torch.uint8, device=absmax.device)
    step = torch.empty((nb + 255) // 256, dtype=torch.float32, device=absmax.device)
    check(lib().qlora_double_quant(_ptr(absmax), nb, 256, _ptr(q), _ptr(step), _stream_ptr()),
          "qlora_double_quant")
    return q, step


def quantize_nf4_dq(w) -> Tuple[object, object, object, object]:
    """fp32 device tensor -> (codes, absmax, qscale, dq_step) in one pass:
    the outputs of quantize_nf4 followed by double_quant, bit for bit."""
    torch = _torch()
    assert w.dtype == torch.float32 and w.is_cuda and w.is_contiguous()
    n = w.numel()
    nb = (n + 63) // 64
    codes = torch.empty((n + 1) // 2, dtype=torch.uint8, device=w.device)
    absmax = torch.empty(nb, dtype=torch.float32, device=w.device)
    q = torch.empty(nb, dtype=torch.uint8, device=w.device)
    step = torch.empty((nb + 255) // 256, dtype=torch.float32, device=w.device)
    check(lib().qlora_quantize_nf4_dq(_ptr(w), n, _ptr(codes), _ptr(absmax), _ptr(q),
                                      _ptr(step), _stream_ptr()),
          "qlora_quantize_nf4_dq")
    return codes, absmax, q, step


def _dqc_workspace(nb, device):
    torch = _torch()
    need = int(lib().qlora_dq_centred_workspace_bytes(nb))
    return torch.empty(max(need, 256), dtype=torch.uint8, device=device), need


def double_quant_centred(absmax) -> Tuple[object, object, object]:
    """fp32 block scales -> (qscale uint8 [nb] two's-complement codes,
    dq_step fp32 [ceil(nb/256)], dq_mean fp32 [1]): the mean-centred format."""
    torch = _torch()
    assert absmax.dtype == torch.float32 and absmax.is_cuda and absmax.is_contiguous()
    nb = absmax.numel()
    q = torch.empty(nb, dtype=torch.uint8, device=absmax.device)
    step = torch.empty((nb + 255) // 256, dtype=torch.float32, device=absmax.device)
    mean = torch.empty(1, dtype=torch.float32, device=absmax.device)
    ws, need = _dqc_workspace(nb, absmax.device)
    check(lib().qlora_double_quant_centred(_ptr(absmax), nb, _ptr(q), _ptr(step), _ptr(mean),
                                           _ptr(ws), ws.numel(), _stream_ptr()),
          "qlora_double_quant_centred")
    return q, step, mean


def quantize_nf4_dq_centred(w) -> Tuple[object, object, object, object, object]:
    """fp32 device tensor -> (codes, absmax, qscale, dq_step, dq_mean): the
    quantiser followed by the mean-centred double quantisation."""
    torch = _torch()
    assert w.dtype == torch.float32 and w.is_cuda and w.is_contiguous()
    n = w.numel()
    nb = (n + 63) // 64
    codes = torch.empty((n + 1) // 2, dtype=torch.uint8, device=w.device)
    absmax = torch.empty(nb, dtype=torch.float32, device=w.device)
    q = torch.empty(nb, dtype=torch.uint8, device=w.device)
    step = torch.empty((nb + 255) // 256, dtype=torch.float32, device=w.device)
    mean = torch.empty(1, dtype=torch.float32, device=w.device)
    ws, need = _dqc_workspace(nb, w.device)
    check(lib().qlora_quantize_nf4_dq_centred(_ptr(w), n, _ptr(codes), _ptr(absmax), _ptr(q),
                                              _ptr(step), _ptr(mean), _ptr(ws), ws.numel(),
                                              _stream_ptr()),
          "qlora_quantize_nf4_dq_centred")
    return codes, absmax, q, step, mean


def quantize_weight_centred(w) -> PackedWeight:
    """fp32 [N, K] device weight -> PackedWeight in the mean-centred format."""
    N, K = w.shape
    codes, _, q, step, mean = quantize_nf4_dq_centred(w.contiguous().view(-1))
    return PackedWeight(codes, q, step, N, K, dq_mean=mean)


def quantize_weight(w) -> PackedWeight:
    """fp32 [N, K] device weight -> PackedWeight (quantise and double-quantise
    in one pass)."""
    N, K = w.shape
    codes, _, q, step = quantize_nf4_dq(w.contiguous().view(-1))
    return PackedWeight(codes, q, step, N, K)


def dequantize(pw: PackedWeight):
    """PackedWeight -> bf16 bit patterns as an int16 device tensor [N, K]."""
    torch = _torch()
    out = torch.empty((pw.N, pw.K), dtype=torch.int16, device=pw.codes.device)
    s = pw.struct()
    check(lib().qlora_dequantize_nf4(ctypes.byref(s), _ptr(out), _stream_ptr()),
          "qlora_dequantize_nf4")
    return out


def _ws(op, M, N, K, r, device, workspace=None):
    torch = _torch()
    need = workspace_bytes(op, M, N, K, r)
    if workspace is not None:
        return workspace, need
    if need == 0:
        return None, 0
    return torch.empty(need, dtype=torch.uint8, device=device), need


def linear_fwd(pw: PackedWeight, x, A, B, alpha: float, y=None, workspace=None):
    """y = x.deq(W)^T + (alpha/r).(x.A^T).B^T; x/A/B bf16 (or int16 bit
    patterns) device tensors.  Returns y with x's dtype."""
    torch = _torch()
    M = x.shape[0]
    r = 0 if A is None else A.shape[0]
    if y is None:
        y = torch.empty((M, pw.N), dtype=x.dtype, device=x.device)
    ws, need = _ws(0, M, pw.N, pw.K, r, x.device, workspace)
    s = pw.struct()
    check(lib().qlora_linear_fwd(ctypes.byref(s), _ptr(x), M, _ptr(A), _ptr(B), r, float(alpha),
                                 _ptr(y), _ptr(ws), need if workspace is None else ws.numel(),
                                 _stream_ptr()), "qlora_linear_fwd")
    return y


def linear_fwd_noalloc(pw: PackedWeight, x, A, B, alpha: float, y=None):
    """The forward of :func:`linear_fwd` through qlora_linear_fwd_noalloc: no
    workspace argument (the library's static scratch buffer serves); the
    call allocates nothing when ``y`` is given."""
    torch = _torch()
    M = x.shape[0]
    r = 0 if A is None else A.shape[0]
    if y is None:
        y = torch.empty((M, pw.N), dtype=x.dtype, device=x.device)
    s = pw.struct()
    check(lib().qlora_linear_fwd_noalloc(ctypes.byref(s), _ptr(x), M, _ptr(A), _ptr(B), r,
                                         float(alpha), _ptr(y), _stream_ptr()),
          "qlora_linear_fwd_noalloc")
    return y


def linear_bwd(pw: PackedWeight, x, dy, A, B, alpha: float, need_dx: bool = True,
               dA=None, dB=None, accumulate: bool = False, workspace=None, dx=None):
    """Returns (dx or None, dA fp32 [r, K] or None, dB fp32 [N, r] or None);
    dx, dA, dB may be passed in as output tensors."""
    torch = _torch()
    M = dy.shape[0]
    r = 0 if A is None else A.shape[0]
    if need_dx and dx is None:
        dx = torch.empty((M, pw.K), dtype=dy.dtype, device=dy.device)
    if not need_dx:
        dx = None
    if r > 0:
        if dA is None:
            dA = torch.empty((r, pw.K), dtype=torch.float32, device=dy.device)
        if dB is None:
            dB = torch.empty((pw.N, r), dtype=torch.float32, device=dy.device)
    ws, need = _ws(1, M, pw.N, pw.K, r, dy.device, workspace)
    s = pw.struct()
    check(lib().qlora_linear_bwd(ctypes.byref(s), _ptr(x), _ptr(dy), M, _ptr(A), _ptr(B), r,
                                 float(alpha), _ptr(dx), _ptr(dA), _ptr(dB), int(accumulate),
                                 _ptr(ws), need if workspace is None else ws.numel(),
                                 _stream_ptr()), "qlora_linear_bwd")
    return dx, dA, dB


def dequantize_f16(pw: PackedWeight):
    """PackedWeight -> fp16 bit patterns as an int16 device tensor [N, K]."""
    torch = _torch()
    out = torch.empty((pw.N, pw.K), dtype=torch.int16, device=pw.codes.device)
    s = pw.struct()
    check(lib().qlora_dequantize_nf4_f16(ctypes.byref(s), _ptr(out), _stream_ptr()),
          "qlora_dequantize_nf4_f16")
    return out


def linear_fwd_f16(pw: PackedWeight, x, A, B, alpha: float, y=None, workspace=None):
    """The fp16 compute-type forward: x, A, B (fp16 or int16 bit patterns)
    and y in fp16."""
    torch = _torch()
    M = x.shape[0]
    r = 0 if A is None else A.shape[0]
    if y is None:
        y = torch.empty((M, pw.N), dtype=x.dtype, device=x.device)
    ws, need = _ws(6, M, pw.N, pw.K, r, x.device, workspace)
    s = pw.struct()
    check(lib().qlora_linear_fwd_f16(ctypes.byref(s), _ptr(x), M, _ptr(A), _ptr(B), r,
                                     float(alpha), _ptr(y), _ptr(ws),
                                     need if workspace is None else ws.numel(), _stream_ptr()),
          "qlora_linear_fwd_f16")
    return y


def linear_bwd_f16(pw: PackedWeight, x, dy, A, B, alpha: float, need_dx: bool = True, dA=None,
                   dB=None, accumulate: bool = False, workspace=None):
    """The fp16 compute-type backward: (dx fp16 or None, dA fp32, dB fp32)."""
    torch = _torch()
    M = dy.shape[0]
    r = 0 if A is None else A.shape[0]
    dx = torch.empty((M, pw.K), dtype=dy.dtype, device=dy.device) if need_dx else None
    if r > 0:
        if dA is None:
            dA = torch.empty((r, pw.K), dtype=torch.float32, device=dy.device)
        if dB is None:
            dB = torch.empty((pw.N, r), dtype=torch.float32, device=dy.device)
    ws, need = _ws(7, M, pw.N, pw.K, r, dy.device, workspace)
    s = pw.struct()
    check(lib().qlora_linear_bwd_f16(ctypes.byref(s), _ptr(x), _ptr(dy), M, _ptr(A), _ptr(B), r,
                                     float(alpha), _ptr(dx), _ptr(dA), _ptr(dB), int(accumulate),
                                     _ptr(ws), need if workspace is None else ws.numel(),
                                     _stream_ptr()), "qlora_linear_bwd_f16")
    return dx, dA, dB


def linear_fwd_dropout(pw: PackedWeight, x, A, B, alpha: float, keep, p: float, y=None,
                       workspace=None):
    """The forward pass with LoRA dropout on the adapter's input; ``keep`` is
    the packed mask, uint8 [M, K/8] (bit k mod 8 of byte (m, k/8))."""
    torch = _torch()
    M = x.shape[0]
    r = 0 if A is None else A.shape[0]
    if y is None:
        y = torch.empty((M, pw.N), dtype=x.dtype, device=x.device)
    ws, need = _ws(4, M, pw.N, pw.K, r, x.device, workspace)
    s = pw.struct()
    check(lib().qlora_linear_fwd_dropout(ctypes.byref(s), _ptr(x), M, _ptr(A), _ptr(B), r,
                                         float(alpha), _ptr(keep), float(p), _ptr(y), _ptr(ws),
                                         need if workspace is None else ws.numel(),
                                         _stream_ptr()), "qlora_linear_fwd_dropout")
    return y


def linear_bwd_dropout(pw: PackedWeight, x, dy, A, B, alpha: float, keep, p: float,
                       need_dx: bool = True, dA=None, dB=None, accumulate: bool = False,
                       workspace=None):
    """Backward of :func:`linear_fwd_dropout` with the same mask."""
    torch = _torch()
    M = dy.shape[0]
    r = 0 if A is None else A.shape[0]
    dx = torch.empty((M, pw.K), dtype=dy.dtype, device=dy.device) if need_dx else None
    if r > 0:
        if dA is None:
            dA = torch.empty((r, pw.K), dtype=torch.float32, device=dy.device)
        if dB is None:
            dB = torch.empty((pw.N, r), dtype=torch.float32, device=dy.device)
    ws, need = _ws(5, M, pw.N, pw.K, r, dy.device, workspace)
    s = pw.struct()
    check(lib().qlora_linear_bwd_dropout(ctypes.byref(s), _ptr(x), _ptr(dy), M, _ptr(A), _ptr(B),
                                         r, float(alpha), _ptr(keep), float(p), _ptr(dx),
                                         _ptr(dA), _ptr(dB), int(accumulate), _ptr(ws),
                                         need if workspace is None else ws.numel(),
                                         _stream_ptr()), "qlora_linear_bwd_dropout")
    return dx, dA, dB


def dropout_keep_mask(M: int, K: int, p: float, seed: int, offset: int, device=None, keep=None):
    """The packed keep mask [M, K/8] (uint8) that the library's drawn LoRA
    dropout uses for (p, seed, offset)."""
    torch = _torch()
    if keep is None:
        keep = torch.empty((M, K // 8), dtype=torch.uint8, device=device or "cuda")
    check(lib().qlora_dropout_keep_mask(M, K, float(p), int(seed), int(offset), _ptr(keep),
                                        _stream_ptr()), "qlora_dropout_keep_mask")
    return keep


def linear_fwd_dropout_rng(pw: PackedWeight, x, A, B, alpha: float, p: float, seed: int,
                           offset: int, y=None, workspace=None):
    """The forward with LoRA dropout drawn by the library (Philox4x32-10 from
    (seed, offset); no mask argument)."""
    torch = _torch()
    M = x.shape[0]
    r = 0 if A is None else A.shape[0]
    if y is None:
        y = torch.empty((M, pw.N), dtype=x.dtype, device=x.device)
    ws, need = _ws(8, M, pw.N, pw.K, r, x.device, workspace)
    s = pw.struct()
    check(lib().qlora_linear_fwd_dropout_rng(ctypes.byref(s), _ptr(x), M, _ptr(A), _ptr(B), r,
                                             float(alpha), float(p), int(seed), int(offset),
                                             _ptr(y), _ptr(ws),
                                             need if workspace is None else ws.numel(),
                                             _stream_ptr()), "qlora_linear_fwd_dropout_rng")
    return y


def linear_bwd_dropout_rng(pw: PackedWeight, x, dy, A, B, alpha: float, p: float, seed: int,
                           offset: int, need_dx: bool = True, dA=None, dB=None,
                           accumulate: bool = False, workspace=None, dx=None):
    """Backward of :func:`linear_fwd_dropout_rng` with the same (p, seed,
    offset): the library draws the same keep bits again."""
    torch = _torch()
    M = dy.shape[0]
    r = 0 if A is None else A.shape[0]
    if need_dx and dx is None:
        dx = torch.empty((M, pw.K), dtype=dy.dtype, device=dy.device)
    if not need_dx:
        dx = None
    if r > 0:
        if dA is None:
            dA = torch.empty((r, pw.K), dtype=torch.float32, device=dy.device)
        if dB is None:
            dB = torch.empty((pw.N, r), dtype=torch.float32, device=dy.device)
    ws, need = _ws(9, M, pw.N, pw.K, r, dy.device, workspace)
    s = pw.struct()
    check(lib().qlora_linear_bwd_dropout_rng(ctypes.byref(s), _ptr(x), _ptr(dy), M, _ptr(A),
                                             _ptr(B), r, float(alpha), float(p), int(seed),
                                             int(offset), _ptr(dx), _ptr(dA), _ptr(dB),
                                             int(accumulate), _ptr(ws),
                                             need if workspace is None else ws.numel(),
                                             _stream_ptr()), "qlora_linear_bwd_dropout_rng")
    return dx, dA, dB


def linear_bf16_fwd(W, x, A, B, alpha: float, y=None, workspace=None):
    """The same layer on an unquantised bf16 weight W [N, K] (bf16 or int16
    bit patterns): y = x.W^T + (alpha/r).(x.A^T).B^T."""
    torch = _torch()
    N, K = W.shape
    M = x.shape[0]
    r = 0 if A is None else A.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=x.dtype, device=x.device)
    ws, need = _ws(2, M, N, K, r, x.device, workspace)
    check(lib().qlora_linear_bf16_fwd(_ptr(W), N, K, _ptr(x), M, _ptr(A), _ptr(B), r,
                                      float(alpha), _ptr(y), _ptr(ws),
                                      need if workspace is None else ws.numel(), _stream_ptr()),
          "qlora_linear_bf16_fwd")
    return y


def linear_bf16_bwd(W, x, dy, A, B, alpha: float, need_dx: bool = True, dA=None, dB=None,
                    accumulate: bool = False, workspace=None):
    """Backward of :func:`linear_bf16_fwd`: (dx or None, dA fp32 or None,
    dB fp32 or None)."""
    torch = _torch()
    N, K = W.shape
    M = dy.shape[0]
    r = 0 if A is None else A.shape[0]
    dx = torch.empty((M, K), dtype=dy.dtype, device=dy.device) if need_dx else None
    if r > 0:
        if dA is None:
            dA = torch.empty((r, K), dtype=torch.float32, device=dy.device)
        if dB is None:
            dB = torch.empty((N, r), dtype=torch.float32, device=dy.device)
    ws, need = _ws(3, M, N, K, r, dy.device, workspace)
    check(lib().qlora_linear_bf16_bwd(_ptr(W), N, K, _ptr(x), _ptr(dy), M, _ptr(A), _ptr(B), r,
                                      float(alpha), _ptr(dx), _ptr(dA), _ptr(dB),
                                      int(accumulate), _ptr(ws),
                                      need if workspace is None else ws.numel(), _stream_ptr()),
          "qlora_linear_bf16_bwd")
    return dx, dA, dB


def merge_adapter(base, A, B, alpha: float, out_f32: bool = True, out_bf16: bool = True,
                  requantize=False):
    """W_m = W_base + (alpha/r).B.A for export.  ``base`` is a PackedWeight
    (merge into the decoded 4-bit base) or an fp32 [N, K] device tensor (the
    original weights).  Returns ``(fp32 [N, K] or None, bf16 bits [N, K]
    (int16) or None, PackedWeight, U4Weight, I8Weight or None)``; the last is
    the fp32 merge quantised again (needs the fp32 output): to NF4 with
    ``requantize=True`` or ``"nf4"``, to the 4-bit group format (groups of 64)
    with ``requantize="u4"``, to the 8-bit row format with
    ``requantize="i8"``; other texts are refused."""
    torch = _torch()
    if isinstance(requantize, str) and requantize not in ("", "nf4", "u4", "i8"):
        raise ValueError(f"requantize: True, False, 'nf4', 'u4' or 'i8', not {requantize!r}")
    if requantize and not out_f32:
        raise ValueError("requantize needs the fp32 merge")
    packed = isinstance(base, PackedWeight)
    if packed:
        N, K, device = base.N, base.K, base.codes.device
    else:
        N, K = base.shape
        device = base.device
    r = 0 if A is None else A.shape[0]
    f = torch.empty((N, K), dtype=torch.float32, device=device) if out_f32 else None
    b = torch.empty((N, K), dtype=torch.int16, device=device) if out_bf16 else None
    s = base.struct() if packed else None
    check(lib().qlora_merge_adapter(ctypes.byref(s) if packed else None,
                                    None if packed else base.data_ptr(), N, K, _ptr(A),
                                    _ptr(B), r, float(alpha), _ptr(f), _ptr(b),
                                    _stream_ptr()), "qlora_merge_adapter")
    if requantize == "u4":
        from .u4 import quantize_u4
        return f, b, quantize_u4(f)
    if requantize == "i8":
        from .i8 import quantize_i8
        return f, b, quantize_i8(f)
    q = quantize_weight(f) if requantize else None
    return f, b, q
