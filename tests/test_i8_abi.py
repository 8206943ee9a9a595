"""Refusals of the 8-bit serving calls, without a GPU: every one comes from
validation before any HIP call (the addresses are fake) or from the Python
checks."""

import ctypes
import os

import pytest

import bit_quantized_lora_03_amd as q
from bit_quantized_lora_03_amd import _lib

pytestmark = pytest.mark.skipif(not os.path.exists(q.LIB_PATH), reason="libqlora.so not built")

MB = 1 << 20
OK, EINVAL, ESHAPE, EALIGN, ENOTSUP = 0, -1, -2, -3, -4
TAILS = pytest.mark.parametrize("tail", ["", "_f16"])
SIZES = [((0, 64), EINVAL), ((-1, 64), EINVAL), ((16, 0), EINVAL), ((16, -64), EINVAL),
         ((1 << 23, 64), ESHAPE), ((16, (1 << 17) - 127), ESHAPE), ((16, 1 << 40), ESHAPE)]


def at(i):
    return (i + 1) * 64 * MB


def call(name, *args):
    return getattr(q.lib(), name)(*args)


@pytest.mark.parametrize("size,status", SIZES)
def test_quantize_sizes(size, status):
    assert call("qlora_quantize_i8", at(0), *size, at(1), at(2), None) == status


def test_quantize_refusals():
    def f(w=at(0), t=at(1), s=at(2)):
        return call("qlora_quantize_i8", w, 100, 300, t, s, None)
    assert [f(w=None), f(t=None), f(s=None)] == [EINVAL] * 3
    assert [f(w=at(0) + 2), f(t=at(1) + 8), f(s=at(2) + 2)] == [EALIGN] * 3
    assert f(t=at(0) + 16) == EINVAL                       # tiles inside w
    assert f(s=at(0) + 100 * 300 * 4 - 4) == EINVAL        # scales on w's last value
    assert f(s=at(1) + 112 * 384 - 4) == EINVAL            # scales on the last tile


def weight(**kw):
    d = dict(tiles=at(0), scales=at(1), N=100, K=300)
    d.update(kw)
    return ctypes.byref(_lib.I8WeightStruct(d["tiles"], d["scales"], d["N"], d["K"]))


def tokens(**kw):
    d = dict(codes=at(2), scales=at(3), M=5, K=300)
    d.update(kw)
    return ctypes.byref(_lib.I8TokensStruct(d["codes"], d["scales"], d["M"], d["K"]))


BAD_WEIGHTS = [(dict(tiles=None), EINVAL), (dict(scales=None), EINVAL),
               (dict(tiles=at(0) + 8), EALIGN), (dict(scales=at(1) + 1), EALIGN)] + \
    [(dict(N=s[0], K=s[1]), st) for s, st in SIZES]
BAD_TOKENS = [(dict(codes=None), EINVAL), (dict(scales=None), EINVAL), (dict(M=-1), EINVAL),
              (dict(K=0), EINVAL), (dict(M=1 << 31), ESHAPE), (dict(K=1 << 17), ESHAPE),
              (dict(codes=at(2) + 8), EALIGN), (dict(scales=at(3) + 2), EALIGN)]


@TAILS
@pytest.mark.parametrize("kw,status", BAD_WEIGHTS)
def test_bad_weights(kw, status, tail):
    assert call("qlora_dequantize_i8" + tail, weight(**kw), at(5), None) == status
    assert call("qlora_linear_i8_fwd" + tail, weight(**kw), tokens(), at(5), 100, None) == status
    for a, b in ((weight(**kw), weight()), (weight(), weight(**kw))):
        assert call("qlora_gated_i8_fwd" + tail, a, b, 0, tokens(), at(5), 100, None) == status


@TAILS
@pytest.mark.parametrize("kw,status", BAD_TOKENS)
def test_bad_tokens(kw, status, tail):
    assert call("qlora_dequantize_tokens_i8" + tail, tokens(**kw), at(5), None) == status
    assert call("qlora_linear_i8_fwd" + tail, weight(), tokens(**kw), at(5), 100, None) == status
    d = dict(codes=at(2), scales=at(3), M=5, K=300)
    d.update(kw)
    assert call("qlora_quantize_tokens_i8" + tail, at(5), 1 << 20, d["M"], d["K"], d["codes"],
                d["scales"], None) == status
    assert call("qlora_rms_norm_i8" + tail, at(5), 1 << 20, None, 0, at(6), 1e-5, d["M"], d["K"],
                None, 0, d["codes"], d["scales"], None) == status


@TAILS
def test_null_handles(tail):
    assert call("qlora_dequantize_i8" + tail, None, at(5), None) == EINVAL
    assert call("qlora_dequantize_tokens_i8" + tail, None, at(5), None) == EINVAL
    assert call("qlora_linear_i8_fwd" + tail, None, tokens(), at(5), 100, None) == EINVAL
    assert call("qlora_linear_i8_fwd" + tail, weight(), None, at(5), 100, None) == EINVAL
    assert call("qlora_gated_i8_fwd" + tail, weight(), None, 0, tokens(), at(5), 100, None) == EINVAL


@TAILS
def test_outputs_of_the_readers(tail):
    for name, h, n, near in (("qlora_dequantize_i8", weight, 100 * 300 * 2, at(1)),
                             ("qlora_dequantize_tokens_i8", tokens, 5 * 300 * 2, at(3))):
        f = lambda out: call(name + tail, h(), out, None)  # noqa: E731
        assert f(None) == EINVAL and f(at(5) + 1) == EALIGN
        assert f(near - n + 2) == EINVAL                   # its last value is the first scale


@TAILS
def test_nothing_to_do(tail):
    none = tokens(codes=None, scales=None, M=0)
    assert call("qlora_dequantize_tokens_i8" + tail, none, None, None) == OK
    assert call("qlora_linear_i8_fwd" + tail, weight(), none, None, 0, None) == OK
    assert call("qlora_gated_i8_fwd" + tail, weight(), weight(), 1, none, None, 0, None) == OK
    assert call("qlora_quantize_tokens_i8" + tail, None, 0, 0, 300, None, None, None) == OK
    assert call("qlora_rms_norm_i8" + tail, None, 0, None, 0, None, 1e-5, 0, 300, None, 0, None,
                None, None) == OK


@TAILS
def test_quantize_tokens_refusals(tail):
    def f(x=at(5), ld=300, codes=at(2), scales=at(3)):
        return call("qlora_quantize_tokens_i8" + tail, x, ld, 5, 300, codes, scales, None)
    assert f(x=None) == EINVAL and f(ld=299) == EINVAL and f(ld=1 << 31) == ESHAPE
    assert f(x=at(5) + 1) == EALIGN
    assert f(codes=at(5) + 4 * 600 + 592) == EINVAL        # on x's last values
    assert f(codes=at(5) + 4 * 600 + 592, ld=400) == EINVAL  # in a gap, but in x's range
    assert f(scales=at(2) + 5 * 384 - 4) == EINVAL


@TAILS
def test_norm_refusals(tail):
    def f(x=at(5), ldx=300, r=at(6), ldr=300, w=at(7), eps=1e-5, h=at(8), ldh=300, codes=at(2),
          scales=at(3)):
        return call("qlora_rms_norm_i8" + tail, x, ldx, r, ldr, w, eps, 5, 300, h, ldh, codes,
                    scales, None)
    assert [f(x=None), f(w=None), f(r=None), f(h=None)] == [EINVAL] * 4
    for eps in (-1e-9, float("nan"), float("inf")):
        assert f(eps=eps) == EINVAL
    assert [f(ldx=299), f(ldr=299), f(ldh=299)] == [EINVAL] * 3
    assert [f(ldx=1 << 31), f(ldr=1 << 31), f(ldh=1 << 31)] == [ESHAPE] * 3
    assert [f(x=at(5) + 1), f(r=at(6) + 1), f(h=at(8) + 1), f(w=at(7) + 1)] == [EALIGN] * 4
    # h may be x or the residual, but not lie across them, nor on the others
    assert f(h=at(5) + 2) == EINVAL and f(h=at(6) + 600) == EINVAL
    assert f(h=at(5), ldh=400) == EINVAL and f(h=at(6), ldh=400) == EINVAL
    assert f(h=at(7)) == EINVAL and f(h=at(2)) == EINVAL and f(h=at(3)) == EINVAL
    for t in (at(5), at(6), at(7), at(8)):
        assert f(codes=t) == EINVAL and f(scales=t) == EINVAL


@TAILS
def test_product_refusals(tail):
    def f(y=at(5), ldy=100, w=None, t=None):
        return call("qlora_linear_i8_fwd" + tail, w or weight(), t or tokens(), y, ldy, None)

    def g(y=at(5), ldy=100, act=0, up=None, t=None):
        return call("qlora_gated_i8_fwd" + tail, weight(), up or weight(tiles=at(6), scales=at(7)),
                    act, t or tokens(), y, ldy, None)
    for h in (f, g):
        assert h(y=None) == EINVAL and h(ldy=99) == EINVAL and h(ldy=1 << 31) == ESHAPE
        assert h(y=at(5) + 1) == EALIGN
        assert h(t=tokens(K=299)) == EINVAL                # same padded width, another K
        assert h(t=tokens(M=(1 << 28) + 1)) == ESHAPE
        assert h(t=tokens(M=1 << 27)) == ESHAPE            # 2^27 * 128
        for other in (at(0), at(1), at(2), at(3)):
            assert h(y=other) == EINVAL
    assert f(w=weight(N=1 << 22, K=64), t=tokens(M=1 << 15, K=64), ldy=1 << 25) == ESHAPE
    assert g(y=at(6)) == EINVAL and g(y=at(7)) == EINVAL
    assert g(act=2) == ENOTSUP and g(act=-1) == ENOTSUP
    assert g(up=weight(N=99)) == EINVAL and g(up=weight(K=301)) == EINVAL


# ---------------------------------------------------------------------------
# the Python checks (CPU tensors are refused before the library is called)
# ---------------------------------------------------------------------------

torch = pytest.importorskip("torch")


def test_python_refuses_cpu_tensors_and_types():
    for f in (lambda: q.quantize_i8(torch.zeros(4, 4)),
              lambda: q.quantize_i8(torch.zeros(4)),
              lambda: q.quantize_tokens_i8(torch.zeros(4, 4)),
              lambda: q.quantize_tokens_i8(torch.zeros(4, 4, dtype=torch.bfloat16)),
              lambda: q.quantize_tokens_i8(torch.zeros(4, 0, dtype=torch.bfloat16)),
              lambda: q.rms_norm_i8(torch.zeros(4, 4, dtype=torch.bfloat16),
                                    torch.zeros(4, dtype=torch.bfloat16), 1e-5),
              lambda: q.rms_norm_i8(torch.zeros(4, 4), torch.zeros(4), 1e-5),
              lambda: q.I8Weight(torch.zeros(1, 2, 4, 16, 16, dtype=torch.int8), torch.zeros(4), 4, 4),
              lambda: q.I8Tokens(torch.zeros(4, 128, dtype=torch.int8), torch.zeros(4), 4),
              lambda: q.I8Tokens.empty(4, 0, device="cpu")):
        with pytest.raises(ValueError):
            f()


@pytest.mark.parametrize("device", ["cpu", "meta"])
def test_room_for_tokens_is_on_the_gpu(device):
    """Tokens of host memory would be given to a kernel."""
    with pytest.raises(ValueError, match="GPU"):
        q.I8Tokens.empty(4, 64, device=device)


def test_merge_takes_i8_by_name():
    with pytest.raises(ValueError, match="fp32 merge"):
        q.merge_adapter(torch.zeros(4, 4), None, None, 1.0, out_f32=False, requantize="i8")
    with pytest.raises(ValueError, match="I8"):
        q.merge_adapter(torch.zeros(4, 4), None, None, 1.0, requantize="I8")
