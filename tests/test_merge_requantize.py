"""What merge_adapter's ``requantize`` takes (CPU: the checks come before
anything is done)."""

import pytest

torch = pytest.importorskip("torch")
import bit_quantized_lora_03_amd as q  # noqa: E402


def refused(value, out_f32=False):
    with pytest.raises(ValueError) as e:
        q.merge_adapter(torch.zeros(4, 4), None, None, 1.0, out_f32=out_f32, requantize=value)
    return str(e.value)


@pytest.mark.parametrize("value", [True, 1, "nf4", "u4"])
def test_formats_need_the_fp32_merge(value):
    assert refused(value) == "requantize needs the fp32 merge"


@pytest.mark.parametrize("value", ["U4", "other"])
def test_other_texts_are_refused(value):
    assert "requantize" in refused(value) and value in refused(value, out_f32=True)


@pytest.mark.parametrize("value", [False, 0, None, ""])
def test_nothing_is_quantised(monkeypatch, value):
    """As false values always were taken, an empty text among them."""
    from types import SimpleNamespace
    from bit_quantized_lora_03_amd import _lib
    monkeypatch.setattr(_lib, "lib", lambda: SimpleNamespace(qlora_merge_adapter=lambda *a: 0))
    monkeypatch.setattr(_lib, "_stream_ptr", lambda: 0)
    f, b, w = q.merge_adapter(torch.zeros(4, 4), None, None, 1.0, requantize=value)
    assert f.shape == b.shape == (4, 4) and w is None


@pytest.mark.gpu
def test_nf4_by_its_name(cuda):
    w = torch.randn(128, 256, device="cuda")
    A, B = (torch.zeros(s, dtype=torch.int16, device="cuda") for s in ((8, 256), (128, 8)))
    (f, b, x), (f2, b2, y) = (q.merge_adapter(w, A, B, 16.0, requantize=v) for v in (True, "nf4"))
    assert torch.equal(f, f2) and torch.equal(b, b2)
    for n in ("codes", "qscale", "dq_step"):
        assert torch.equal(getattr(x, n), getattr(y, n)), n
