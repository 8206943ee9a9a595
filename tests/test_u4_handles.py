"""Calls read the tensors that a 4-bit weight or cache holds when they are
made, not those that it held once (CPU; where the tensors are is not looked at
here)."""

import pytest

torch = pytest.importorskip("torch")
from bit_quantized_lora_03_amd import u4  # noqa: E402

u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)      # noqa: E731
b16 = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731


@pytest.fixture
def handles(monkeypatch):
    monkeypatch.setattr(u4, "_dense", lambda *a: None)
    return (u4.U4Weight(u8(8, 64), b16(8, 2, 2)),
            u4.Kv4Cache(u8(3, 2, 16, 32), b16(3, 2, 16, 2), u8(3, 2, 16, 32), b16(3, 2, 16, 2)))


def names(h):
    return ("codes", "pairs") if isinstance(h, u4.U4Weight) else \
        ("k_codes", "k_pairs", "v_codes", "v_pairs")


def test_tensors_exchanged_or_moved(handles):
    for h in handles:
        before = h.struct
        assert h.now() is before
        for name in names(h):
            for move in (False, True):
                t = getattr(h, name)
                if move:
                    t.data = t.data.clone()
                else:
                    setattr(h, name, t.clone())
                now = h.now()
                for n in names(h):
                    assert getattr(now, n) == getattr(h, n).data_ptr(), (name, n)
                assert h.now() is now


def test_exchanged_tensors_are_checked(handles):
    w, c = handles
    w.codes = u8(4, 32)
    with pytest.raises(ValueError):
        w.now()
    w.pairs = b16(4, 1, 2)
    assert (w.now().N, w.now().K, w.N, w.K, w.group) == (4, 64, 4, 64, 64)
    c.v_codes = u8(2, 2, 16, 32)
    for _ in range(2):                               # not only the first time
        with pytest.raises(ValueError):
            c.now()
    for n in ("k_codes", "v_codes"):
        setattr(c, n, u8(2, 2, 16, 64))
    for n in ("k_pairs", "v_pairs"):
        setattr(c, n, b16(2, 2, 16, 2))
    assert (c.now().pages, c.pages, c.now().head_dim, c.head_dim) == (2, 2, 128, 128)


def test_views_at_the_same_place(handles):
    w, c = handles
    w.codes, w.pairs = w.codes[:3], w.pairs[:3]
    assert (w.now().N, w.N) == (3, 3)
    for n in names(c):
        setattr(c, n, getattr(c, n)[:1])
    assert (c.now().pages, c.pages) == (1, 1)
