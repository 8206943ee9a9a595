"""What the source of the 4-bit kernels has to say for itself (CPU only)."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "bit_quantized_lora_03_amd", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(text, head):
    """The braces that follow ``head``, with what is in them."""
    at = text.index(head)
    assert text.find(head, at + 1) < 0, head
    start = text.index("{", at + len(head) - 1)
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i + 1]
    raise AssertionError(head)


def events(text):
    """Writes (w) and reads (r) of a wave's stage and the exchanges (e) between
    them, in order."""
    kinds = [("e", r"wave_exchange\(\)"), ("w", r"st\.[\w.]+(?:\[[^\n=;]*\])+ = "), ("r", r"st\.[\w.]+")]
    found, text = "", text
    for m in re.finditer("|".join(f"(?P<{k}>{p})" for k, p in kinds), text):
        found += m.lastgroup
    return found


def test_lanes_of_a_wave_exchange_values_in_order():
    """Lanes read what other lanes wrote to the wave's stage: an exchange
    stands between any write and the reads before and behind it, so no
    compiler may move them past each other."""
    text = source("u4_linear.hip")
    # the codes' place is also x's, and X is read by the tiles' work
    assert re.fullmatch(r"e(w+er+e)w", events(body(text, "auto order_x = [&] {")))
    assert re.fullmatch(r"ew+e", events(body(text, "auto store_w = [&] {")))
    assert re.fullmatch(r"r+", events(body(text, "auto work = [&](int u, int r, bool first, bool all) {")))
    walk = text[text.index("if (u0 < u1) {"):]
    calls = re.findall(r"\b(order_x|store_w|work)\(", walk)
    assert calls[:2] == ["order_x", "store_w"] and set(calls[2:]) == {"work"}


def test_no_variant_is_compiled_that_no_call_reaches():
    """Groups of 32 take 8 waves or fewer, so the product's 16-wave variants
    are instantiated for larger groups only."""
    pick = body(source("u4_linear.hip"), "void pick(const uint8_t* codes")
    wide = body(pick, "if constexpr (G > 32) ")
    uses = re.findall(r"QLORA_U4_GO\(1, 1, \d, 16,", pick)
    assert uses and uses == re.findall(r"QLORA_U4_GO\(1, 1, \d, 16,", wide)
