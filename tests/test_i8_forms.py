"""Which form and tile of the 8-bit products the tests' sizes take, by the
library's own rule: it is compiled for the host from the kernels' source, so a
change of it that leaves a form untested is seen (CPU only)."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest

from tests import test_gpu_i8, test_gpu_i8_extremes, test_gpu_i8_rings as rings

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "bit_quantized_lora_03_amd", "csrc")
SMALL = [(16, 16), (32, 16), (32, 32), (64, 32)]
LARGE = [(32, 128), (64, 128), (128, 128), (128, 256)]
STAGES = {32: 8, 64: 6, 128: 4}  # of the tokens' ring, by the tile's tokens


@pytest.fixture(scope="module")
def form(tmp_path_factory):
    """form(gated, M, N, K) -> the tile's tokens and rows."""
    cxx = shutil.which("g++") or shutil.which("clang++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no host compiler")
    with open(os.path.join(CSRC, "i8_linear.hip")) as f:
        text = f.read()
    start, end = text.index("struct Form {"), text.index("template <class DT, int G, int T, int R>\nvoid go(")
    where = tmp_path_factory.mktemp("rule")
    src, lib = str(where / "rule.cpp"), str(where / "rule.so")
    with open(src, "w") as f:
        f.write("#include <cstdint>\nstruct I8LinearArg { int64_t M, N, K; };\n"
                "static int64_t i8_padded(int64_t K) { return (K + 127) / 128 * 128; }\n"
                + text[start:end] +
                'extern "C" int rule(int gated, int64_t M, int64_t N, int64_t K, int* tile) {\n'
                "  const I8LinearArg p{M, N, K};\n"
                "  const int f = gated ? best_of(kGated, p) : best_of(kPlain, p);\n"
                "  const Form& t = gated ? kGated[f] : kPlain[f];\n"
                "  tile[0] = t.tm, tile[1] = t.tn;\n"
                "  return f >= kSmall;\n}\n")
    subprocess.run([cxx, "-O1", "-shared", "-fPIC", "-o", lib, src], check=True)
    rule = ctypes.CDLL(lib).rule
    rule.argtypes = [ctypes.c_int] + [ctypes.c_int64] * 3 + [ctypes.POINTER(ctypes.c_int)]

    def f(gated, M, N, K):
        tile = (ctypes.c_int * 2)()
        large = rule(gated, M, N, K, tile)
        assert large == (tuple(tile) in LARGE)
        return tuple(tile)
    return f


def sizes_of(test):
    """The (M, N, K) that a test is parametrised with."""
    return next(m.args[1] for m in test.pytestmark
                if m.name == "parametrize" and m.args[0] == "M,N,K")


def test_the_rings_have_as_many_stages_as_said():
    with open(os.path.join(CSRC, "i8_gemm.hip")) as f:
        text = f.read()
    assert re.search(r"ST = JT == 1 \? 8 : JT == 2 \? 6 : 4;", text)
    assert re.search(r"TM = 32 \* JT\b", text)


def test_sizes_for_each_form(form):
    assert [form(0, *s) for s in test_gpu_i8.FORMS] == SMALL + LARGE
    assert [form(1, *s) for s in sizes_of(test_gpu_i8.test_gated_in_every_form)] == SMALL + LARGE[:3]


@pytest.mark.parametrize("gated", [0, 1])
def test_rings_go_round_in_each_large_tile(form, gated):
    """Odd and even numbers of K's tiles, enough for the ring to go round twice
    and more; and the small tiles for sixteen tokens, which they are compared
    with."""
    seen = {}
    for M, N, K in rings.GATED if gated else rings.PLAIN:
        tiles = -(-K // 128)
        tile = form(gated, M, N, K)
        assert tile in LARGE and tiles >= 2 * STAGES[tile[0]], (M, N, K)
        seen.setdefault(tile, set()).add(tiles % 2)
        for few in {16, M % 16 or 16}:
            assert form(gated, few, N, K) in SMALL
    assert seen == {t: {0, 1} for t in (LARGE[:3] if gated else LARGE)}


def test_longest_rows_take_each_large_tile(form):
    assert [form(1, M, N, rings.LONGEST) for M, N in rings.GATED_LONGEST] == LARGE[:3]
    plain = next(m.args[1] for m in test_gpu_i8_extremes.test_longest_rows_in_every_tile.pytestmark
                 if m.name == "parametrize" and m.args[0] == "M,N")
    assert {form(0, M, N, rings.LONGEST) for M, N in plain} >= set(LARGE)
