"""Where a sequence's rows and keys lie, as the device works it out from the
batch's arrays (which the host does not see), compiled for the CPU: whatever
the arrays hold, no row outside the call's tensors and no key outside the
block table comes out."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="needs hipcc")

PROGRAM = """
#include "%s/bit_quantized_lora_03_amd/csrc/kv4_common.h"
using namespace qlora;
// out: row0, n, pos0, then lo, hi, chunk, chunks and [t0, t1) of a chunk
extern "C" void look(const int32_t* cu_q, const int32_t* lens, int64_t rows, int max_q, int b,
                     int64_t table_keys, int causal, int window, int group, int r0, int tile,
                     int chunk, int splits, int split, int64_t* out) {
  Kv4BatchArg bt{};
  bt.cu_q = cu_q; bt.seq_lens = lens; bt.rows = rows; bt.max_q = max_q;
  Kv4AttnArg a{};
  a.causal = causal; a.window = window; a.table_keys = table_keys;
  const Kv4Seq q = kv4_seq(bt, b);
  out[0] = q.row0; out[1] = q.n; out[2] = q.pos0;
  const Span s = kv4_span(q, a, group, r0, tile, chunk, splits);
  out[3] = s.lo; out[4] = s.hi; out[5] = s.chunk; out[6] = s.n;
  out[7] = s.begin(split); out[8] = s.end(split);
}
"""


@pytest.fixture(scope="module")
def look(tmp_path_factory):
    at = tmp_path_factory.mktemp("host")
    (at / "look.hip").write_text(PROGRAM % ROOT)
    subprocess.run([HIPCC, "--offload-host-only", "-std=c++17", "-O1", "-fPIC", "-shared",
                    "-fwrapv", "-o", str(at / "look.so"), str(at / "look.hip")], check=True)
    f = ctypes.CDLL(str(at / "look.so")).look
    i32, i64, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
    f.argtypes = [vp, vp, i64, i32, i32, i64, i32, i32, i32, i32, i32, i32, i32, i32, vp]

    def call(cu, lens, rows, max_q, table_keys, causal, window, group, r0, tile, chunk, splits, split, b=0):
        cu, lens = np.array(cu, np.int32), np.array(lens, np.int32)
        out = np.zeros(9, np.int64)
        f(cu.ctypes.data, lens.ctypes.data, rows, max_q, b, table_keys, causal, window, group, r0,
          tile, chunk, splits, split, out.ctypes.data)
        return dict(zip("row0 n pos0 lo hi chunk chunks t0 t1".split(), map(int, out)))
    return call


TOP = 2 ** 31 - 1
LENS = [-TOP - 1, -5, 0, 1, 16, 100, 4096, 2 ** 30 - 1, 2 ** 30, 2 ** 30 + 17, TOP - 300, TOP - 31, TOP]


@pytest.mark.parametrize("causal", [0, 1])
@pytest.mark.parametrize("window", [0, 1, 33, 4096, 2 ** 30, TOP])
def test_keys_stay_inside_the_table(look, causal, window):
    group, tile = 2, 16
    for length in LENS:
        for table_keys in (0, 16, 4096, 2 ** 30):
            for n in (1, 9):
                i1 = min(tile - 1, n * group - 1) // group
                hi = max(min([length, table_keys] + [length - n + i1 + 1] * causal), 0)
                lo = max(length - n - window + 1, 0) if window else 0
                for chunk, splits in ((256, 1), (256, 7), (2 ** 30 + 128, 1), (2 ** 23, 128)):
                    def ask(split):
                        return look([0, n], [length], 100, 9, table_keys, causal, window, group, 0,
                                    tile, chunk, splits, split)
                    s = ask(0)
                    case = (length, table_keys, n, chunk, splits, s)
                    if lo >= hi:                     # nothing to see, nothing to walk
                        assert s["chunks"] == 0 and 0 <= s["t0"] == s["t1"] <= table_keys, case
                        continue
                    assert 1 <= s["chunks"] <= splits and lo - 32 < s["t0"] <= lo, case
                    at = s["t0"]
                    for split in range(s["chunks"]):
                        s = ask(split)
                        assert s["t0"] == at and at % 32 == 0 and at < s["t1"] <= hi, (case, s)
                        at = s["t1"]
                    assert at == hi, case


def test_rows_stay_inside_the_tensors(look):
    edge = [-TOP - 1, -1, 0, 1, 5, 99, 100, 101, TOP - 1, TOP]
    for first in edge:
        for last in edge:
            for length in LENS:
                # a negative number times the query heads of a KV head can be
                # anything in 32 bits: -(2^31 - 1) rows of 8 heads were 8
                s = look([first, last], [length], 100, 9, 4096, 1, 0, 8, 0, 16, 256, 4, 0)
                assert 0 <= s["n"] <= 9, (first, last, s)
                assert s["n"] == 0 or 0 <= s["row0"] <= 100 - s["n"], (first, last, s)
