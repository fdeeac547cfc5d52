"""The slots of a page that a cache write fills, as the kernels compute them
(compiled for the host), against integers without a limit: every position of 32
bits, up to the page numbers that a call can reach."""
from __future__ import annotations

import ctypes
import itertools
import shutil
import subprocess
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parents[1] / "gated_delta_rule_40_amd" / "csrc"

SHIM = """
#include "kv_slots.hpp"
extern "C" void slots(int pos, int n, long long page_no, int page, int* out) {
  const gdr::KvSlots s = gdr::kv_slots(pos, n, page_no, page);
  out[0] = s.u; out[1] = s.w; out[2] = s.had; out[3] = s.first;
}
"""


@pytest.fixture(scope="module")
def slots(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("slots")
    (d / "shim.cpp").write_text(SHIM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-Wall", "-Werror", f"-I{CSRC}",
                    str(d / "shim.cpp"), "-o", str(d / "shim.so")], check=True)
    lib = ctypes.CDLL(str(d / "shim.so"))
    lib.slots.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_longlong, ctypes.c_int,
                          ctypes.POINTER(ctypes.c_int)]

    def call(pos, n, page_no, page):
        out = (ctypes.c_int * 4)()
        lib.slots(pos, n, page_no, page, out)
        return tuple(out)
    return call


LO, HI = -2 ** 31, 2 ** 31 - 1
POS = [LO, LO + 1, LO + 15, LO + 16, LO + 2000, -2001, -17, -16, -2, -1, 0, 1, 15, 16, 17, 1000,
       HI - 128, HI - 1, HI]


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("n", [0, 1, 2, 16, 33, 2047, HI])
def test_slots(slots, n, page):
    for pos, j in itertools.product(POS, (0, 1, 2, 3, 15, 128, 2 ** 24)):
        page_no = max(pos, 0) // page + j
        base = page_no * page
        lo, hi = max(pos, base), min(pos + n, base + page)
        u, w, had, first = slots(pos, n, page_no, page)
        if hi <= lo:
            assert u >= w, (pos, j)
            continue
        assert (u, w) == (lo - base, hi - base) and 0 <= u < w <= page, (pos, j)
        assert had == (u if pos > base else 0) and first == lo - pos, (pos, j)
        assert 0 <= first and first + (w - u) <= n
