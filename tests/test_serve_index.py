"""The index arithmetic of the cache kernels (csrc/q4_kv.h) compiled for the
host: whatever the device-side tables hold, every page that a kernel would
touch lies inside the cache and every token inside the inputs."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "bit_weight_only_int4_amd", "csrc")

SHIM = """
#include "q4_kv.h"
extern "C" {
void span(const int32_t* cu, const int32_t* len, int64_t b, int64_t T, int32_t* out) {
  const q4::SeqSpan s = q4::seq_span(cu, len, b, T);
  out[0] = s.t0; out[1] = s.n; out[2] = s.len; out[3] = s.pos0;
}
int32_t page(const int32_t* row, int64_t max_pages, int64_t pages, int64_t index) {
  return q4::page_at(row, max_pages, pages, index);
}
int64_t touched(int64_t n, int64_t page) { return q4::pages_touched(n, page); }
void keys(int64_t lo, int64_t hi, int64_t window, int64_t max_len, int64_t* out) {
  const q4::KeyRange r = q4::key_range(lo, hi, window, max_len);
  out[0] = r.lo; out[1] = r.hi;
}
}
"""


@pytest.fixture(scope="module")
def shim(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("kv")
    (d / "shim.cpp").write_text(SHIM)
    so = d / "shim.so"
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", f"-I{CSRC}", str(d / "shim.cpp"),
                    "-o", str(so)], check=True)
    L = ctypes.CDLL(str(so))
    I = ctypes.c_int64
    L.span.argtypes = [ctypes.c_void_p, ctypes.c_void_p, I, I, ctypes.c_void_p]
    L.page.argtypes = [ctypes.c_void_p, I, I, I]
    L.page.restype = ctypes.c_int32
    L.touched.argtypes = [I, I]
    L.touched.restype = I
    L.keys.argtypes = [I, I, I, I, ctypes.c_void_p]
    L.keys.restype = None
    return L


def i32(*v):
    return np.array(v, dtype=np.int32)


def test_spans_stay_inside_the_inputs(shim):
    big = (1 << 31) - 1
    for cu, n, T, want in (
            (i32(0, 3), i32(10), 3, (0, 3, 10, 7)), (i32(0, 3), i32(2), 3, (0, 3, 2, -1)),
            (i32(0, 4), i32(10), 3, (0, 0, 10, 10)), (i32(-1, 3), i32(10), 3, (0, 0, 10, 10)),
            (i32(2, 1), i32(10), 3, (0, 0, 10, 10)), (i32(0, 3), i32(-7), 3, (0, 3, 0, -3)),
            (i32(1, big), i32(big), 3, (0, 0, big, big)), (i32(3, 3), i32(0), 3, (3, 0, 0, 0))):
        out = np.zeros(4, np.int32)
        shim.span(cu.ctypes.data, n.ctypes.data, 0, T, out.ctypes.data)
        assert tuple(out) == want, (cu, n)


def test_pages_are_in_the_cache_or_none(shim):
    big = (1 << 31) - 1
    row = i32(0, 5, 6, -1, big, -big - 1, 2)
    for index, want in ((0, 0), (1, 5), (2, -1), (3, -1), (4, -1), (5, -1), (6, 2), (7, -1), (-1, -1),
                        (1 << 40, -1)):
        assert shim.page(row.ctypes.data, 7, 6, index) == want, index


def test_pages_touched_is_the_most_any_start_gives(shim):
    for page in (16, 32, 64, 128):
        for n in list(range(0, 40)) + [63, 64, 65, 127, 128, 129, 1000]:
            want = max((s + n - 1) // page + 1 for s in range(page)) if n else 0
            assert shim.touched(n, page) == want, (n, page)


def test_key_ranges(shim):
    for lo, hi, window, most, want in (
            (9, 12, 0, 100, (0, 13)), (9, 12, 4, 100, (6, 13)), (-3, -1, 0, 100, (0, 0)),
            (-3, 2, 2, 100, (0, 3)), (9, 12, 0, 5, (0, 5)), (90, 120, 10, 50, (50, 50))):
        out = np.zeros(2, np.int64)
        shim.keys(lo, hi, window, most, out.ctypes.data)
        assert tuple(out) == want
