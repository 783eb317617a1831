"""Whether rows share memory (csrc/rows_overlap.h), compiled for the host and
compared with a look at every byte."""
import ctypes
import itertools
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SHIM = """
#include "rows_overlap.h"
extern "C" int share(int64_t a, int64_t a_row, int64_t a_stride, int64_t b, int64_t b_row, int64_t b_stride, int64_t n) {
    const minisgl::Rows x = {reinterpret_cast<const void *>(a), a_row, a_stride};
    const minisgl::Rows y = {reinterpret_cast<const void *>(b), b_row, b_stride};
    return minisgl::rows_overlap(x, y, n);
}
"""


@pytest.fixture(scope="module")
def share(tmp_path_factory):
    d = tmp_path_factory.mktemp("rows")
    (d / "rows.cc").write_text(SHIM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "paged_kv_cache_row_gb300", "csrc"), str(d / "rows.cc"), "-o",
                    str(d / "rows.so")], check=True)
    f = ctypes.CDLL(str(d / "rows.so")).share
    f.argtypes = [ctypes.c_int64] * 7
    return f


def rows(base, row, stride, n):
    return {base + i * stride + c for i in range(n) for c in range(row)}


@pytest.mark.parametrize("n", [1, 2, 3, 5])
def test_every_small_case(share, n):
    for a_row, a_gap, b_row, b_gap in itertools.product((1, 2, 3), (0, 1, 4), (1, 2, 4), (0, 2, 3)):
        a_stride, b_stride = a_row + a_gap, b_row + b_gap
        a = rows(100, a_row, a_stride, n)
        for base in range(100 - n * b_stride - 2, 100 + n * a_stride + 3):
            want = bool(a & rows(base, b_row, b_stride, n))
            assert share(100, a_row, a_stride, base, b_row, b_stride, n) == want, (a_row, a_stride, base, b_row, b_stride)


def test_slices_of_a_projections_output(share):
    """q, q_out and k of 4 KB, 4 KB and 1 KB in rows of 9 KB, a quarter of a million of them, and one byte too near."""
    base, n, row = 1 << 40, 1 << 18, 9216
    assert not share(base, 4096, row, base + 4096, 4096, row, n) and not share(base + 4096, 4096, row, base, 4096, row, n)
    assert not share(base, 4096, row, base + 8192, 1024, row, n)
    assert share(base, 4096, row, base + 4095, 4096, row, n) and share(base, 4096, row, base + 9215, 2, row, n)
    # the same buffer, rows further apart on one side
    assert share(base, 4096, row, base + 4096, 4096, 2 * row + 16, n)
    assert not share(base, 4096, row, base + 4096, 4096, 2 * row, n)
    assert not share(base, 4096, row, base + n * row, 4096, row, n) and share(base, 4096, row, base, 4096, 4096, n)
