"""Range checks of the positions that a caller hands the paged kernels on the device.

The kernels decide with positions_fit whether a table entry is read; here the same function runs on
the host, for starts up to the ends of the 64-bit range.
"""

import ctypes
import os
import subprocess

import pytest

from tests.test_build_resources import CSRC, NVCC
from tests.test_build_resources import pytestmark as needs_nvcc

pytestmark = needs_nvcc

SOURCE = """
#include "swa_paged.cuh"
extern "C" int fits(int64_t start, int64_t n, int64_t max_pos) {
  return swa::positions_fit(start, n, max_pos);
}
"""
LAST = (1 << 63) - 1


@pytest.fixture(scope="module")
def fits(tmp_path_factory):
    where = tmp_path_factory.mktemp("positions")
    src, lib = where / "fits.cu", where / "fits.so"
    src.write_text(SOURCE)
    res = subprocess.run([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-O3",
                          "-I", CSRC, "-Xcompiler", "-fPIC", "-shared", "-o", str(lib), str(src)],
                         capture_output=True, text=True, timeout=600)
    assert res.returncode == 0, res.stderr[-2000:]
    fn = ctypes.CDLL(os.fspath(lib)).fits
    fn.argtypes = [ctypes.c_int64] * 3
    return fn


@pytest.mark.parametrize("max_pos", [8, 4096, (1 << 31) - 1025])
def test_positions_fit(fits, max_pos):
    starts = [-LAST - 1, -LAST, -1, 0, 1, max_pos - 1, max_pos, max_pos + 1, 1 << 31, 1 << 32,
              LAST - max_pos, LAST - 7, LAST - 1, LAST]
    for start in starts:
        for n in (0, 1, 2, 7, max_pos - 1, max_pos, max_pos + 1, (1 << 31) - 257, LAST):
            want = 0 <= start and start + n <= max_pos  # Python integers do not wrap
            assert bool(fits(start, n, max_pos)) == want, (start, n)
