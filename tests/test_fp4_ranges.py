"""The index arithmetic of the MXFP4 kernels (csrc/fp4_ranges.hpp) at the ends of its range, compiled for
the host and compared with Python's unbounded integers."""
import ctypes
import os
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mxfp8_block_scaled_03_amd", "csrc")
SHIM = """
#include "fp4_ranges.hpp"
extern "C" {
int column_groups(int n) { return mxq::column_groups(n); }
int whole_group(int col, int n) { return mxq::whole_group(col, n); }
void grid_of(int64_t n, uint32_t out[2]) { const mxq::Grid g = mxq::grid_of(n); out[0] = g.x; out[1] = g.y; }
int64_t workgroup_at(uint32_t x, uint32_t y) { return mxq::workgroup_at(x, y); }
uint32_t scale_bytes(int64_t rows, int64_t ld, int nb, int words) { return mxq::scale_bytes(rows, ld, nb, words); }
}
"""
TOP = 2 ** 31 - 1


@pytest.fixture(scope="module")
def ranges(tmp_path_factory):
    d = tmp_path_factory.mktemp("ranges")
    (d / "shim.cpp").write_text(SHIM)
    # -fwrapv: an overflow wraps, as it does on the GPU, instead of leaving the compiler free
    subprocess.run(["g++", "-O1", "-std=c++17", "-fwrapv", "-shared", "-fPIC", "-I", CSRC, str(d / "shim.cpp"), "-o",
                    str(d / "shim.so")], check=True)
    return ctypes.CDLL(str(d / "shim.so"))


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8, 1000, 2 ** 24 + 1, TOP - 4, TOP - 3, TOP - 2, TOP - 1, TOP])
def test_column_groups(ranges, n):
    groups = -(-n // 4)
    assert ranges.column_groups(n) == groups
    for col in {0, 4 * (groups // 2), 4 * max(groups - 2, 0), 4 * (groups - 1)}:
        assert ranges.whole_group(col, n) == (col + 4 <= n), col


@pytest.mark.parametrize("n", [1, 2, 255, 2 ** 20 + 1, 2 ** 22 - 1, 2 ** 22, 2 ** 22 + 1, 3 * 2 ** 22, 2 ** 24, 2 ** 26 + 5, TOP])
def test_grid(ranges, n):
    """Every number below n exactly once (the rows of the grid are whole but for the last), below 2^32
    threads along x and 2^16 workgroups along y, the launch's limits, at up to 512 threads a workgroup."""
    ranges.workgroup_at.restype = ctypes.c_int64
    out = (ctypes.c_uint32 * 2)()
    ranges.grid_of(ctypes.c_int64(n), out)
    x, y = out
    assert 1 <= x and x * 512 < 2 ** 32 and 1 <= y < 2 ** 16
    assert x * (y - 1) < n <= x * y
    for c, r in ((0, 0), (x - 1, 0), (0, y - 1), (x - 1, y - 1), (x // 2, y // 2)):
        assert ranges.workgroup_at(c, r) == r * x + c


@pytest.mark.parametrize("rows,ld,nb", [(1, 1, 1), (16, 5, 5), (11, 5, 5), (3, 7, 6), (9, 21, 18), (64, 2 ** 24 - 1, 2 ** 19)])
def test_scale_bytes(ranges, rows, ld, nb):
    """Read byte by byte, scales end with the last row's last one, wherever that lies; read by words (rows
    that are whole 4-byte words apart), with the word that holds it."""
    ranges.scale_bytes.restype = ctypes.c_uint32
    args = ctypes.c_int64(rows), ctypes.c_int64(ld), nb
    assert ranges.scale_bytes(*args, 0) == (rows - 1) * ld + nb
    ld = -(-ld // 4) * 4
    assert ranges.scale_bytes(args[0], ctypes.c_int64(ld), nb, 1) == -(-((rows - 1) * ld + nb) // 4) * 4
