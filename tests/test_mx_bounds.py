"""The index arithmetic of the microscaled operators (csrc/mx_bounds.h, the
header the kernels and their launches include), compiled for the CPU and
evaluated there: counts of blocks, and which bytes a load touches.  CPU only."""
import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OOB = 0x80000000

SHIM = """
#include "mx_bounds.h"
using namespace gemm::mx;
extern "C" int64_t blocks(int64_t cols) { return blocks_of(cols); }
extern "C" unsigned value_load_4(int row, int rows, unsigned row_bytes, int c, int left, int h) {
  return value_load<4>(row, rows, row_bytes, c, left, h);
}
extern "C" unsigned value_load_2(int row, int rows, unsigned row_bytes, int c, int left, int h) {
  return value_load<2>(row, rows, row_bytes, c, left, h);
}
"""


def compiled(source, out):
    src = out + ".cc"
    with open(src, "w") as f:
        f.write(source)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", os.path.join(ROOT, "dense_gemm_row_amd", "csrc"),
                    src, "-o", out], check=True)
    return ctypes.CDLL(out)


@pytest.fixture(scope="module")
def bounds(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    lib = compiled(SHIM, str(tmp_path_factory.mktemp("bounds") / "bounds.so"))
    for name in ("value_load_4", "value_load_2"):
        getattr(lib, name).restype = ctypes.c_uint
        getattr(lib, name).argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_uint] + [ctypes.c_int] * 3
    lib.blocks.restype, lib.blocks.argtypes = ctypes.c_int64, [ctypes.c_int64]
    return lib


@pytest.mark.parametrize("cols", [0, 1, 32, 33, 2 ** 31 - 33, 2 ** 31 - 32, 2 ** 31 - 31, 2 ** 31 - 1])
def test_blocks_of_a_row(bounds, cols):
    assert bounds.blocks(cols) == -(-cols // 32)


@pytest.mark.parametrize("size", [2, 4])
@pytest.mark.parametrize("k", list(range(1, 18)) + [31, 33, 511, 512, 513, 516, 1060, 4100, 4108])
def test_values_of_few_rows_are_read_inside_their_matrix(bounds, k, size):
    """Every lane and turn of the product that encodes X's rows: a load that
    is made starts at an existing value, so it stays in that value's aligned
    16 bytes, and every existing value is loaded."""
    load = getattr(bounds, f"value_load_{size}")
    per = 16 // size  # values of a load
    for rows, slack in ((1, 0), (3, 0), (3, 16), (16, 0)):
        row_bytes = -(-k * size // 16) * 16 + slack
        for row in range(16):
            seen = set()
            for chunk in range(64 * (k // 512 + 1)):  # whole turns of 512 columns
                c = 8 * chunk
                for h in range(8 // per):
                    at = load(row, rows, row_bytes, c, k - c, h)
                    first = c + h * per
                    if row < rows and first < k:
                        assert at == row * row_bytes + size * first and at % 16 == 0
                        seen.update(range(first, min(first + per, k)))
                    else:
                        assert at >= OOB, (rows, row, c, h, at)
            assert seen == (set(range(k)) if row < rows else set())
