"""What the launches of the grouped and 4-bit products pass to their kernels at
the ends of the documented ranges, on the CPU.  (tests/experts_dry_run.py)"""
import re
import shutil
import subprocess

import pytest

from dense_gemm_row_amd import gemm, w4
from tests import experts_dry_run
from tests.experts4_sizes import READS, SHAPES
from tests.mx_dry_run import STAND_IN

TOP = 2 ** 31 - 1
F32, F16, BF16 = gemm.DTYPE_F32, gemm.DTYPE_F16, gemm.DTYPE_BF16
O, X, W, Y, Q, S, Z = (i << 52 for i in range(1, 8))  # never dereferenced


@pytest.fixture(scope="module")
def dry(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    first = '{"matmul_direct", "48"}'
    assert first in STAND_IN
    with pytest.MonkeyPatch.context() as m:  # (records the kernels' tiles and columns of tiles too)
        m.setattr(experts_dry_run, "STAND_IN", STAND_IN.replace(first, first + ', {"matmul_few", "44"}'))
        return experts_dry_run.compile_dry(str(tmp_path_factory.mktemp("dry")))


def coded(group, K, N):
    ng = -(-K // group)
    ldq = -(-K // 32) * 16
    return w4.GemmW4(Q, ldq, N * ldq, S, ng, N * ng, Z, ng, N * ng, group)


def shape_of(name):
    """(k of a scale, blocks of 16 rows, waves along k, waves) of the kernel for few rows."""
    gb, mb, nb, kw, waves = map(int, re.search(r"5ShapeILi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)ELi(\d+)E", name).groups())
    assert nb == 1
    return gb, mb, kw, waves


def shape(launch):
    return shape_of(launch.name.decode())


def kernel_names(dry):
    """Every kernel that the library registers."""
    return subprocess.run(["strings", "-n", "20", dry.lib._name], check=True, capture_output=True, text=True).stdout.split()


@pytest.mark.parametrize("group", w4.GROUPS)
@pytest.mark.parametrize("N", [TOP, TOP - 1, TOP - 31, TOP - 63, TOP - 127, TOP - 128])
def test_columns_of_tiles_of_4_bit_products(dry, N, group):
    """Two experts of a row each, and dense products: a tile's columns are
    counted without leaving 31 bits."""
    for call in [("gemm_w4_grouped", BF16, 2, 2, N, 32, O, X, 32, coded(group, 32, N), Y, N, 0, None, 0, None)] + [
            ("gemm_w4_matmul", BF16, M, N, K, X, K, coded(group, K, N), Y, N, None, 0, None)
            for M in (1, 16, 17, 40, 128) for K in (32, 256)]:
        status, launches = dry(*call)
        assert status == gemm.GEMM_OK and len(launches) == 1
        _, mb, kw, waves = shape(launches[0])
        rows = 2 if call[0] == "gemm_w4_grouped" else -(-call[2] // (16 * mb))
        cols = -(-N // (16 * (waves // kw)))
        assert launches[0].arg[1] == cols and launches[0].arg[0] == rows * cols


@pytest.mark.parametrize("group", w4.GROUPS)
@pytest.mark.parametrize("N", [2 ** 28, 2 ** 28 + 1, 2 ** 30, TOP])
def test_grids_of_4_bit_products_of_any_rows(dry, N, group):
    """Fewer than 2^32 work-items, for workgroups of 8 and of 16 waves."""
    sizes = set()
    for M in (1, 33, 40, 48, 64, 128):
        for K in (64, 128, 4096):
            status, (one,) = dry("gemm_w4_matmul", BF16, M, N, K, X, K, coded(group, K, N), Y, N, None, 0, None)
            assert status == gemm.GEMM_OK and one.grid[0] * one.block < 2 ** 32, (M, K, one.name, tuple(one.grid), one.block)
            sizes.add(one.block)
    assert sizes == {512, 1024}


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("group", w4.GROUPS)
@pytest.mark.parametrize("want", SHAPES, ids=str)
def test_shapes_of_4_bit_products(dry, want, group, dtype):
    for rows, N, offsets in SHAPES[want]:
        for reads, ks in READS.items():
            for K in ks:
                q = coded(group, K, N)
                if offsets is None:
                    status, (one,) = dry("gemm_w4_matmul", dtype, rows, N, K, X, K, q, Y, N, None, 0, None)
                else:
                    status, (one,) = dry("gemm_w4_grouped", dtype, len(offsets) - 1, rows, N, K, O, X, K, q, Y, N, 1, None, 0, None)
                got = re.search(r"5ReadsE(\d)E", one.name.decode()).group(1)
                assert status == gemm.GEMM_OK and shape(one) == (group, *want) and int(got) == reads, (rows, N, K, one.name)


def test_every_shape_has_sizes(dry):
    """The kernels that are built, but for the one by element (blocks of one,
    a wave along k), are those of the table."""
    built = {(shape_of(n), int(re.search(r"5ReadsE(\d)E", n).group(1))) for n in kernel_names(dry) if "5Shape" in n}
    assert built == {((group, *s), reads) for s in SHAPES for reads in READS for group in w4.GROUPS} | {
        ((group, 1, 1, 8), 0) for group in w4.GROUPS}
