"""Launches of the microscaled operators at the ends of the documented range
of sizes (up to 2^31 - 1): every grid holds between one and 2^32 - 1
work-items and covers the whole matrix.  CPU only (tests/mx_dry_run.py)."""
import shutil

import pytest

from dense_gemm_row_amd import gemm
from tests.mx_dry_run import compile_dry
from tests.mx_sizes import LARGE_GRADS, LARGE_PRODUCTS

TOP = 2 ** 31 - 1
F32, F16, BF16 = gemm.DTYPE_F32, gemm.DTYPE_F16, gemm.DTYPE_BF16
A, AS, B, BS, C, X, W = (i << 50 for i in range(1, 8))  # never dereferenced


def up(n, d):
    return -(-n // d)


def whole(n, d):
    return up(n, d) * d


@pytest.fixture(scope="module")
def dry(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    return compile_dry(str(tmp_path_factory.mktemp("dry")))


def launched(dry, name, *args):
    status, launches = dry(name, *args)
    assert status == gemm.GEMM_OK and launches
    for one in launches:
        items = one.grid[0] * one.block, one.grid[1]
        assert 0 < items[0] < 2 ** 32 and 0 < items[1] < 2 ** 16, (one.name, tuple(one.grid), one.block)
    return launches


def product(dry, m, n, k, lds, c_dtype=BF16):
    ldq = up(k, 32) * 16
    return launched(dry, "gemm_mx_matmul", c_dtype, m, n, k, A, ldq, AS, lds, B, ldq, BS, lds, C, n, None, None)


FAR = [TOP, TOP - 30, TOP - 31, TOP - 126, TOP - 127, TOP - 254, TOP - 255, 2 ** 30, 2 ** 30 + 1]


@pytest.mark.parametrize("lds", [3, 4, 16])
@pytest.mark.parametrize("far", FAR)
@pytest.mark.parametrize("near", [1, 17, 300])
def test_products_of_far_sizes(dry, far, near, lds):
    for m, n in ((far, near), (near, far)):
        one, = product(dry, m, n, 32, lds)
        bm, bn = (16, 16) if m <= 16 else (64, 64)
        if one.kernel == "matmul_skinny":
            assert m <= 16 and one.grid[0] == up(n, 16)
        elif one.kernel == "matmul_pipe":
            assert one.grid[0] in (up(m, s) * up(n, s) for s in (128, 256))
        else:
            assert one.arg[0] == up(n, bn) and one.arg[1] == up(m, bm) * up(n, bn)
            assert one.grid[0] == min(one.arg[1], 1 << 22)


@pytest.mark.parametrize("n", [2 ** 26 - 17, 2 ** 26 - 16, 2 ** 26 - 15, 2 ** 26 - 1, 2 ** 26, 2 ** 26 + 1])
@pytest.mark.parametrize("k", [4096, 4097])
def test_few_rows_and_very_many_columns(dry, n, k):
    one, = product(dry, 16, n, k, whole(up(k, 32), 4))
    assert one.grid[0] >= min(up(n, 16), 1 << 22)


@pytest.mark.parametrize("n", [2 ** 26 - 16, 2 ** 26 - 15, 2 ** 26])
def test_few_rows_of_values_and_very_many_columns(dry, n):
    """The documented border: one launch without a workspace up to it."""
    k = 8192
    args = (BF16, BF16, 16, n, k, X, k, B, k // 2, BS, k // 32, C, n)
    if n <= 2 ** 26 - 16:
        one, = launched(dry, "gemm_mx_matmul_values", *args, None, 0, None, None)
        assert one.kernel == "matmul_skinny" and one.grid[0] == up(n, 16)
    else:
        assert dry("gemm_mx_matmul_values", *args, None, 0, None, None) == (gemm.GEMM_ERR_INVALID_ARG, [])
        first, second = launched(dry, "gemm_mx_matmul_values", *args, W, 1 << 20, None, None)
        assert first.kernel == "quantize_rows" and second.kernel == "matmul_direct"


@pytest.mark.parametrize("name, step", [("gemm_mx_quantize", 32), ("gemm_mx_dequantize", 8)])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("far", FAR)
def test_rows_and_columns_of_far_sizes(dry, name, step, dtype, pad, far):
    for rows, cols in ((1, far), (3, far), (far, 1), (far, 33)):
        for trans in (0, 1):
            coded = whole(rows, 32) if trans else whole(cols, 32)
            ldx = cols + pad
            x, codes = (X, ldx), (A, coded, AS, coded // 32)
            launches = launched(dry, name, dtype, 1, trans, rows, cols, *(x + codes if "_mx_q" in name else codes + x), None)
            covered = 0
            for one in launches:
                if trans:
                    blocks, tiles_x = one.arg[0], one.arg[1]
                    rb, span = (4, 64 * (16 // (4 if dtype == F32 else 2))) if ldx * (4 if dtype == F32 else 2) % 16 == 0 else (1, 256)
                    assert tiles_x == up(cols, span) and one.grid[0] == tiles_x * up(blocks, rb)
                    covered += 32 * blocks
                else:
                    chunks, width, tiles_x = one.arg[0], 1 << one.arg[1], one.arg[2]
                    assert chunks == (up(cols, 32) * 4 if step == 32 else up(cols, 8))
                    unroll = up(chunks, tiles_x * width)
                    assert unroll in (1, 2, 3, 4) and one.grid[0] % tiles_x == 0
                    covered += one.grid[0] // tiles_x * (256 // width)
            assert covered >= rows


@pytest.mark.parametrize("far", FAR)
def test_gradients_of_far_sizes(dry, far):
    for t, f, n in ((1, far, 3), (1, 3, far), (64, far, 3), (64, 3, far), (far, 3, 3)):
        nb = up(t, 32)
        one, = [k for k in launched(dry, "gemm_mx_wgrad", BF16, F32, t, f, n, A, 32 * nb, AS, whole(nb, 4), X, n, C, n, 1.0, 0.0,
                                    None, 0, None)]
        assert one.kernel == "wgrad_general"
        assert one.arg[0] == up(n, 64) and one.arg[1] == up(n, 64) * up(f, 64)
        assert one.grid[0] == min(one.arg[1], 1 << 22)


@pytest.mark.parametrize("m, n, k", LARGE_PRODUCTS)
@pytest.mark.parametrize("lds", [4, 16])
def test_large_tile_of_products(dry, m, n, k, lds):
    one, = product(dry, m, n, k, whole(up(k, 32), 16) + lds % 16)
    assert one.kernel == "matmul_pipe" and f"ELi{lds}EEE" in one.name.decode()
    assert one.grid[0] == up(m, 256) * up(n, 256)


@pytest.mark.parametrize("t, f, n", LARGE_GRADS)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_large_tile_of_gradients(dry, t, f, n, dtype):
    chunks = LARGE_GRADS[t, f, n][dtype != BF16]
    need = dry.lib.gemm_mx_wgrad_workspace_bytes(dtype, t, f, n)
    launches = launched(dry, "gemm_mx_wgrad", dtype, F32, t, f, n, A, whole(t, 32), AS, whole(up(t, 32), 4), X, n, C, n, 1.0, 0.0,
                        W, need, None)
    pipe = [one for one in launches if one.kernel == "wgrad_pipe"][0]
    assert ("Li256ELi256" in pipe.name.decode()) == (chunks > 0)
    if chunks:
        assert tuple(pipe.grid) == (up(f, 256) * up(n, 256), chunks)
        assert (launches[-1].kernel == "reduce_partials") == (chunks > 1)
    assert (launches[0].kernel == "split_planes") == (dtype != BF16 or n % 8 != 0)
