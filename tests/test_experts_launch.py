"""Launches of the grouped and 4-bit products on the CPU: which kernel takes
which operands, and grids at the ends of the documented ranges.
(tests/experts_dry_run.py)"""
import shutil

import pytest

from dense_gemm_row_amd import gemm, w4
from tests.experts_dry_run import compile_dry, kernel, tile
from tests.experts_sizes import GRADIENTS, PRODUCTS

TOP = 2 ** 31 - 1
F32, F16, BF16 = gemm.DTYPE_F32, gemm.DTYPE_F16, gemm.DTYPE_BF16
O, X, W, Y, Q, S, Z, K = (i << 52 for i in range(1, 9))  # never dereferenced


def whole(n, d):
    return -(-n // d) * d


@pytest.fixture(scope="module")
def dry(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    return compile_dry(str(tmp_path_factory.mktemp("dry")))


def launched(dry, name, *args):
    status, launches = dry(name, *args)
    assert status == gemm.GEMM_OK, (name, args)
    for one in launches:
        assert 0 < one.grid[0] * one.block < 2 ** 32 and 0 < one.grid[1] < 2 ** 16, (one.name, tuple(one.grid), one.block)
    return launches


def product(dry, T, k, N, G, trans=0, dtype=BF16, c=None, x=X, ldx=None, w=W, ldw=None, stride=None, ldy=None, fill=1):
    ldx, ldw = ldx or max(k, 1), ldw or max(k if trans else N, 1)
    stride = (N if trans else k) * ldw if stride is None else stride
    return launched(dry, "gemm_grouped_matmul", dtype, dtype if c is None else c, trans, G, T, N, k, O, x, ldx, w, ldw, stride, Y,
                    ldy or max(N, 1), fill, None)


def gradient(dry, T, k, N, G, dtype=BF16, c=F32, x=X, ldx=None, ldw=None):
    ldw = ldw or max(N, 1)
    return launched(dry, "gemm_grouped_wgrad", dtype, c, G, T, k, N, O, x, ldx or max(k, 1), Y, max(N, 1), W, ldw, k * ldw, 1.0, 0.0,
                    None)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("shape", PRODUCTS, ids=str)
def test_tiles_of_products(dry, shape, dtype):
    for T, k, N, offsets in PRODUCTS[shape]:
        for trans in (0, 1):
            for c in (dtype, F32):
                one, = product(dry, T, k, N, len(offsets) - 1, trans, dtype, c)
                if shape == 16:
                    assert kernel(one) == "matmul_few", (T, k, N, one.name)
                else:
                    assert kernel(one) == "matmul_pipe" and tile(one) == shape, (T, k, N, one.name)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("shape", GRADIENTS, ids=str)
def test_tiles_of_gradients(dry, shape, dtype):
    for T, k, N, offsets in GRADIENTS[shape]:
        for c in (dtype, F32):
            one, = gradient(dry, T, k, N, len(offsets) - 1, dtype, c)
            assert kernel(one) == "wgrad_pipe" and tile(one) == shape, (T, k, N, one.name)


def test_what_the_general_kernels_take(dry):
    for kw in (dict(dtype=F32), dict(k=65), dict(N=65), dict(x=X + 2), dict(ldx=66), dict(ldx=1 << 20), dict(w=W + 8),
               dict(ldw=68), dict(ldw=1 << 20), dict(stride=64 * 64 + 4), dict(ldy=1 << 20)):
        one, = product(dry, **dict(dict(T=100, k=64, N=64, G=3), **kw))
        assert kernel(one) == "matmul_general", kw
    one, = product(dry, 100, 64, 65, 3, trans=1)  # (columns are rows of W then)
    assert kernel(one) != "matmul_general"
    for kw in (dict(dtype=F32), dict(k=65), dict(N=65), dict(x=X + 2), dict(ldx=66), dict(ldw=1 << 20)):
        one, = gradient(dry, **dict(dict(T=100, k=64, N=64, G=3), **kw))
        assert kernel(one) == "wgrad_general", kw


FAR = [TOP, TOP - 63, TOP - 127, TOP - 255, 2 ** 30, 2 ** 30 + 1, 2 ** 30 - 8]


@pytest.mark.parametrize("far", FAR)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_products_and_gradients_of_far_sizes(dry, far, dtype):
    for T, k, N, G in ((far, 8, 8, 1), (far, 8, 8, 65535), (3, 8, far, 2), (3, 8, whole(far, 8) - 8, 2), (3, far, 8, 2), (1, 8, 8, 65535)):
        for trans in (0, 1):
            product(dry, T, k, N, G, trans, dtype)
        gradient(dry, T, k, N, G, dtype)


def coded(group, k, N, zeros=True, lds=None):
    ng = -(-k // group)
    lds = lds or whole(max(ng, 1), 256 // group)
    ldq = -(-k // 32) * 16
    return w4.GemmW4(Q, ldq, N * ldq, S, lds, N * lds, Z if zeros else None, lds, N * lds, group)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("group", w4.GROUPS)
def test_4_bit_products(dry, group, dtype):
    for M in (1, 16, 17, 33, 64, 128):
        one, = launched(dry, "gemm_w4_matmul", dtype, M, 136, 512, X, 512, coded(group, 512, 136), Y, 136, None, 0, None)
        assert kernel(one) == "matmul_few"
    one, two = launched(dry, "gemm_w4_matmul", dtype, 129, 136, 512, X, 512, coded(group, 512, 136), Y, 136, K, 1 << 20, None)
    assert kernel(one) == "dequantize_rows" and kernel(two) == ("gemm_bf16_bt" if dtype == BF16 else "gemm_f16_bt")
    for x, ldx, k in ((X + 2, 512, 512), (X, 513, 512), (X, 512, 511)):  # rows that do not begin on 16 bytes
        one, two = launched(dry, "gemm_w4_matmul", dtype, 300, 136, k, x, ldx, coded(group, k, 136), Y, 136, K, 1 << 20, None)
        assert kernel(one) == "dequantize_rows" and kernel(two) == "matmul_general"
        one, = launched(dry, "gemm_w4_matmul", dtype, 16, 136, k, x, ldx, coded(group, k, 136), Y, 136, None, 0, None)
        assert kernel(one) == "matmul_few"
    one, two = launched(dry, "gemm_w4_matmul", dtype, 300, 149, 512, X, 512, coded(group, 512, 149), Y, 149, K, 1 << 20, None)
    assert kernel(one) == "dequantize_rows" and kernel(two) in ("matmul_pipe", "matmul_few")
    one, two = launched(dry, "gemm_w4_grouped", dtype, 2, 257, 136, 512, O, X, 512, coded(group, 512, 136), Y, 136, 1, K, 1 << 20,
                        None)
    assert kernel(one) == "dequantize_rows" and one.grid[1] == 2 and kernel(two) in ("matmul_pipe", "matmul_few")


@pytest.mark.parametrize("far", FAR)
@pytest.mark.parametrize("group", w4.GROUPS)
def test_4_bit_products_of_far_sizes(dry, far, group):
    k = min(far, 2 ** 30)
    for N, kk in ((far, 64), (3, k), (far, 63), (3, k - 3)):
        one, = launched(dry, "gemm_w4_matmul", BF16, 16, N, kk, X, kk, coded(group, kk, N), Y, N, None, 0, None)
        assert one.grid[0] >= min(-(-N // 128), 1 << 22)
        for trans in (0, 1):
            launched(dry, "gemm_w4_quantize", BF16, BF16, trans, N, kk, X, N if trans else kk, coded(group, kk, N), None)
        launched(dry, "gemm_w4_dequantize", F32, BF16, N, kk, coded(group, kk, N), X, kk, None)
    for G, T in ((65535, 65535 * 128), (65535, 1), (1, 128)):
        launched(dry, "gemm_w4_grouped", BF16, G, T, 264, 512, O, X, 512, coded(group, 512, 264), Y, 264, 1, None, 0, None)
