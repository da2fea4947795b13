"""The product of values with a coded matrix on the host: refusals before any
launch and the workspace's size.  CPU only."""
import pytest

from dense_gemm_row_amd import gemm, mx

PX, PQ, PC, PW = 0x10000000, 0x20000000, 0x30000000, 0x40000000  # never dereferenced
INVALID, UNSUPPORTED, ALIAS = gemm.GEMM_ERR_INVALID_ARG, gemm.GEMM_ERR_UNSUPPORTED, gemm.GEMM_ERR_ALIAS


def values(a=2, c=2, M=32, N=8, K=64, X=PX, ldx=64, B=PQ, ldb=32, Bs=PQ + 4096, ldbs=4, C=PC, ldc=8, ws=PW, nws=1 << 20,
           epi=None):
    return mx.gemm_mx_matmul_values(a, c, M, N, K, X, ldx, B, ldb, Bs, ldbs, C, ldc, ws, nws, None, epi)


@pytest.mark.parametrize("kw, want", [
    (dict(a=3), INVALID), (dict(a=-1), INVALID), (dict(c=4), INVALID), (dict(M=-1), INVALID), (dict(N=-1), INVALID),
    (dict(K=1 << 31), INVALID), (dict(ldx=63), INVALID), (dict(ldb=16), INVALID), (dict(ldbs=1), INVALID),
    (dict(ldc=7), INVALID), (dict(X=0), INVALID), (dict(B=0), INVALID), (dict(Bs=0), INVALID), (dict(C=0), INVALID),
    (dict(nws=-1), INVALID), (dict(epi=gemm.GemmEpilogue(1.0, 0.0, None, 5)), INVALID),
    (dict(ws=None), INVALID), (dict(nws=16), INVALID), (dict(ws=PW + 8), INVALID),
    # Few rows need the workspace too where they are not on whole 16 bytes,
    # or the scales not on whole words.
    (dict(M=4, ws=None, X=PX + 2), INVALID), (dict(M=4, ws=None, ldx=65), INVALID), (dict(M=4, ws=None, ldbs=3), INVALID),
    (dict(M=17, ws=None), INVALID), (dict(M=4, N=1, ws=None, ldb=1 << 26), INVALID),
    (dict(X=PX + 1), UNSUPPORTED), (dict(B=PQ + 8), UNSUPPORTED), (dict(ldb=40), UNSUPPORTED), (dict(C=PC + 1), UNSUPPORTED),
    (dict(C=PX), ALIAS), (dict(C=PQ + 32), ALIAS), (dict(C=PQ + 4096), ALIAS),
    (dict(ws=PX), ALIAS), (dict(ws=PQ), ALIAS), (dict(ws=PC), ALIAS),
    (dict(epi=gemm.GemmEpilogue(1.0, 0.0, PC + 16, 0)), ALIAS),
    (dict(epi=gemm.GemmEpilogue(1.0, 0.0, PW + 16, 0)), ALIAS),
])
def test_refusals(kw, want):
    assert values(**kw) == want, gemm.gemm_last_error()
    assert gemm.gemm_last_error() != ""


def test_empty_products_launch_nothing():
    assert values(M=0, X=0, C=0, ws=None, nws=0) == gemm.GEMM_OK
    assert values(N=0, B=0, Bs=0, C=0, ws=None, nws=0) == gemm.GEMM_OK


def test_workspace_bytes():
    size = mx.gemm_mx_matmul_values_workspace_bytes
    assert size(-1, 4) == -1 and size(4, 1 << 31) == -1
    assert size(0, 64) == 0 and size(5, 0) == 0
    # Whole blocks of 16 bytes, and scale rows of whole words.
    assert size(17, 65) == 17 * (3 * 16 + 4)
    assert size(2 ** 31 - 1, 2 ** 31 - 1) > 0
