"""The workspace of the 4-bit products with many rows must not overlap an
operand, `offsets` among them: the dequantised weights would be written over
what the product still has to read.  CPU only."""
import pytest

from dense_gemm_row_amd import gemm, w4

BF16 = gemm.DTYPE_BF16
PX, PQ, PS, PZ, PY, PO, PK = (i << 28 for i in range(1, 8))  # never dereferenced
G, T, N, K = 3, 385, 48, 128
NEED = G * N * K * 2
Q = w4.GemmW4(PQ, 64, 64 * N, PS, 1, N, PZ, 1, N, 128)
ALIAS = gemm.GEMM_ERR_ALIAS


def experts(ws, offsets=PO):
    return w4.gemm_w4_grouped(BF16, G, T, N, K, offsets, PX, K, Q, PY, N, 1, ws, NEED)


@pytest.mark.parametrize("ws", [PO, PO - NEED + 16, PX, PY, PQ, PS, PZ])
def test_a_workspace_over_an_operand_is_refused(ws):
    assert experts(ws) == ALIAS, gemm.gemm_last_error()
    assert "workspace" in gemm.gemm_last_error()


def test_every_offset_counts():
    assert experts(PK, PK + NEED - 4) == ALIAS            # the first one
    assert experts(PK, PK - 4 * G) == ALIAS               # the last of G + 1
    assert w4.gemm_w4_grouped_workspace_bytes(G, T, N, K) == NEED
