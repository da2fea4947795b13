"""A single column expanded over rows has a row stride of 0.  The library must be
told so, and refuses it: taken for 1, it would read or write as many elements as
there are rows from one element's storage.  CPU only: tensors in host memory that
say they are on the GPU, never dereferenced."""
import pytest

from dense_gemm_row_amd import gemm, grouped, mx

torch = pytest.importorskip("torch")


class OnGpu:
    """What the bindings ask of a tensor before they look at its memory."""
    is_cuda = True

    def __init__(self, t):
        self.t, self.dtype, self.shape = t, t.dtype, t.shape

    def dim(self):
        return self.t.dim()

    def stride(self, *at):
        return self.t.stride(*at)


def column(rows, *lead):
    return torch.zeros(*(1,) * len(lead), 1, 1).expand(*lead, rows, 1)


@pytest.mark.parametrize("rows", [2, 5, 4096])
def test_row_strides_of_an_expanded_column(rows):
    assert gemm._ld(OnGpu(column(rows))) == 0
    assert mx._dense(OnGpu(column(rows)), "x")[3] == 0
    assert grouped._stack(OnGpu(column(rows, 3)), "w")[4] == 0


@pytest.mark.parametrize("t, ld", [(torch.zeros(5, 1), 1), (torch.zeros(5, 7)[:, :1], 7), (torch.zeros(1, 1).expand(1, 1), 1),
                                   (torch.zeros(1, 6).expand(1, 6), 6), (torch.zeros(5, 6), 6), (torch.zeros(5, 9)[:, :6], 9),
                                   (torch.zeros(5, 0), 1), (torch.zeros(0, 6), 6), (torch.zeros(1, 0), 1), (torch.zeros(0, 0), 1)])
def test_other_row_strides_are_as_before(t, ld):
    assert gemm._ld(OnGpu(t)) == ld
    assert mx._dense(OnGpu(t), "x")[3] == ld
    assert grouped._stack(OnGpu(t[None]), "w")[4] == ld


PX, PW, PY, PO, PB = (i << 28 for i in range(1, 6))
INVALID = gemm.GEMM_ERR_INVALID_ARG


def test_the_library_refuses_a_stride_of_0():
    L = gemm.lib()
    for lda, ldb, ldc in ((0, 4, 4), (1, 0, 4), (1, 4, 0)):
        assert L.gemm_f32(8, 4, 1, PX, lda, PB, ldb, PY, ldc, None) == INVALID
    assert grouped.gemm_grouped_matmul(gemm.DTYPE_F32, gemm.DTYPE_F32, 0, 2, 8, 4, 1, PO, PX, 0, PW, 4, 4, PY, 4) == INVALID
    assert grouped.gemm_grouped_matmul(gemm.DTYPE_F32, gemm.DTYPE_F32, 0, 2, 8, 1, 4, PO, PX, 4, PW, 0, 4, PY, 1) == INVALID
    assert grouped.gemm_grouped_matmul(gemm.DTYPE_F32, gemm.DTYPE_F32, 0, 2, 8, 1, 4, PO, PX, 4, PW, 1, 4, PY, 0) == INVALID
    assert grouped.gemm_grouped_wgrad(gemm.DTYPE_F32, gemm.DTYPE_F32, 2, 8, 1, 4, PO, PX, 0, PY, 4, PW, 4, 4) == INVALID
    assert mx.gemm_mx_quantize(gemm.DTYPE_F32, 0, 0, 8, 1, PX, 0, PW, 16, PY, 4) == INVALID
    assert mx.gemm_mx_dequantize(gemm.DTYPE_F32, 0, 0, 8, 1, PW, 16, PY, 4, PX, 0) == INVALID
