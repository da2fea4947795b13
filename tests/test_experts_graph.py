"""The products that record no autograd graph refuse operands whose gradient
would be lost.  CPU only: the refusal comes before any other check."""
import pytest

from dense_gemm_row_amd import grouped, w4

torch = pytest.importorskip("torch")


def operands(*shape, grad=False):
    return torch.zeros(*shape, dtype=torch.bfloat16, requires_grad=grad)


def coded(*lead, grad=False):
    return w4.W4Tensor(torch.zeros(*lead, 64, dtype=torch.uint8), operands(*lead, 1, grad=grad), None, 128)


OFFSETS = torch.tensor([0, 1, 4], dtype=torch.int32)
CALLS = [
    lambda g: grouped.matmul(operands(4, 128, grad=g), operands(2, 128, 6), OFFSETS),
    lambda g: grouped.matmul(operands(4, 128), operands(2, 128, 6, grad=g), OFFSETS),
    lambda g: grouped.matmul(operands(4, 128), operands(2, 6, 128, grad=g), OFFSETS, transposed=True, out=operands(4, 6)),
    lambda g: w4.matmul(operands(4, 128, grad=g), coded(6)),
    lambda g: w4.matmul(operands(4, 128), coded(6, grad=g)),
    lambda g: w4.grouped_matmul(operands(4, 128, grad=g), coded(2, 6), OFFSETS),
    lambda g: w4.grouped_matmul(operands(4, 128), coded(2, 6, grad=g), OFFSETS, out=operands(4, 6)),
]


@pytest.mark.parametrize("call", CALLS)
def test_a_gradient_that_would_be_lost_is_refused(call):
    with pytest.raises(RuntimeError, match="records no graph"):
        call(True)
    # Without one, or where none is recorded, the next check speaks: the
    # operands are not on the GPU.
    with pytest.raises(ValueError, match="GPU"):
        call(False)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        call(True)
    with torch.inference_mode(), pytest.raises(ValueError, match="GPU"):
        call(False)
