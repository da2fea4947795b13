"""Results into a caller's tensors: autograd is told that they were written, so
that a graph which has saved one refuses its backward pass instead of taking the
new values for the old."""
import pytest

from dense_gemm_row_amd import grouped, w4

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def ones(*shape):
    return torch.ones(*shape, dtype=BF16, device="cuda")


def calls():
    at = torch.tensor([0, 3, 8], dtype=torch.int32, device="cuda")
    x, w, dy = ones(8, 64), ones(2, 64, 32), ones(8, 32)
    q, stack = w4.quantize(ones(32, 64), 32), w4.quantize(ones(2, 32, 64), 32)
    return {
        "matmul": ((8, 32), lambda out: grouped.matmul(x, w, at, out=out)),
        "weight_grad": ((2, 64, 32), lambda out: grouped.weight_grad(x, dy, at, out=out)),
        "w4.matmul": ((8, 32), lambda out: w4.matmul(x, q, out=out)),
        "w4.grouped_matmul": ((8, 32), lambda out: w4.grouped_matmul(x, stack, at, out=out)),
        "w4.dequantize": ((32, 64), lambda out: w4.dequantize(q, out=out)),
        "w4.dequantize of a stack": ((2, 32, 64), lambda out: w4.dequantize(stack, out=out)),
    }


@pytest.mark.parametrize("name", ["matmul", "weight_grad", "w4.matmul", "w4.grouped_matmul", "w4.dequantize",
                                  "w4.dequantize of a stack"])
def test_a_saved_tensor_that_was_written_is_refused(name):
    shape, call = calls()[name]
    out, leaf = ones(*shape), ones(*shape).requires_grad_(True)
    loss = (leaf * out).sum()
    before = out._version
    assert call(out) is out and out._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with torch.inference_mode():  # (such tensors have no version)
        call(ones(*shape))


@pytest.mark.parametrize("zeros", [True, False])
def test_coded_results(zeros):
    for w in (ones(32, 64), ones(2, 32, 64)):
        q = w4.quantize(w, 32, zeros)
        parts = [t for t in (q.codes, q.scales, q.zeros) if t is not None]
        before = [t._version for t in parts]
        assert w4.quantize(w, out=q) is q
        assert all(t._version > b for t, b in zip(parts, before))


def test_stacks_of_results_that_overlap_are_refused():
    w = ones(2, 32, 64)
    q = w4.quantize(w, 32)
    same = w4.W4Tensor(q.codes[:1].expand(2, 32, 32), q.scales, q.zeros, 64, 32)
    scales = w4.W4Tensor(q.codes, q.scales[:1].expand(2, 32, 2), q.zeros, 64, 32)
    zeros = w4.W4Tensor(q.codes, q.scales, q.zeros[:1].expand(2, 32, 2), 64, 32)
    for out in (same, scales, zeros):
        with pytest.raises(ValueError, match="overlap"):
            w4.quantize(w, out=out)
    with pytest.raises(ValueError, match="overlap"):
        w4.dequantize(q, out=ones(32, 64).expand(2, 32, 64))
    for out in (ones(32, 2, 64).transpose(0, 1), ones(2, 32, 70)[..., :64]):  # apart
        assert torch.equal(w4.dequantize(q, out=out), w)
