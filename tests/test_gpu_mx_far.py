"""Microscaled operators on rows as long as the documented range allows."""
import pytest

from dense_gemm_row_amd import mx

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TOP = 2 ** 31 - 1


def ones(k):
    """One coded row of k ones (E2M1 code 2, scale 127), zeros after them."""
    q = mx.empty(1, k, mx.E2M1, "cuda")
    q.codes.fill_(0x22)
    q.scales.fill_(127)
    for c in range(k, q.codes.shape[1] * 2):
        q.codes[0, c // 2] &= 0xF0 if c % 2 == 0 else 0x0F
    return q


@pytest.mark.parametrize("k", [TOP, TOP - 30, TOP - 31])
def test_product_sums_over_the_whole_of_k(k):
    """Each of the eight partial sums is a multiple of 128 until its last
    step, so exact in FP32 (below 2^24 * 128); the last step may lose a unit
    of 2^28 (16), and each of seven additions half a unit of 2^31 (64)."""
    got = mx.matmul(ones(k), ones(k), out_dtype=torch.float32)
    assert abs(float(got[0, 0]) - k) <= 8 * 16 + 7 * 64


@pytest.mark.parametrize("cols", [TOP, TOP - 30])
def test_quantise_one_row_and_back(cols):
    x = torch.ones(1, cols, dtype=torch.bfloat16, device="cuda")
    x[0, -3:] = 3.0  # in blocks of other scales: 6 and 2 times 1/2 in place of 4 times 1/4
    q = mx.quantize(x)
    first = (cols - 3) // 32
    assert q.scales.shape == (1, -(-cols // 32))
    assert bool((q.scales[0, :first] == 125).all()) and bool((q.scales[0, first:] == 126).all())
    back = mx.dequantize(q)
    assert torch.equal(back, x)
