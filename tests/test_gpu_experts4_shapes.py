"""Results of 4-bit products of few rows at sizes that take each of their
kernels: whole numbers, whose FP32 sums are exact, against 64 bits bit for bit,
and nothing written outside the result.  (tests/experts4_sizes.py)"""
import pytest

from dense_gemm_row_amd import w4
from tests.experts4_sizes import READS, SHAPES
from tests.test_gpu_experts_ends import four_bits, whole

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


# (Sums of up to K * 31 * 2 * 1 in the kernel's order are exact in FP32.)
@pytest.mark.parametrize("group", w4.GROUPS)
@pytest.mark.parametrize("K", [k for ks in READS.values() for k in ks])
@pytest.mark.parametrize("case", [(s, *c) for s, cases in SHAPES.items() for c in cases],
                         ids=lambda c: f"{'x'.join(map(str, c[0]))}-{c[1]}x{c[2]}" + ("-experts" if c[3] else ""))
def test_products(case, K, group):
    _, rows, N, offsets = case
    dtype = torch.float16 if (rows + group) % 3 == 0 else torch.bfloat16
    zeros = (N + group // 32) % 2 == 0
    lead = (N,) if offsets is None else (len(offsets) - 1, N)
    q, value = four_bits(lead, K, group, dtype, zeros)
    x = whole(4, -1, 2, (rows, K), dtype)
    y = torch.full((rows + 1, N + 3), 7.0, dtype=dtype, device="cuda")
    out = y[:rows, :N]
    if offsets is None:
        w4.matmul(x, q, out=out)
        a, b, exact = 0, rows, x.double() @ value.T.contiguous()
    else:
        w4.grouped_matmul(x, q, torch.tensor(offsets, dtype=torch.int32, device="cuda"), out=out)
        a, b = offsets[0], offsets[-1]
        exact = torch.zeros(rows, N, dtype=torch.float64, device="cuda")
        for g, (i, j) in enumerate(zip(offsets, offsets[1:])):
            exact[i:j] = x[i:j].double() @ value[g].T.contiguous()
    assert torch.equal(out[a:b], exact[a:b].to(dtype))
    out[a:b] = 7.0
    assert bool((y == 7.0).all()), "wrote outside the result"
