"""Results of grouped products and their gradients at sizes that take each
tile: whole numbers, whose FP32 sums are exact, against 64 bits bit for bit.
(tests/experts_sizes.py)"""
import pytest

from dense_gemm_row_amd import grouped
from tests.experts_sizes import GRADIENTS, PRODUCTS

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def whole(seed, shape, dtype):
    return torch.randint(-4, 5, shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


def spans(offsets):
    return list(zip(offsets, offsets[1:]))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("case", [c for cases in PRODUCTS.values() for c in cases], ids=lambda c: "x".join(map(str, c[:3])))
def test_products(case, transposed, dtype):
    T, K, N, offsets = case
    G = len(offsets) - 1
    x = whole(1, (T, K), dtype)
    w = whole(2, (G, N, K) if transposed else (G, K, N), dtype)
    exact = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    for g, (a, b) in enumerate(spans(offsets)):
        exact[a:b] = x[a:b].double() @ (w[g].T if transposed else w[g]).double()
    o = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    for out in (dtype, torch.float32):
        y = torch.full((T + 1, N + 8), 7.0, dtype=out, device="cuda")
        grouped.matmul(x, w, o, transposed=transposed, out=y[:T, :N])
        assert torch.equal(y[offsets[0]:offsets[-1], :N], exact[offsets[0]:offsets[-1]].to(out))
        y[offsets[0]:offsets[-1], :N] = 7.0
        assert bool((y == 7.0).all()), "wrote outside the groups' rows"


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("case", [c for cases in GRADIENTS.values() for c in cases], ids=lambda c: "x".join(map(str, c[:3])))
def test_gradients(case, dtype):
    T, K, N, offsets = case
    x, dy = whole(3, (T, K), dtype), whole(4, (T, N), dtype)
    exact = torch.stack([x[a:b].double().T.contiguous() @ dy[a:b].double() for a, b in spans(offsets)])
    o = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    for out in (dtype, torch.float32):
        dw = torch.full((len(offsets) - 1, K + 1, N + 8), float("nan"), dtype=out, device="cuda")
        view = dw[:, :K, :N]
        grouped.weight_grad(x, dy, o, out=view)
        assert torch.equal(view, exact.to(out))
        view.copy_(whole(5, exact.shape, out))
        old = view.double()
        grouped.weight_grad(x, dy, o, out=view, alpha=0.5, beta=2.0)
        assert torch.equal(view, (0.5 * exact + 2.0 * old).to(out))
        view.fill_(float("nan"))
        assert bool(dw.isnan().all()), "wrote outside the result"
