"""Grouped and 4-bit products of operands that end where their allocation does
(allocations of whole 2 MiB), of odd widths: whole numbers, whose FP32 sums are
exact, against 64 bits bit for bit."""
import pytest

from dense_gemm_row_amd import grouped, w4

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

UNIT = 2 << 20  # torch maps blocks of 10 MiB and more in whole units of this


def at_end(t):
    """t in the last bytes of a block of its own."""
    size = t.numel() * t.element_size()
    block = torch.empty(max(-(-size // UNIT) * UNIT, 5 * UNIT), dtype=torch.uint8, device="cuda")
    out = block[block.numel() - size:].view(t.dtype).view(t.shape)
    return out.copy_(t)


def whole(seed, low, high, shape, dtype):
    return torch.randint(low, high, shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


def four_bits(lead, K, group, dtype, zeros):
    """(weights, their values); scales 1 and 2."""
    ng = -(-K // group)
    codes = whole(1, 0, 256, (*lead, -(-K // 32) * 16), torch.uint8)
    scales, z = whole(2, 1, 3, (*lead, ng), dtype), whole(3, 0, 16, (*lead, ng), torch.uint8)
    column = torch.arange(K, device="cuda")
    q = (codes[..., column // 2] >> (4 * (column % 2))) & 15
    value = scales.double()[..., column // group] * (q.double() - (z.double()[..., column // group] if zeros else 8))
    return w4.W4Tensor(at_end(codes), at_end(scales), at_end(z) if zeros else None, K, group), value


# (Sums of up to K * 2 * 15 * 1 are exact in FP32 and rounded once.)
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("group", w4.GROUPS)
@pytest.mark.parametrize("M", [1, 16, 40, 64, 128, 140])
@pytest.mark.parametrize("N, K", [(10240, 2047), (1000, 2017), (257, 4097), (72, 289), (40, 257), (5, 31)])
def test_4_bit_products(M, N, K, group, zeros):
    dtype = torch.bfloat16 if M % 3 else torch.float16
    q, value = four_bits((N,), K, group, dtype, zeros)
    x = at_end(whole(4, -1, 2, (M, K), dtype))
    assert torch.equal(w4.matmul(x, q), (x.double() @ value.T).to(dtype))


@pytest.mark.parametrize("group", w4.GROUPS)
@pytest.mark.parametrize("T, N, K, bounds", [(64, 1024, 2047, range(0, 65)), (9, 1024, 2047, [2, 2, 8]), (70, 520, 1001, [0, 33, 70]),
                                             (300, 130, 515, [0, 100, 290])])
def test_4_bit_experts(T, N, K, bounds, group):
    bounds = list(bounds)
    q, value = four_bits((len(bounds) - 1, N), K, group, torch.bfloat16, True)
    x = at_end(whole(5, -1, 2, (T, K), torch.bfloat16))
    exact = torch.zeros(T, N, dtype=torch.float64, device="cuda")
    for g, (a, b) in enumerate(zip(bounds, bounds[1:])):
        exact[a:b] = x[a:b].double() @ value[g].T
    offsets = at_end(torch.tensor(bounds, dtype=torch.int32, device="cuda"))
    assert torch.equal(w4.grouped_matmul(x, q, offsets), exact.to(torch.bfloat16))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=str)
@pytest.mark.parametrize("T, K, N, bounds", [(1, 1, 1, [0, 1]), (9, 301, 77, [0, 1, 9]), (40, 1001, 515, [3, 20, 20, 39]),
                                             (700, 1001, 1203, [0, 350, 700]), (1500, 257, 2049, [0, 1500]), (33, 7, 9, [0, 33]),
                                             (33, 9, 7, [1, 33]), (200, 1000, 1001, [0, 90, 200]), (200, 1001, 1000, [0, 90, 200]),
                                             # few tiles, long sums
                                             (9, 2049, 77, [0, 1, 9]), (70, 1601, 130, [0, 33, 70]), (1, 4097, 5, [0, 1]),
                                             (300, 1025, 65, [2, 2, 290]), (5000, 65, 131, [3, 2500, 4990]),
                                             (2100, 7, 9, [0, 2100]), (4100, 63, 5, [1, 1, 4100])])
def test_products_and_gradients(T, K, N, bounds, dtype):
    G = len(bounds) - 1
    x, dy = at_end(whole(6, -4, 5, (T, K), dtype)), at_end(whole(7, -4, 5, (T, N), dtype))
    w = at_end(whole(8, -4, 5, (G, K, N), dtype))
    wt = at_end(w.transpose(1, 2).contiguous())
    offsets = at_end(torch.tensor(bounds, dtype=torch.int32, device="cuda"))
    y, dw = torch.zeros(T, N, dtype=torch.float64, device="cuda"), torch.zeros(G, K, N, dtype=torch.float64, device="cuda")
    for g, (a, b) in enumerate(zip(bounds, bounds[1:])):
        y[a:b] = x[a:b].double() @ w[g].double()
        dw[g] = x[a:b].double().T.contiguous() @ dy[a:b].double()
    for out in {dtype, torch.float32}:
        assert torch.equal(grouped.matmul(x, w, offsets, out_dtype=out), y.to(out))
        assert torch.equal(grouped.matmul(x, wt, offsets, transposed=True, out_dtype=out), y.to(out))
        assert torch.equal(grouped.weight_grad(x, dy, offsets, out_dtype=out), dw.to(out))
        into = at_end(torch.full((T, N), 3.0, dtype=out, device="cuda"))
        grouped.matmul(x, w, offsets, out=into)
        assert torch.equal(into[bounds[0]:bounds[-1]], y[bounds[0]:bounds[-1]].to(out))
        into = at_end(torch.zeros((G, K, N), dtype=out, device="cuda"))
        grouped.weight_grad(x, dy, offsets, out=into)
        assert torch.equal(into, dw.to(out))
