"""Operands of more than 2^31 elements or bytes: stacks of many wide experts,
long batches, wide coded layers.  Whole numbers, whose sums are exact in FP32, or
the same call on a part of the operand, bit for bit."""
import pytest

from dense_gemm_row_amd import grouped, w4

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def memory():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GiB of GPU memory")
    yield
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def whole(seed, shape, dtype=BF16, top=4):
    return torch.randint(-top, top + 1, shape, generator=gen(seed), device="cuda", dtype=torch.int8).to(dtype)


def at(*bounds):
    return torch.tensor(bounds, dtype=torch.int32, device="cuda")


def product(x, w):
    """In FP32, exact for whole numbers of this size."""
    return x.float() @ w.float()


# Rows a group that take the kernels for few rows, the pipelined tiles and (odd
# widths) the general one.
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("rows", [1, 40, 300])
@pytest.mark.parametrize("K, N", [(7168, 2048), (7163, 2047)])
def test_stack_of_experts(K, N, rows, transposed):
    G = 256
    assert (G - 1) * K * N > 2 ** 31
    w = torch.zeros((G, N, K) if transposed else (G, K, N), dtype=BF16, device="cuda")
    used = (0, 150, 255)  # (2^31 elements end inside expert 146)
    for e in used:
        w[e] = whole(e, w.shape[1:])
    bounds = [rows * sum(e < g for e in used) for g in range(G + 1)]
    x = whole(7, (3 * rows, K), top=2)
    y = grouped.matmul(x, w, at(*bounds), transposed=transposed, out_dtype=F32)
    for i, e in enumerate(used):
        part = slice(i * rows, (i + 1) * rows)
        assert torch.equal(y[part], product(x[part], w[e].T.contiguous() if transposed else w[e])), e


@pytest.mark.parametrize("K, N, dtype, out", [(2048, 128, BF16, BF16), (2047, 65, BF16, F32), (2048, 65, F32, F32)])
def test_long_batch(K, N, dtype, out):
    """Rows of x past 2^31 elements; its gradient's sums from such rows."""
    T = 2 ** 31 // K + 3000
    x = torch.zeros(T, K, dtype=dtype, device="cuda")
    dy = torch.zeros(T, N, dtype=dtype, device="cuda")
    tail = slice(T - 2500, T)
    x[tail], dy[tail] = whole(1, (2500, K), dtype, 2), whole(2, (2500, N), dtype, 2)
    w = whole(3, (2, K, N), dtype, 2)
    offsets = at(0, T - 1200, T)
    y = grouped.matmul(x, w, offsets, out_dtype=out)
    assert not bool(y[:T - 2500].any())
    assert torch.equal(y[T - 2500:T - 1200], product(x[T - 2500:T - 1200], w[0]).to(out))
    assert torch.equal(y[T - 1200:], product(x[T - 1200:], w[1]).to(out))
    dw = grouped.weight_grad(x, dy, offsets)
    assert torch.equal(dw[0], product(x[T - 2500:T - 1200].T.contiguous(), dy[T - 2500:T - 1200]))
    assert torch.equal(dw[1], product(x[T - 1200:].T.contiguous(), dy[T - 1200:]))


@pytest.mark.parametrize("K, N, out", [(64, 4096, BF16), (63, 4095, F32)])
def test_large_result(K, N, out):
    T = 2 ** 31 // N + 5000
    x, w = whole(4, (T, K)), whole(5, (2, K, N))
    y = grouped.matmul(x, w, at(0, T - 4000, T), out_dtype=out)
    step = 1 << 16
    for i in range(0, T - 4000, step):
        j = min(i + step, T - 4000)
        assert torch.equal(y[i:j], product(x[i:j], w[0]).to(out)), i
    assert torch.equal(y[T - 4000:], product(x[T - 4000:], w[1]).to(out))


@pytest.mark.parametrize("K, N, out", [(7168, 2048, BF16), (7163, 2047, F32)])
def test_gradient_of_a_stack_of_experts(K, N, out):
    G = 256
    used = {0: slice(0, 40), 150: slice(40, 140), 255: slice(140, 400)}
    bounds = [0] + [max([s.stop for e, s in used.items() if e <= g], default=0) for g in range(G)]
    x, dy = whole(8, (400, K), top=2), whole(9, (400, N), top=2)
    dw = grouped.weight_grad(x, dy, at(*bounds), out_dtype=out)
    for e in range(G):
        if e in used:
            assert torch.equal(dw[e], product(x[used[e]].T.contiguous(), dy[used[e]]).to(out)), e
        else:
            assert not bool(dw[e].any()), e


def values(q, rows):
    """The values of some rows of a coded matrix in 32 bits (scales of 1)."""
    c = q.codes[rows]
    return torch.stack([c & 15, c >> 4], dim=-1).flatten(-2)[..., :q.cols].float() - q.zeros[rows].float().repeat_interleave(
        q.group, dim=-1)[..., :q.cols]


@pytest.mark.parametrize("rows", [1, 20, 200])
@pytest.mark.parametrize("K", [7168, 7165])
def test_stack_of_coded_experts(K, rows):
    """(200 rows: through the dequantised copy of all experts.)"""
    G, N = 320, 2048
    q = w4.empty((G, N, K), 128, "cuda", BF16)
    assert q.codes[: G - 1].numel() > 2 ** 31
    q.codes.random_(generator=gen(10))
    q.scales.fill_(1.0)
    q.zeros.copy_(torch.randint(0, 16, q.zeros.shape, generator=gen(11), device="cuda", dtype=torch.uint8))
    used = (0, 300, 319)
    if rows == 200:  # (more than 128 rows a group on average)
        q = q[295:]
        used, G = (0, 5, 24), 25
        rows = 1200
    bounds = [rows * sum(e < g for e in used) for g in range(G + 1)]
    x = whole(12, (3 * rows, K), top=1)
    y = w4.grouped_matmul(x, q, at(*bounds))
    for i, e in enumerate(used):
        part = slice(i * rows, (i + 1) * rows)
        assert torch.equal(y[part], product(x[part], values(q[e], slice(None)).T.contiguous()).to(BF16)), e


@pytest.mark.parametrize("N, K", [(300000, 16384), (300001, 16382)])
def test_wide_coded_layer(N, K):
    """Codes past 2^31 bytes: quantised, read back and multiplied as parts of it
    are."""
    w = torch.empty(N, K, dtype=BF16, device="cuda")
    for i in range(0, N, 50000):
        w[i:i + 50000].normal_(generator=gen(i))
    q = w4.quantize(w)
    assert q.codes.numel() > 2 ** 31
    back = w4.dequantize(q)
    x = torch.randn(3, K, generator=gen(13), device="cuda", dtype=BF16)
    for i, j in ((0, 4096), (N - 5000, N)):
        part = w4.quantize(w[i:j])
        assert torch.equal(q.codes[i:j], part.codes) and torch.equal(q.scales[i:j], part.scales) and torch.equal(q.zeros[i:j], part.zeros)
        assert torch.equal(back[i:j], w4.dequantize(part))
    y = w4.matmul(x, q)
    exact = x.double() @ w4.dequantize(w4.quantize(w[N - 5000:]), F32).double().T.contiguous()
    # (Half a step of the result, and FP32 sums of K terms that pass through
    # (16 + q) + (16 + z), at most 62, times their weights' scales.)
    size = 62 * x.double().abs().sum(dim=1, keepdim=True) * q.scales[N - 5000:].double().amax(dim=1)
    bound = torch.finfo(BF16).eps / 2 * y[:, N - 5000:].double().abs() + (2 * K + 4 * K // 128 + 24) * 2.0 ** -23 * size
    assert bool(((y[:, N - 5000:].double() - exact).abs() <= bound).all())


@pytest.mark.parametrize("K, N", [(16384, 150000), (16382, 150001)])
def test_wide_layer_quantised_down_its_columns(K, N):
    w = torch.empty(K, N, dtype=BF16, device="cuda")
    for i in range(0, K, 2048):
        w[i:i + 2048].normal_(generator=gen(i))
    q = w4.quantize(w, transposed=True)
    for i, j in ((0, 1000), (N - 1000, N)):
        part = w4.quantize(w[:, i:j].T.contiguous())
        assert torch.equal(q.codes[i:j], part.codes) and torch.equal(q.scales[i:j], part.scales) and torch.equal(q.zeros[i:j], part.zeros)


def test_coded_experts_of_the_most_columns():
    """2^31 - 1 of them; the second expert's results are twice the first one's."""
    N, K = 2 ** 31 - 1, 32
    codes = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda").random_(generator=gen(14))
    scales = torch.empty(2, N, 1, dtype=BF16, device="cuda")
    scales[0], scales[1] = 1.0, 2.0
    q = w4.W4Tensor(codes.expand(2, N, K // 2), scales, None, K, 32)
    x = whole(15, (1, K)).expand(2, K).contiguous()
    y = w4.grouped_matmul(x, q, at(0, 1, 2))
    for i, j in ((0, 100000), (N - 100000, N)):
        c = codes[i:j]
        value = torch.stack([c & 15, c >> 4], dim=-1).flatten(-2).float() - 8
        assert torch.equal(y[0, i:j], (value @ x[0].float()).to(BF16))
    step = 1 << 28
    for i in range(0, N, step):
        assert torch.equal(y[1, i:i + step], 2 * y[0, i:i + step]), i
