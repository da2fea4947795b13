"""Grouped products on the GPU against the 64-bit oracle.

Inputs chosen so that every FP32 partial sum is exact must give the exact
result bit for bit, and general inputs must be within

    |C - exact| <= (n + 8) * 2^-23 * sum|a b| + half(type) * |C|

(n FP32 additions, each off by at most one unit in the last place, whatever
their order; half(type) the output's half step relative to the value, plus
half the smallest subnormal)."""
import numpy as np
import pytest

from dense_gemm_row_amd import gemm, grouped
from tests import grouped_oracle as oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {t: (torch.finfo(TYPES[t]).eps / 2, torch.finfo(TYPES[t]).smallest_normal * torch.finfo(TYPES[t]).eps / 2)
        for t in TYPES}


def rng(*seed):
    return np.random.default_rng(seed)


def whole(r, shape, top=4):
    """Whole numbers: products and sums of up to 2^16 of them are exact in FP32."""
    return r.integers(-top, top + 1, shape).astype(np.float64)


def near_normal(r, shape):
    return r.standard_normal(shape) * np.exp(r.uniform(-3, 3, shape[:-1] + (1,)))


def dense(x, kind, pad=0, shift=0, apart=0):
    """x (2-D, or a stack of matrices) on the GPU in a type: rows `pad`
    elements longer, the start moved by `shift` elements, matrices `apart`
    rows further; (tensor, its exact values)."""
    stack = x if x.ndim == 3 else x[None]
    g, rows, cols = stack.shape
    flat = torch.full((g * (rows + apart) * (cols + pad) + shift,), 9.0, dtype=TYPES[kind], device="cuda")
    t = flat[shift:].view(g, rows + apart, cols + pad)[:, :rows, :cols]
    t.copy_(torch.from_numpy(np.ascontiguousarray(stack)))
    t = t if x.ndim == 3 else t[0]
    return t, t.double().cpu().numpy()


def gpu(offsets):
    return torch.tensor(list(offsets), dtype=torch.int32, device="cuda")


def check(got, exact, size, n, kind):
    half, tiny = HALF[kind]
    c = got.double().cpu().numpy()
    bound = (n + 8) * 2.0 ** -23 * size + half * np.abs(c) + tiny
    wrong = ~(np.abs(c - exact) <= bound)
    assert not wrong.any(), (int(wrong.sum()), np.argwhere(wrong)[:3].tolist(), float(np.abs(c - exact).max()))


def check_exact(got, exact, kind):
    want = torch.from_numpy(exact).to(TYPES[kind])
    assert torch.equal(got.cpu(), want), int((got.cpu() != want).sum())


# (T, K, N, offsets): one row, one group; empty groups in front, between and
# behind; rows of no group on both sides; odd sizes; many groups.
CASES = [
    (1, 1, 1, [0, 1]),
    (1, 8, 8, [0, 1]),
    (1, 33, 7, [0, 0, 1, 1]),
    (8, 64, 128, [0, 1, 2, 3, 4, 5, 6, 7, 8]),
    (5, 40, 24, [0, 0, 5, 5, 5]),
    (70, 96, 40, [3, 10, 10, 61, 66]),
    (130, 130, 129, [0, 64, 65, 130]),
    (257, 264, 520, [0, 1, 130, 257]),
    (300, 64, 72, [20, 20, 20, 280]),
    (333, 520, 264, [0, 100, 101, 101, 229, 333]),
    (513, 128, 256, [0, 256, 513]),
    (64, 1000, 1337, [0, 30, 64]),
    (200, 72, 48, list(range(0, 201))),              # 200 groups of one row
    (150, 24, 16, sorted([0] + [7 * i % 150 for i in range(64)] + [150])),  # 65 groups
    (90, 32, 64, [0] * 60 + [45] + [90] * 70),       # most of 130 groups empty
]
ODD = [  # what no router gives: descending, negative and too large offsets
    (100, 64, 64, [50, 20, 80, 60, 90]),
    (100, 64, 64, [-5, 30, -2 ** 31, 70, 2 ** 31 - 1]),
    (40, 32, 32, [100, 20, 30]),
]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("T, K, N, offsets", CASES + ODD)
def test_product_is_exact_on_whole_numbers(T, K, N, offsets, transposed, kind):
    r = rng(T, K, N)
    x, ex = dense(whole(r, (T, K)), kind)
    w, ew = dense(whole(r, (len(offsets) - 1, N, K) if transposed else (len(offsets) - 1, K, N)), kind)
    if transposed:
        ew = ew.transpose(0, 2, 1)
    exact, _ = oracle.product(ex, ew, offsets)
    for out in {kind, "f32"}:
        check_exact(grouped.matmul(x, w, gpu(offsets), transposed=transposed, out_dtype=TYPES[out]), exact, out)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("T, K, N, offsets", CASES + ODD)
def test_gradient_is_exact_on_whole_numbers(T, K, N, offsets, kind):
    r = rng(T, K, N, 1)
    x, ex = dense(whole(r, (T, K)), kind)
    dy, ey = dense(whole(r, (T, N)), kind)
    exact, _ = oracle.gradient(ex, ey, offsets)
    for out in {kind, "f32"}:
        check_exact(grouped.weight_grad(x, dy, gpu(offsets), out_dtype=TYPES[out]), exact, out)


LAYOUTS = [dict(), dict(pad=3), dict(pad=8), dict(shift=1), dict(pad=8, shift=8), dict(pad=1, shift=3)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
def test_product_of_any_layout(layout, transposed, kind):
    """General values, strided operands and results; nothing outside a result
    is written, rows of no group are left as they were."""
    T, K, N, offsets = 203, 136, 200, [2, 2, 90, 91, 180]
    r = rng(len(str(layout)), transposed)
    x, ex = dense(near_normal(r, (T, K)), kind, **layout)
    shape = (4, N, K) if transposed else (4, K, N)
    w, ew = dense(near_normal(r, shape), kind, apart=layout.get("pad", 0), **layout)
    if transposed:
        ew = ew.transpose(0, 2, 1)
    exact, size = oracle.product(ex, ew, offsets)
    free = oracle.outside(offsets, T)
    for out in {kind, "f32"}:
        y, _ = dense(np.full((T, N), 5.0), out, **layout)
        base = y._base
        base.fill_(7.0)
        assert grouped.matmul(x, w, gpu(offsets), transposed=transposed, out=y) is y
        assert bool((y[torch.from_numpy(free).cuda()] == 7.0).all()), "wrote a row of no group"
        check(y[torch.from_numpy(~free).cuda()], exact[~free], size[~free], K, out)
        y.fill_(7.0)
        assert bool((base == 7.0).all()), "wrote outside the result"
        check(grouped.matmul(x, w, gpu(offsets), transposed=transposed, out_dtype=TYPES[out]), exact, size, K, out)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("layout", LAYOUTS, ids=str)
def test_gradient_of_any_layout(layout, kind):
    T, K, N, offsets = 203, 136, 200, [2, 2, 90, 91, 180]
    r = rng(len(str(layout)), 2)
    x, ex = dense(near_normal(r, (T, K)), kind, **layout)
    dy, ey = dense(near_normal(r, (T, N)), kind, **layout)
    exact, size = oracle.gradient(ex, ey, offsets)
    for out in {kind, "f32"}:
        dw, _ = dense(np.zeros((4, K, N)), out, apart=layout.get("pad", 0), **layout)
        base = dw._base
        base.fill_(float("nan"))  # (beta = 0: the old values do not count)
        grouped.weight_grad(x, dy, gpu(offsets), out=dw)
        check(dw, exact, size, T, out)
        dw.fill_(float("nan"))
        assert bool(base.isnan().all()), "wrote outside the result"
        dw.fill_(2.0)
        grouped.weight_grad(x, dy, gpu(offsets), out=dw, alpha=0.5, beta=-1.5)
        check(dw, 0.5 * exact - 3.0, 0.5 * size + 3.0, T + 2, out)


@pytest.mark.parametrize("kind", TYPES)
def test_one_matrix_for_all_groups(kind):
    r = rng(5)
    x, ex = dense(whole(r, (60, 64)), kind)
    w, ew = dense(whole(r, (1, 64, 32)), kind)
    offsets = [0, 10, 40, 60]
    exact, _ = oracle.product(ex, np.repeat(ew, 3, axis=0), offsets)
    check_exact(grouped.matmul(x, w.expand(3, 64, 32), gpu(offsets)), exact, kind)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("width", [64, 65])
def test_infinities_and_nan_stay_where_they_are(kind, width):
    """Weights of groups without rows, rows of no group and a row's own
    values: what they hold reaches no other result."""
    offsets = [4, 20, 20, 70]
    r = rng(6, width)
    x, w, dy = whole(r, (80, width)), whole(r, (3, width, width)), whole(r, (80, width))
    x[:4], x[70:], dy[:4], dy[70:] = np.nan, np.inf, np.inf, np.nan
    w[1] = np.nan
    exact, _ = oracle.product(x, w, offsets)
    dexact, _ = oracle.gradient(x, dy, offsets)
    tx, tw, ty = dense(x, kind)[0], dense(w, kind)[0], dense(dy, kind)[0]
    check_exact(grouped.matmul(tx, tw, gpu(offsets)), exact, kind)
    check_exact(grouped.matmul(tx, tw.transpose(1, 2).contiguous(), gpu(offsets), transposed=True), exact, kind)
    check_exact(grouped.weight_grad(tx, ty, gpu(offsets), out_dtype=TYPES[kind]), dexact, kind)
    x[30, 5] = np.nan  # one row of group 2: its row of y, its feature of dw
    tx = dense(x, kind)[0]
    y = grouped.matmul(tx, tw, gpu(offsets)).double().cpu().numpy()
    assert np.isnan(y[30]).all() and np.array_equal(np.delete(y, 30, 0), np.delete(exact, 30, 0))
    dw = grouped.weight_grad(tx, ty, gpu(offsets)).double().cpu().numpy()
    assert np.isnan(dw[2, 5]).all() and not np.isnan(np.delete(dw, 5, 1)).any()


@pytest.mark.parametrize("kind", TYPES)
def test_empty_sizes(kind):
    t = TYPES[kind]
    zero = gpu([0, 0, 0])
    empty = lambda *s: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    assert grouped.matmul(empty(0, 8), empty(2, 8, 16), zero).shape == (0, 16)
    assert grouped.matmul(empty(4, 8), empty(2, 8, 0), gpu([0, 1, 4])).shape == (4, 0)
    y = grouped.matmul(empty(4, 0), empty(2, 0, 16), gpu([0, 1, 4]))
    assert y.shape == (4, 16) and bool((y == 0).all())
    y = grouped.matmul(empty(4, 8), empty(0, 8, 16), gpu([0]))
    assert bool((y == 0).all())
    dw = grouped.weight_grad(empty(0, 8), empty(0, 16), zero)
    assert dw.shape == (2, 8, 16) and bool((dw == 0).all())
    assert grouped.weight_grad(empty(4, 0), empty(4, 16), gpu([0, 1, 4])).shape == (2, 0, 16)
    assert grouped.weight_grad(empty(4, 8), empty(4, 16), gpu([0])).shape == (0, 8, 16)


@pytest.mark.parametrize("kind", TYPES)
def test_captured_calls_follow_new_offsets(kind):
    """One captured graph, replayed with the offsets and inputs of the moment."""
    T, K, N, G = 200, 128, 96, 5
    r = rng(8)
    x, w, dy = (dense(whole(r, s), kind)[0] for s in ((T, K), (G, K, N), (T, N)))
    offsets = gpu([0, 10, 10, 50, 120, 200])
    y, dx, dw = (torch.empty(s, dtype=TYPES[kind], device="cuda") for s in ((T, N), (T, K), (G, K, N)))

    def step():
        y.copy_(grouped.matmul(x, w, offsets))
        dx.copy_(grouped.matmul(dy, w, offsets, transposed=True))
        grouped.weight_grad(x, dy, offsets, out=dw)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        bounds = np.sort(r.integers(0, T + 1, G + 1))
        offsets.copy_(torch.from_numpy(bounds.astype(np.int32)))
        x.copy_(torch.from_numpy(whole(r, (T, K))))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (y, dx, dw)]
        for t in (y, dx, dw):
            t.fill_(3.0)
        torch.cuda.synchronize()
        step()
        for a, b in zip(got, (y, dx, dw)):
            assert torch.equal(a, b)
        check_exact(got[0], oracle.product(x.double().cpu().numpy(), w.double().cpu().numpy(), bounds)[0], kind)


@pytest.mark.parametrize("kind", TYPES)
def test_calls_on_another_stream(kind):
    r = rng(9)
    offsets = [0, 100, 300]
    x, ex = dense(whole(r, (300, 256)), kind)
    w, ew = dense(whole(r, (2, 256, 256)), kind)
    exact, _ = oracle.product(ex, ew, offsets)
    at = gpu(offsets)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    results = [grouped.matmul(x, w, at, stream=s) for s in streams for _ in range(3)]
    for s in streams:
        s.synchronize()
    for y in results:
        check_exact(y, exact, kind)


@pytest.mark.parametrize("kind", TYPES)
def test_results_repeat(kind):
    r = rng(10)
    offsets = gpu([0, 37, 400, 700])
    x, w, dy = (dense(near_normal(r, s), kind)[0] for s in ((700, 520), (3, 520, 264), (700, 264)))
    y, dw = grouped.matmul(x, w, offsets), grouped.weight_grad(x, dy, offsets)
    for _ in range(5):
        assert torch.equal(grouped.matmul(x, w, offsets), y) and torch.equal(grouped.weight_grad(x, dy, offsets), dw)


# ---------------------------------------------------------------------------
# The layer
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("T, K, N, offsets", [(70, 96, 40, [3, 10, 10, 61, 66]), (1, 33, 1, [0, 0, 1]), (130, 64, 128, [0, 64, 130])])
def test_linear_has_the_formulas_gradients(T, K, N, offsets, transposed, kind):
    r = rng(11, T)
    x, ex = dense(near_normal(r, (T, K)), kind)
    G = len(offsets) - 1
    w, ew = dense(near_normal(r, (G, N, K) if transposed else (G, K, N)), kind)
    dy, ey = dense(near_normal(r, (T, N)), kind)
    x.requires_grad_(True)
    w.requires_grad_(True)
    y = grouped.linear(x, w, gpu(offsets), transposed)
    y.backward(dy)
    kn = ew.transpose(0, 2, 1) if transposed else ew
    check(y.detach(), *oracle.product(ex, kn, offsets), K, kind)
    check(x.grad, *oracle.product(ey, kn.transpose(0, 2, 1), offsets), N, kind)
    dw, size = oracle.gradient(ex, ey, offsets)
    if transposed:
        dw, size = dw.transpose(0, 2, 1), size.transpose(0, 2, 1)
    check(w.grad, dw, size, T, kind)
    assert x.grad.dtype == x.dtype and w.grad.dtype == w.dtype


def test_linear_against_differences():
    """The derivative of sum(c * y) along a direction, by central differences
    in 64 bits of the oracle (the product is bilinear: the difference quotient
    has no error of its own beyond rounding)."""
    T, K, N, offsets = 50, 40, 24, [5, 20, 20, 45]
    r = rng(12)
    ex, ew, c = (r.standard_normal(s) for s in ((T, K), (3, K, N), (T, N)))
    x, w, dy = (torch.tensor(v, dtype=torch.float32, device="cuda") for v in (ex, ew, c))
    ex, ew, c = (t.double().cpu().numpy() for t in (x, w, dy))
    x.requires_grad_(True)
    w.requires_grad_(True)
    grouped.linear(x, w, gpu(offsets)).backward(dy)
    h = 2.0 ** -10
    for leaf, at in ((x, 0), (w, 1)):
        d = r.standard_normal(leaf.shape)
        move = [(ex + s * h * d, ew) if at == 0 else (ex, ew + s * h * d) for s in (1, -1)]
        slope = sum(s * (c * oracle.product(*m, offsets)[0]).sum() for s, m in zip((1, -1), move)) / (2 * h)
        got = float((leaf.grad.double().cpu().numpy() * d).sum())
        # each gradient element is within (n + 8) 2^-23 of its sum of magnitudes
        n = N if at == 0 else T
        mags = (oracle.product(np.abs(c), np.abs(ew).transpose(0, 2, 1), offsets)[0] if at == 0
                else oracle.gradient(np.abs(ex), np.abs(c), offsets)[0])
        assert abs(got - slope) <= (n + 8) * 2.0 ** -23 * (mags * np.abs(d)).sum() + 1e-9


def test_linear_keeps_only_what_it_needs_and_refuses_a_second_derivative():
    r = rng(13)
    offsets = gpu([0, 20, 50])
    x, w = dense(whole(r, (50, 32)), "bf16")[0], dense(whole(r, (2, 32, 16)), "bf16")[0]
    for leaf, kept in ((x, w), (w, x)):
        packed = []
        leaf.requires_grad_(True)
        with torch.autograd.graph.saved_tensors_hooks(lambda t: (packed.append(t), t)[1], lambda t: t):
            y = grouped.linear(x, w, offsets)
        leaf.requires_grad_(False)
        assert [t.shape for t in packed] == [kept.shape, offsets.shape]
    x.requires_grad_(True)
    y = grouped.linear(x, w, offsets)
    dx, = torch.autograd.grad((y * y).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dx.sum().backward()


def test_linear_takes_expanded_and_transposed_gradients():
    r = rng(14)
    x, w = dense(whole(r, (50, 32)), "f32")[0], dense(whole(r, (2, 32, 16)), "f32")[0]
    offsets = gpu([0, 20, 50])
    grads = []
    for dy in (torch.ones(1, 1, device="cuda").expand(50, 16), torch.ones(16, 50, device="cuda").t(),
               torch.ones(50, 16, device="cuda")):
        x.requires_grad_(True)
        w.requires_grad_(True)
        x.grad = w.grad = None
        grouped.linear(x, w, offsets).backward(dy)
        grads.append((x.grad, w.grad))
    for a, b in grads[:2]:
        assert torch.equal(a, grads[2][0]) and torch.equal(b, grads[2][1])


def test_torch_forms_refuse():
    x = torch.zeros(8, 16, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(2, 16, 24, device="cuda", dtype=torch.bfloat16)
    dy = torch.zeros(8, 24, device="cuda", dtype=torch.bfloat16)
    at = gpu([0, 4, 8])
    for error, call in [
        (ValueError, lambda: grouped.matmul(x[0], w, at)), (ValueError, lambda: grouped.matmul(x, w[0], at)),
        (TypeError, lambda: grouped.matmul(x.float(), w, at)), (TypeError, lambda: grouped.matmul(x.double(), w, at)),
        (ValueError, lambda: grouped.matmul(x.t(), w, at)), (ValueError, lambda: grouped.matmul(x, w.transpose(1, 2), at)),
        (ValueError, lambda: grouped.matmul(x[:, :8], w, at)), (ValueError, lambda: grouped.matmul(x, w, at, transposed=True)),
        (ValueError, lambda: grouped.matmul(x, w, at[:2])), (TypeError, lambda: grouped.matmul(x, w, at.long())),
        (TypeError, lambda: grouped.matmul(x, w, [0, 4, 8])), (ValueError, lambda: grouped.matmul(x, w, at.cpu())),
        (TypeError, lambda: grouped.matmul(x, w, at, out_dtype=torch.float16)),
        (ValueError, lambda: grouped.matmul(x, w, at, out=dy[:4])), (ValueError, lambda: grouped.matmul(x.cpu(), w, at)),
        (TypeError, lambda: grouped.matmul(x, w, at, out=dy.half())),
        (ValueError, lambda: grouped.matmul(x, w, gpu([0, 0, 4, 4, 8])[::2])),
        (gemm.GemmError, lambda: grouped.matmul(x, w[:, :, :16], at, out=x)),
        (TypeError, lambda: grouped.weight_grad(x, dy.half(), at)), (ValueError, lambda: grouped.weight_grad(x, dy[:4], at)),
        (TypeError, lambda: grouped.weight_grad(x, dy, at.long())), (TypeError, lambda: grouped.weight_grad(x, dy, at[:0])),
        (ValueError, lambda: grouped.weight_grad(x, dy, at, beta=1.0)),
        (TypeError, lambda: grouped.weight_grad(x, dy, at, out_dtype=torch.float16)),
        (ValueError, lambda: grouped.weight_grad(x, dy, at, out=w[:1])),
    ]:
        with pytest.raises(error):
            call()
