"""4-bit weights with group scales on the GPU against the 64-bit oracle.

Quantisation is exact: codes, scales and zero points are compared bit for bit,
values with their one rounding.  Products of inputs whose FP32 sums are all
exact must be exact.  General ones must be within

    |Y - exact| <= (2 K + 4 ng + 24) 2^-23 S + half(type) |Y|,
    S = sum |s| ((16 + q) + (16 + z)) |x|

for few rows (codes are multiplied as 16 + q, and 16 + z times the sum of x is
taken off): of each term, K additions of (16 + q) x and K of x (times 16 + z),
then for each of ng groups two fused operations and an addition, 8 additions
over the waves and the rest for the roundings themselves; half(type) as for the other
products.  With more rows the weights are rounded to the type first:

    ((K + 8) 2^-23 + half(type)) sum |w x| (1 + half(type)) + half(type) |Y|."""
import numpy as np
import pytest

from dense_gemm_row_amd import gemm, grouped, w4
from tests import grouped_oracle, w4_oracle as oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SCALES = ["f16", "bf16"]
HALF = {t: (torch.finfo(TYPES[t]).eps / 2, torch.finfo(TYPES[t]).smallest_normal * torch.finfo(TYPES[t]).eps / 2)
        for t in TYPES}
GUARD = 0xA5


def rng(*seed):
    return np.random.default_rng(seed)


def dense(x, kind, pad=0, shift=0):
    """x (2-D or a stack) on the GPU in a type, rows `pad` elements longer and
    the start moved by `shift` elements; (tensor, its exact values)."""
    flat = torch.full((int(np.prod(x.shape[:-1])) * (x.shape[-1] + pad) + shift,), 9.0, dtype=TYPES[kind], device="cuda")
    t = flat[shift:].view(*x.shape[:-1], x.shape[-1] + pad)[..., :x.shape[-1]]
    t.copy_(torch.from_numpy(np.ascontiguousarray(x)))
    return t, t.double().cpu().numpy()


def gpu(offsets):
    return torch.tensor(list(offsets), dtype=torch.int32, device="cuda")


def guarded(shape, group, kind, zeros, pad=0):
    """An output inside larger buffers full of a guard byte; (W4Tensor, buffers)."""
    *lead, K = shape
    width, ng = -(-K // 32) * 16, -(-K // group)
    make = lambda n, t: torch.full((*lead[:-1], lead[-1] + 1, n), GUARD, dtype=torch.uint8, device="cuda").view(t)  # noqa: E731
    codes, scales, points = make(width + 16 * pad, torch.uint8), make(2 * (ng + pad), TYPES[kind]), make(ng + pad, torch.uint8)
    n = lead[-1]
    q = w4.W4Tensor(codes[..., :n, :width], scales[..., :n, :ng], points[..., :n, :ng] if zeros else None, K, group)
    return q, (codes, scales, points)


def assert_guards(q, buffers):
    for t, part in zip(buffers, (q.codes, q.scales, q.zeros)):
        b = t.view(torch.uint8)
        width = 0 if part is None else part.shape[-1] * part.element_size()
        assert bool((b[..., -1, :] == GUARD).all()) and bool((b[..., width:] == GUARD).all())


def check_codes(q, exact, group, kind):
    codes, s, z = oracle.quantize(exact, group, q.zeros is not None, kind)
    got = q.scales.double().cpu().numpy()
    assert np.array_equal(got, s, equal_nan=True), np.argwhere(~((got == s) | (np.isnan(got) & np.isnan(s))))[:3]
    if q.zeros is not None:
        assert np.array_equal(q.zeros.cpu().numpy(), z)
    got = oracle.unpack(q.codes.cpu().numpy(), exact.shape[1])
    assert np.array_equal(got, codes), np.argwhere(got != codes)[:3].tolist()


def weights(r, N, K):
    """Rows of very different size, zeros, an all-zero stretch, one-sided rows."""
    w = r.standard_normal((N, K)) * np.exp(r.uniform(-6, 4, (N, 1)))
    w[r.random((N, K)) < 0.05] = 0
    w[N // 2, 32:64] = 0
    w[N // 3] = np.abs(w[N // 3])
    return w


SIZES = [(1, 1), (1, 31), (3, 32), (2, 33), (5, 100), (64, 128), (65, 129), (7, 1000), (33, 2090), (130, 257)]


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("N, K", SIZES)
def test_quantise_and_back(N, K, kind, scale):
    r = rng(N, K)
    exact0 = weights(r, N, K)
    for i, group in enumerate(w4.GROUPS):
        for zeros in (True, False):
            for trans in (False, True):
                pad, shift = [(0, 0), (3, 0), (8, 0), (0, 1)][(i + 2 * zeros + trans) % 4]
                t, e = dense(exact0.T if trans else exact0, kind, pad, shift)
                e = e.T if trans else e
                q, buffers = guarded((N, K), group, scale, zeros, pad=i)
                assert w4.quantize(t, group, transposed=trans, out=q) is q
                check_codes(q, e, group, scale)
                assert_guards(q, buffers)
                made = w4.quantize(t, group, zeros, trans, scale_dtype=TYPES[scale])
                assert torch.equal(made.scales, q.scales) and torch.equal(made.codes[:, :K // 2], q.codes[:, :K // 2])
                value = oracle.values(*oracle.quantize(e, group, zeros, scale), group)[0]
                for back in TYPES:
                    out, _ = dense(np.zeros((N, K)), back, pad, shift)
                    out._base.fill_(3.0)
                    w4.dequantize(q, out=out)
                    assert torch.equal(out.cpu(), torch.from_numpy(value).to(TYPES[back]))
                    out.fill_(3.0)
                    assert bool((out._base == 3.0).all()), "wrote outside the matrix"


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("kind", TYPES)
def test_quantise_every_midpoint(kind, scale):
    """Groups whose scale is a power of two (down to the subnormals) with every
    midpoint between two codes and its neighbours in the type."""
    eps = torch.finfo(TYPES[kind]).eps
    for zeros in (True, False):
        top = 15 if zeros else 7
        points = np.arange(0, 2 * top + 1) / 2.0
        points = np.concatenate([points, points[1:] * (1 - eps), points[:-1] * (1 + eps)]).clip(0, top)
        points = points if zeros else np.concatenate([points, -points])
        points = np.concatenate([points, np.zeros(-len(points) % 31)]).reshape(-1, 31)
        base = np.concatenate([np.full((len(points), 1), float(top)), points], axis=1)
        for e in (0, 4, -6, -14, -20) + (() if "f16" in (kind, scale) else (100, -100, -126, -130)):
            t, exact = dense(base * 2.0 ** e, kind)
            q = w4.quantize(t, 32, zeros, scale_dtype=TYPES[scale])
            check_codes(q, exact, 32, scale)
            check_codes(w4.quantize(t.t().contiguous(), 32, zeros, True, TYPES[scale]), exact, 32, scale)


@pytest.mark.parametrize("scale", SCALES)
@pytest.mark.parametrize("kind", TYPES)
def test_quantise_special_values(kind, scale):
    fi = torch.finfo(TYPES[kind])
    x = np.zeros((11, 70))
    x[0, 3] = np.nan
    x[1, 40] = np.inf
    x[2, 69] = -np.inf  # in the partial group
    x[3, :] = fi.max
    x[4, ::2], x[4, 1::2] = fi.max, fi.min  # a span beyond the type
    x[5, :] = fi.smallest_normal * fi.eps
    x[6, ::2] = -0.0
    x[7, :] = -fi.smallest_normal
    x[8, 5] = fi.min
    x[9, :] = np.linspace(1, 2, 70)
    x[10, :] = -1.0
    t, exact = dense(x, kind)
    for zeros in (True, False):
        for group in w4.GROUPS:
            for q in (w4.quantize(t, group, zeros, scale_dtype=TYPES[scale]),
                      w4.quantize(t.t().contiguous(), group, zeros, True, TYPES[scale])):
                check_codes(q, exact, group, scale)
        back = w4.dequantize(w4.quantize(t, 32, zeros, scale_dtype=TYPES[scale]), torch.float32).cpu().numpy()
        assert np.isnan(back[0, :32]).all() and np.isnan(back[1, 32:64]).all() and np.isnan(back[2, 64:]).all()
        assert not np.isnan(back[3:]).any() and not np.isnan(back[0, 32:]).any()


def coded(r, shape, group, kind, zeros, low=-3, high=4, pad=0, whole=False):
    """Random codes; scales powers of two (whole) or general, some negative."""
    *lead, K = shape
    ng = -(-K // group)
    q, buffers = guarded(shape, group, kind, zeros, pad)
    codes = r.integers(0, 16, (int(np.prod(lead)), K)).astype(np.uint8)
    s = 2.0 ** r.integers(low, high, (len(codes), ng)) * (1 if whole else r.uniform(1, 2, (len(codes), ng)))
    s = np.where(r.random(s.shape) < 0.1, -s, s)
    s = torch.from_numpy(s).to(TYPES[kind])
    z = r.integers(0, 16, (len(codes), ng)).astype(np.uint8) if zeros else np.full((len(codes), ng), 8, np.uint8)
    packed = oracle.pack(codes)
    packed[:, K // 2 + K % 2:] = 0xFF  # (the filling holds anything)
    if K % 2:
        packed[:, K // 2] |= 0xF0
    q.codes.copy_(torch.from_numpy(packed).view(*lead, -1))
    q.scales.copy_(s.view(*lead, ng))
    if zeros:
        q.zeros.copy_(torch.from_numpy(z).view(*lead, ng))
    value, size = oracle.values(codes, s.double().numpy(), z, group)
    return q, value.reshape(shape), size.reshape(shape)


def whole(r, shape, top=2):
    return r.integers(-top, top + 1, shape).astype(np.float64)


def check(got, exact, size, q, kind, rows, magnitude):
    """`size` and `magnitude`: sums of |s| (q + z) |x| and of |w x|."""
    half, tiny = HALF[kind]
    c = got.double().cpu().numpy()
    K, ng = q.cols, -(-q.cols // q.group)
    bound = (2 * K + 4 * ng + 24) * 2.0 ** -23 * size + half * np.abs(c) + tiny
    if rows > w4.ROWS:
        bound = ((K + 8) * 2.0 ** -23 + half) * (1 + half) * magnitude + half * np.abs(c) + K * tiny
    wrong = ~(np.abs(c - exact) <= bound)
    assert not wrong.any(), (int(wrong.sum()), np.argwhere(wrong)[:3].tolist(), float(np.abs(c - exact).max()))


PRODUCTS = [(1, 1, 1), (1, 16, 32), (1, 100, 4096), (2, 33, 95), (3, 17, 31), (16, 48, 1024), (17, 31, 130), (5, 520, 2090),
            (32, 64, 256), (33, 72, 257), (64, 130, 1000), (65, 15, 512), (128, 200, 640), (129, 40, 96), (200, 136, 1000),
            (7, 40, 8192)]


@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("group", w4.GROUPS)
@pytest.mark.parametrize("kind", SCALES)
@pytest.mark.parametrize("M, N, K", PRODUCTS)
def test_product(M, N, K, kind, group, zeros):
    r = rng(M, N, K, group)
    # Whole numbers: sums of up to K * 2 * 15 * 2^2 are exact, results are
    # rounded once.
    q, value, _ = coded(r, (N, K), group, kind, zeros, -1, 2, whole=True)
    x, ex = dense(whole(r, (M, K)), kind)
    want = torch.from_numpy(ex @ value.T).to(TYPES[kind])
    assert torch.equal(w4.matmul(x, q).cpu(), want)
    # General values, strided operands and results.
    for pad, shift in ((0, 0), (8, 0), (3, 1)):
        q, value, size = coded(r, (N, K), group, kind, zeros, pad=pad)
        x, ex = dense(r.standard_normal((M, K)) * np.exp(r.uniform(-3, 3, (M, 1))), kind, pad, shift)
        y, _ = dense(np.zeros((M, N)), kind, pad, shift)
        y._base.fill_(7.0)
        assert w4.matmul(x, q, out=y) is y
        check(y, ex @ value.T, np.abs(ex) @ size.T, q, kind, M, np.abs(ex) @ np.abs(value).T)
        y.fill_(7.0)
        assert bool((y._base == 7.0).all()), "wrote outside the result"


@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("kind", SCALES)
@pytest.mark.parametrize("N, K, group", [(40, 128, 64), (33, 128, 32), (17, 384, 128), (50, 4224, 128), (16, 96, 32)])
def test_scale_rows_longer_than_their_groups(N, K, group, kind, zeros):
    """Rows of scales and zero points as `empty` lays them out, whole 256 k,
    where the last has fewer: the bytes behind the groups hold anything."""
    r = rng(6, N, K)
    for M in (1, 20, 70):
        q, value, _ = coded(r, (N, K), group, kind, zeros, -1, 2, whole=True)
        own = w4.empty((N, K), group, "cuda", TYPES[kind], zeros)
        own.scales._base.fill_(float("nan"))
        own.scales.copy_(q.scales)
        own.codes.copy_(q.codes)
        if zeros:
            own.zeros._base.fill_(GUARD)
            own.zeros.copy_(q.zeros)
        x, ex = dense(whole(r, (M, K)), kind)
        assert torch.equal(w4.matmul(x, own).cpu(), torch.from_numpy(ex @ value.T).to(TYPES[kind]))


EXPERTS = [
    (1, 1, 1, [0, 1]),
    (8, 128, 64, [0, 1, 2, 3, 4, 5, 6, 7, 8]),
    (1, 33, 7, [0, 0, 1, 1]),
    (5, 256, 24, [0, 0, 5, 5, 5]),
    (70, 512, 40, [3, 10, 10, 61, 66]),
    (130, 130, 129, [0, 64, 65, 130]),
    (200, 72, 48, list(range(0, 201))),
    (90, 288, 33, [0] * 60 + [45] + [90] * 70),
    (300, 1000, 72, [20, 20, 20, 280]),
    (400, 96, 40, [10, 300, 390]),          # more than 128 rows a group: dequantised
    (100, 64, 64, [-5, 30, -2 ** 31, 70, 2 ** 31 - 1]),
    (100, 64, 64, [50, 20, 80, 60, 90]),
]


@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("group", w4.GROUPS)
@pytest.mark.parametrize("kind", SCALES)
@pytest.mark.parametrize("T, K, N, offsets", EXPERTS)
def test_grouped_product(T, K, N, offsets, kind, group, zeros):
    r = rng(T, N, K, group, 1)
    G = len(offsets) - 1
    q, value, _ = coded(r, (G, N, K), group, kind, zeros, -1, 2, whole=True)
    x, ex = dense(whole(r, (T, K)), kind)
    exact, _ = grouped_oracle.product(ex, value.transpose(0, 2, 1), offsets)
    assert torch.equal(w4.grouped_matmul(x, q, gpu(offsets)).cpu(), torch.from_numpy(exact).to(TYPES[kind]))
    rows = T if T > w4.ROWS * G else 1
    free = grouped_oracle.outside(offsets, T)
    for pad, shift in ((0, 0), (3, 1)):
        q, value, size = coded(r, (G, N, K), group, kind, zeros, pad=pad)
        x, ex = dense(r.standard_normal((T, K)) * np.exp(r.uniform(-3, 3, (T, 1))), kind, pad, shift)
        exact, mag = grouped_oracle.product(ex, value.transpose(0, 2, 1), offsets)
        size = grouped_oracle.product(np.abs(ex), size.transpose(0, 2, 1), offsets)[0]
        check(w4.grouped_matmul(x, q, gpu(offsets)), exact, size, q, kind, rows, mag)
        y, _ = dense(np.zeros((T, N)), kind, pad, shift)
        y._base.fill_(7.0)
        w4.grouped_matmul(x, q, gpu(offsets), out=y)
        assert bool((y[torch.from_numpy(free).cuda()] == 7.0).all()), "wrote a row of no group"
        keep = torch.from_numpy(~free).cuda()
        check(y[keep], exact[~free], size[~free], q, kind, rows, mag[~free])
        y.fill_(7.0)
        assert bool((y._base == 7.0).all()), "wrote outside the result"


@pytest.mark.parametrize("kind", SCALES)
@pytest.mark.parametrize("T", [12, 300])
@pytest.mark.parametrize("K", [256, 250])
def test_nan_stays_where_it_is(K, T, kind):
    """A NaN scale reaches its own column of its own expert, a NaN activation
    its own row; experts without rows and rows of no group reach nothing."""
    r = rng(2, K, T)
    q, value, _ = coded(r, (3, 40, K), 64, kind, True, -1, 2, whole=True)
    offsets = [2, T // 2, T // 2, T - 2]
    q.scales[1] = float("nan")
    x, ex = dense(whole(r, (T, K)), kind)
    x[:2], x[-2:] = float("nan"), float("inf")
    ex[:2] = ex[-2:] = 0
    exact, _ = grouped_oracle.product(ex, value.transpose(0, 2, 1), offsets)
    want = torch.from_numpy(exact).to(TYPES[kind])
    assert torch.equal(w4.grouped_matmul(x, q, gpu(offsets)).cpu(), want)
    q.scales[0, 5, 1] = float("nan")
    x[T // 2 + 1, 7] = float("nan")
    y = w4.grouped_matmul(x, q, gpu(offsets)).cpu()
    bad = torch.zeros(T, 40, dtype=torch.bool)
    bad[2:T // 2, 5] = True
    bad[T // 2 + 1] = True
    assert torch.equal(y.isnan(), bad) and torch.equal(y[~bad], want[~bad])


@pytest.mark.parametrize("kind", SCALES)
def test_empty_sizes(kind):
    t = TYPES[kind]
    x = lambda *s: torch.ones(*s, dtype=t, device="cuda")  # noqa: E731
    for zeros in (True, False):
        q = w4.quantize(x(40, 64), 32, zeros)
        assert w4.matmul(x(0, 64), q).shape == (0, 40)
        none = w4.empty((0, 64), 32, "cuda", t, zeros)
        assert w4.matmul(x(5, 64), none).shape == (5, 0) and w4.dequantize(none).shape == (0, 64)
        narrow = w4.empty((40, 0), 32, "cuda", t, zeros)
        for rows in (5, 200):
            y = w4.matmul(x(rows, 0), narrow)
            assert y.shape == (rows, 40) and bool((y == 0).all())
        stack = w4.quantize(x(2, 40, 64), 32, zeros)
        assert w4.grouped_matmul(x(0, 64), stack, gpu([0, 0, 0])).shape == (0, 40)
        y = w4.grouped_matmul(x(300, 64), stack, gpu([0, 0, 0]))
        assert bool((y == 0).all())
        y = w4.grouped_matmul(x(5, 64), w4.empty((0, 40, 64), 32, "cuda", t, zeros), gpu([0]))
        assert y.shape == (5, 40) and bool((y == 0).all())


@pytest.mark.parametrize("kind", SCALES)
@pytest.mark.parametrize("T", [9, 400])
def test_captured_calls(T, kind):
    r = rng(3, T)
    K, N, G = 288, 136, 3
    q, _, _ = coded(r, (G, N, K), 32, kind, True, -1, 2, whole=True)
    x = dense(whole(r, (T, K)), kind)[0]
    offsets = gpu([0, 2, 5, T])
    y, z = (torch.empty(T, N, dtype=TYPES[kind], device="cuda") for _ in range(2))
    one = q[1]

    def step():
        w4.grouped_matmul(x, q, offsets, out=y)
        w4.matmul(x, one, out=z)

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
        y.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone(), z.clone()
        y.fill_(3.0)
        z.fill_(3.0)
        torch.cuda.synchronize()
        step()
        assert torch.equal(got[0], y) and torch.equal(got[1], z)


@pytest.mark.parametrize("kind", SCALES)
@pytest.mark.parametrize("M", [1, 40, 150])
def test_calls_on_other_streams_and_repeated_ones_agree(M, kind):
    r = rng(4, M)
    q, value, _ = coded(r, (264, 1024), 128, kind, True)
    x, ex = dense(r.standard_normal((M, 1024)), kind)
    first = w4.matmul(x, q)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    results = [w4.matmul(x, q, stream=s) for s in streams for _ in range(3)]
    for s in streams:
        s.synchronize()
    assert all(torch.equal(y, first) for y in results)


# ---------------------------------------------------------------------------
# The operators together, as they are used
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("kind", SCALES)
def test_a_trained_layer_of_experts_served_in_4_bits(kind):
    """Two training steps of a layer of experts, its weights to 4 bits, and a
    decoding step: the products see the weights that the codes stand for."""
    r = rng(5)
    T, K, N, G = 96, 128, 72, 4
    half, tiny = HALF[kind]
    w = dense(r.standard_normal((G, K, N)) / 8, kind)[0].requires_grad_(True)
    for step in range(2):
        x, dy = dense(r.standard_normal((T, K)), kind)[0], dense(r.standard_normal((T, N)), kind)[0]
        offsets = gpu(np.sort(r.integers(0, T + 1, G + 1)))
        grouped.linear(x, w, offsets).backward(dy)
        dw, size = grouped_oracle.gradient(x.double().cpu().numpy(), dy.double().cpu().numpy(), offsets.cpu().numpy())
        g = w.grad.double().cpu().numpy()
        assert (np.abs(g - dw) <= (T + 8) * 2.0 ** -23 * size + half * np.abs(g) + tiny).all()
        with torch.no_grad():
            w -= 0.05 * w.grad
        w.grad = None
    q = w4.quantize(w.detach(), 64, transposed=True)
    assert q.shape == (G, N, K)
    for e in range(G):
        check_codes(q[e], w[e].detach().t().double().cpu().numpy(), 64, kind)
    value = w4.dequantize(q, torch.float32).double().cpu().numpy()
    codes = np.stack([oracle.unpack(c, K) for c in q.codes.cpu().numpy()])
    spread = np.repeat(q.scales.double().cpu().numpy(), 64, axis=2) * (32.0 + codes + np.repeat(q.zeros.cpu().numpy(), 64, axis=2))
    x, ex = dense(r.standard_normal((6, K)), kind)
    offsets = [0, 1, 1, 4, 6]
    exact, mag = grouped_oracle.product(ex, value.transpose(0, 2, 1), offsets)
    size = grouped_oracle.product(np.abs(ex), np.abs(spread).transpose(0, 2, 1), offsets)[0]
    check(w4.grouped_matmul(x, q, gpu(offsets)), exact, size, q, kind, 1, mag)


def test_torch_forms_refuse():
    x = torch.zeros(4, 128, device="cuda", dtype=torch.bfloat16)
    w = torch.zeros(2, 6, 128, device="cuda", dtype=torch.bfloat16)
    stack, q = w4.quantize(w), w4.quantize(w[0])
    at = gpu([0, 1, 4])
    for error, call in [
        (TypeError, lambda: w4.matmul(x.half(), q)), (TypeError, lambda: w4.matmul(x.float(), q)),
        (ValueError, lambda: w4.matmul(x[:, :96], q)), (ValueError, lambda: w4.matmul(x, stack)),
        (ValueError, lambda: w4.matmul(x.t(), q)), (ValueError, lambda: w4.matmul(x[0], q)),
        (ValueError, lambda: w4.matmul(x, q, out=x)), (ValueError, lambda: w4.matmul(x, q, out=x[:, :6].float())),
        (ValueError, lambda: w4.grouped_matmul(x, q, at)), (ValueError, lambda: w4.grouped_matmul(x, stack, at[:2])),
        (TypeError, lambda: w4.grouped_matmul(x, stack, at.long())), (TypeError, lambda: w4.grouped_matmul(x.half(), stack, at)),
        (ValueError, lambda: w4.quantize(w, 16)), (TypeError, lambda: w4.quantize(w, scale_dtype=torch.float32)),
        (TypeError, lambda: w4.quantize(w.double())), (ValueError, lambda: w4.quantize(w[0, 0])),
        (ValueError, lambda: w4.quantize(w, out=q)), (ValueError, lambda: w4.quantize(w[:0])),
        (TypeError, lambda: w4.dequantize(q, torch.float64)), (ValueError, lambda: w4.dequantize(q, out=x)),
        (TypeError, lambda: w4.dequantize(w)),
        (gemm.GemmError, lambda: w4.matmul(x, w4.W4Tensor(q.codes, q.scales, q.zeros, 128, 128), out=x[:, :6])),
    ]:
        with pytest.raises(error):
            call()
