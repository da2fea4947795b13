"""Microscaled operators on the GPU against the 64-bit oracle.

Quantisation is exact: codes and scales are compared bit for bit.  Products
and gradients are compared two ways: inputs chosen so that every FP32
partial sum is exact must give the exact result bit for bit, and general
inputs must be within

    |C - exact| <= (n + 8) * 2^-23 * sum|a b| + half(type) * |C|

(n FP32 additions, each off by at most one unit in the last place, whatever
their order; half(type) the output's half step relative to the value, plus
half the smallest subnormal)."""
import numpy as np
import pytest

from dense_gemm_row_amd import gemm, mx
from tests import mx_oracle as oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF = {t: (torch.finfo(TYPES[t]).eps / 2, torch.finfo(TYPES[t]).smallest_normal * torch.finfo(TYPES[t]).eps / 2)
        for t in TYPES}
GUARD = 0xA5


def rng(*seed):
    return np.random.default_rng(seed)


def values(r, rows, cols):
    """Rows of very different size, zeros, zero blocks and both signs."""
    x = r.standard_normal((rows, cols)) * np.exp(r.uniform(-8, 8, (rows, 1)))
    x[r.random((rows, cols)) < 0.05] = 0
    if cols > 40:
        x[rows // 2, 32:64] = 0
    return x


def dense(x, kind, pad=0, shift=0):
    """x on the GPU in a type, its rows pad elements longer and its start
    moved by shift elements; (tensor, its exact values)."""
    rows, cols = x.shape
    flat = torch.full((rows * (cols + pad) + shift,), 9.0, dtype=TYPES[kind], device="cuda")
    t = flat[shift:].view(rows, cols + pad)[:, :cols]
    t.copy_(torch.from_numpy(np.ascontiguousarray(x)))
    return t, t.double().cpu().numpy()


def guarded(rows, cols, fmt, pad=0):
    """A coded matrix in larger buffers filled with a guard byte."""
    nb = -(-cols // 32)
    width = nb * mx.BLOCK_BYTES[fmt]
    codes = torch.full((rows + 1, width + 16 * pad), GUARD, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows + 1, nb + pad), GUARD, dtype=torch.uint8, device="cuda")
    return mx.MxTensor(codes[:rows, :width], scales[:rows, :nb], cols, fmt), codes, scales


def assert_guards(rows, q, codes, scales):
    assert bool((codes[rows:] == GUARD).all()) and bool((codes[:, q.codes.shape[1]:] == GUARD).all())
    assert bool((scales[rows:] == GUARD).all()) and bool((scales[:, q.scales.shape[1]:] == GUARD).all())


def check_codes(q, exact, fmt):
    want_c, want_s = oracle.quantize(exact, fmt)
    got_s, got_c = q.scales.cpu().numpy(), q.codes.cpu().numpy()
    assert np.array_equal(got_s, want_s)
    assert np.array_equal(got_c, oracle.pack(want_c, fmt))


SIZES = [(1, 1), (1, 31), (1, 32), (2, 33), (3, 257), (5, 1000), (64, 64), (33, 4096), (257, 130), (128, 96)]


@pytest.mark.parametrize("fmt", [mx.E2M1, mx.E4M3])
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("rows, cols", SIZES)
def test_quantise_rows_and_columns(rows, cols, kind, fmt):
    for pad, shift in ((0, 0), (3, 0), (8, 0), (0, 1)):
        x, exact = dense(values(rng(rows, cols), rows, cols).clip(-6e4, 6e4), kind, pad, shift)
        for trans in (False, True):
            e = exact.T if trans else exact
            q, codes, scales = guarded(e.shape[0], e.shape[1], fmt, pad=1 if pad else 0)
            mx.quantize(x, fmt, transposed=trans, out=q)
            torch.cuda.synchronize()
            check_codes(q, e, fmt)
            assert_guards(e.shape[0], q, codes, scales)


@pytest.mark.parametrize("fmt", [mx.E2M1, mx.E4M3])
@pytest.mark.parametrize("kind", TYPES)
def test_quantise_every_midpoint_and_border(kind, fmt):
    """Each grid value, midpoint and their neighbours in the type, in blocks
    whose scale is one, then scaled by the type's powers of two; blocks whose
    largest magnitude is at and next to the borders of the scale's rule."""
    g = oracle.GRID[fmt]
    top = g[-1]
    pts = np.concatenate([g, (g[1:] + g[:-1]) / 2])
    t = torch.from_numpy(pts).to(TYPES[kind])
    around = torch.cat([t, torch.nextafter(t, torch.full_like(t, 1e4)), torch.nextafter(t, torch.full_like(t, -1e4))])
    p = around.double().numpy()
    p = p[np.abs(p) <= top]
    p = np.concatenate([p, -p])
    p = np.concatenate([p, np.zeros(-len(p) % 31)]).reshape(-1, 31)
    rows = [np.concatenate([[top], r]) for r in p]
    for border in (top, 4 * top / 3, 256.0, 512.0, 4.0, 8.0):
        b = torch.tensor([border]).to(TYPES[kind])
        for v in (b, torch.nextafter(b, torch.full_like(b, 1e4)), torch.nextafter(b, torch.zeros_like(b))):
            rows.append(np.concatenate([[float(v)], np.linspace(-1, 1, 31) * float(v)]))
    base = np.stack(rows)
    for e in ((0, 3, -6) if kind == "f16" else (0, 3, -100, 100)):
        for x, exact in [dense(base * 2.0 ** e, kind), dense((base * 2.0 ** e).T, kind)]:
            trans = exact.shape[0] == 32 and exact.shape[1] != 32
            q = mx.quantize(x, fmt, transposed=trans)
            check_codes(q, exact.T if trans else exact, fmt)


@pytest.mark.parametrize("fmt", [mx.E2M1, mx.E4M3])
@pytest.mark.parametrize("kind", TYPES)
def test_quantise_special_values(kind, fmt):
    fi = torch.finfo(TYPES[kind])
    x = np.zeros((9, 70))
    x[0, 3] = np.nan
    x[1, 40] = np.inf
    x[2, 69] = -np.inf  # in the partial block
    x[3, :] = fi.max
    x[4, :] = fi.smallest_normal * fi.eps  # smallest subnormal
    x[5, 5] = -fi.min
    x[6, ::2] = -0.0
    x[7, :] = fi.smallest_normal
    x[8, 31] = fi.max
    x[8, :31] = 1.0
    t, exact = dense(x, kind)
    for trans in (False, True):
        src = t.t().contiguous() if trans else t
        q = mx.quantize(src, fmt, transposed=trans)
        check_codes(q, exact, fmt)
        back = mx.dequantize(q, dtype=torch.float32).double().cpu().numpy()
        want = oracle.values(q.codes.cpu().numpy(), q.scales.cpu().numpy(), 70, fmt)
        assert np.array_equal(back, want.astype(np.float32).astype(np.float64), equal_nan=True)
        assert np.isnan(back[0, :32]).all() and np.isnan(back[1, 32:64]).all() and np.isnan(back[2, 64:]).all()
        assert not np.isnan(back[3:]).any() and not np.isnan(back[0, 32:]).any()


@pytest.mark.parametrize("fmt", [mx.E2M1, mx.E4M3])
@pytest.mark.parametrize("kind", TYPES)
def test_dequantise_every_code_and_scale(kind, fmt):
    """Every code with every scale byte, rounded to the type once."""
    n = 256
    codes = np.tile(np.arange(256, dtype=np.uint8), (n, 1))  # 8 blocks of 4-bit pairs 16 bytes, or of 8-bit codes
    nb = 256 // mx.BLOCK_BYTES[fmt]
    scales = np.tile(np.arange(n, dtype=np.uint8)[:, None], (1, nb))
    q = mx.MxTensor(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), nb * 32, fmt)
    with np.errstate(all="ignore"):
        want = torch.from_numpy(oracle.values(codes, scales, nb * 32, fmt)).to(TYPES[kind])
    for trans in (False, True):
        got = mx.dequantize(q, dtype=TYPES[kind], transposed=trans).cpu()
        assert torch.equal(torch.nan_to_num((got.t() if trans else got).float(), nan=12345.0),
                           torch.nan_to_num(want.float(), nan=12345.0))


@pytest.mark.parametrize("fmt", [mx.E2M1, mx.E4M3])
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("rows, cols", SIZES)
def test_dequantise_sizes_and_strides(rows, cols, kind, fmt):
    r = rng(rows, cols, 7)
    x = values(r, rows, cols).clip(-1e3, 1e3)
    for trans in (False, True):
        q = mx.quantize(dense(x.T if trans else x, "f32")[0], fmt, transposed=trans)  # codes rows x cols
        want = torch.from_numpy(oracle.values(q.codes.cpu().numpy(), q.scales.cpu().numpy(), cols, fmt)).to(TYPES[kind])
        for pad, shift in ((0, 0), (8, 0), (5, 1)):
            shape = (cols, rows) if trans else (rows, cols)
            out, _ = dense(np.zeros(shape), kind, pad, shift)
            whole = out._base if out._base is not None else out
            whole.fill_(3.0)
            mx.dequantize(q, out=out, transposed=trans)
            assert torch.equal((out.t() if trans else out).cpu(), want)
            out.fill_(3.0)
            assert bool((whole == 3.0).all()), "wrote outside the matrix"


def random_coded(r, rows, cols, fmt, lo, hi, pad=0):
    """Random codes (no E4M3 NaN) and scale bytes in [lo, hi), padding zeros."""
    nb = -(-cols // 32)
    elem = r.integers(0, 16 if fmt == mx.E2M1 else 256, (rows, nb * 32)).astype(np.uint8)
    elem[(elem & 0x7f) == 0x7f] = 0x38
    elem[:, cols:] = 0
    packed = oracle.pack(elem, fmt)
    scales = r.integers(lo, hi, (rows, nb)).astype(np.uint8)
    q, codes, sc = guarded(rows, cols, fmt, pad)
    q.codes.copy_(torch.from_numpy(packed))
    q.scales.copy_(torch.from_numpy(scales))
    return q, oracle.values(packed, scales, cols, fmt)


PRODUCTS = [(1, 1, 1), (1, 16, 32), (1, 100, 4096), (2, 33, 95), (16, 48, 1024), (17, 31, 130), (5, 520, 2090),
            (64, 64, 64), (100, 72, 257), (129, 130, 1000), (256, 256, 512), (300, 513, 640), (33, 1000, 4000)]


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("m, n, k", PRODUCTS)
def test_product_of_exact_sums(m, n, k, out):
    """Scales 2^-1 .. 2^0: sums are multiples of 1/16 below 36 * k < 2^20, so
    FP32 holds each exactly, and the result is the exact one, rounded."""
    r = rng(m, n, k)
    a, av = random_coded(r, m, k, mx.E2M1, 126, 128, pad=k % 2)
    b, bv = random_coded(r, n, k, mx.E2M1, 126, 128, pad=n % 2)
    want = torch.from_numpy(av @ bv.T)
    c, _ = dense(np.zeros((m, n)), out, pad=k % 3, shift=n % 2)
    c._base.fill_(7.0)
    mx.matmul(a, b, out=c)
    assert torch.equal(c.cpu(), want.to(TYPES[out]))
    c.fill_(7.0)
    assert bool((c._base == 7.0).all()), "wrote outside the matrix"


def near(got, want, size, n, kind):
    half, tiny = HALF[kind]
    return np.abs(got - want) <= (n + 8) * 2.0 ** -23 * size + half * np.abs(want) + tiny


@pytest.mark.parametrize("out", TYPES)
@pytest.mark.parametrize("m, n, k", PRODUCTS)
def test_product_of_general_scales(m, n, k, out):
    r = rng(m, n, k, 2)
    a, av = random_coded(r, m, k, mx.E2M1, 110, 131)
    b, bv = random_coded(r, n, k, mx.E2M1, 110, 131)
    got = mx.matmul(a, b, out_dtype=TYPES[out]).double().cpu().numpy()
    want, size = av @ bv.T, np.abs(av) @ np.abs(bv).T
    keep = size < 6e4  # in binary16's range
    assert np.all(near(got, want, size, k, out)[keep])


@pytest.mark.parametrize("m", [1, 7, 40])
@pytest.mark.parametrize("kind", TYPES)
def test_product_of_values_is_quantise_then_product(m, kind):
    r = rng(m, 5)
    x, exact = dense(values(r, m, 1000).clip(-1e3, 1e3), kind, pad=8)
    w, wv = random_coded(r, 77, 1000, mx.E2M1, 120, 126)
    got = mx.matmul(x, w, out_dtype=torch.float32)
    assert torch.equal(got, mx.matmul(mx.quantize(x), w, out_dtype=torch.float32))
    xv = oracle.round_trip(exact, "e2m1")
    assert np.all(near(got.double().cpu().numpy(), xv @ wv.T, np.abs(xv) @ np.abs(wv).T, 1000, "f32"))


@pytest.mark.parametrize("m, n, k", [(1, 40, 64), (3, 257, 96), (70, 65, 320), (256, 264, 512)])
@pytest.mark.parametrize("out", TYPES)
def test_product_epilogue(m, n, k, out):
    r = rng(m, n, k, 3)
    a, av = random_coded(r, m, k, mx.E2M1, 126, 128)
    b, bv = random_coded(r, n, k, mx.E2M1, 126, 128)
    bias = torch.from_numpy(r.integers(-64, 64, n) / 4.0).float().cuda()
    old, oldv = dense(r.integers(-32, 32, (m, n)) / 2.0, out)
    exact = 0.5 * (av @ bv.T) + 2.0 * oldv + bias.double().cpu().numpy()
    mx.matmul(a, b, out=old, alpha=0.5, beta=2.0, bias=bias, act=gemm.ACT_RELU)
    assert torch.equal(old.cpu(), torch.from_numpy(np.maximum(exact, 0.0)).to(TYPES[out]))
    # beta 0 does not read C.
    c = torch.full((m, n), float("nan"), dtype=TYPES[out], device="cuda")
    mx.matmul(a, b, out=c, alpha=-1.0)
    assert torch.equal(c.cpu(), torch.from_numpy(-(av @ bv.T)).to(TYPES[out]))


def test_empty_sums_and_sizes():
    for m in (1, 40):
        a, b = mx.empty(m, 0, mx.E2M1, "cuda"), mx.empty(5, 0, mx.E2M1, "cuda")
        assert not mx.matmul(a, b).any()
        c = torch.ones(m, 5, device="cuda")
        mx.matmul(a, b, out=c, beta=3.0, bias=torch.ones(5, device="cuda"))
        assert bool((c == 4.0).all())
    assert mx.matmul(mx.empty(0, 64, mx.E2M1, "cuda"), mx.empty(5, 64, mx.E2M1, "cuda")).shape == (0, 5)
    assert mx.matmul(mx.empty(3, 64, mx.E2M1, "cuda"), mx.empty(0, 64, mx.E2M1, "cuda")).shape == (3, 0)
    kept = mx.checkpoint(torch.empty(0, 6, device="cuda"))
    assert kept.shape == (6, 0)
    dw = torch.ones(6, 4, device="cuda")
    mx.weight_grad(kept, torch.empty(0, 4, device="cuda"), out=dw, beta=2.0)
    assert bool((dw == 2.0).all())
    assert not mx.weight_grad(kept, torch.empty(0, 4, device="cuda")).any()
    assert mx.restore(kept).shape == (0, 6)


@pytest.mark.parametrize("m", [3, 200])
def test_product_with_nan_blocks(m):
    """A NaN scale reaches its row (or column) of the result, no other."""
    r = rng(m, 9)
    a, _ = random_coded(r, m, 320, mx.E2M1, 126, 128)
    b, _ = random_coded(r, 200, 320, mx.E2M1, 126, 128)
    a.scales[m // 2, 3] = 255
    b.scales[77, 9] = 255
    bad = torch.isnan(mx.matmul(a, b, out_dtype=torch.float32)).cpu().numpy()
    want = np.zeros((m, 200), bool)
    want[m // 2] = True
    want[:, 77] = True
    assert np.array_equal(bad, want)


GRADS = [(1, 1, 1), (31, 16, 16), (32, 64, 64), (33, 17, 31), (257, 130, 72), (1000, 64, 65), (64, 300, 256),
         (100, 256, 513), (2048, 128, 136), (333, 520, 263), (4097, 65, 24)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("t, f, n", GRADS)
def test_gradient_of_exact_sums(t, f, n, kind):
    """Integers of |x| <= 8 (exact in E4M3) and |dy| <= 8: sums below 2^24."""
    r = rng(t, f, n)
    x, _ = dense(r.integers(-8, 9, (t, f)).astype(float), "bf16", pad=f % 2)
    dy, dyv = dense(r.integers(-8, 9, (t, n)).astype(float), kind, pad=t % 3, shift=n % 2)
    kept = mx.checkpoint(x)
    xv = x.double().cpu().numpy()
    assert np.array_equal(mx.restore(kept, torch.float32).double().cpu().numpy(), xv)
    for out in TYPES:
        dw, _ = dense(np.zeros((f, n)), out, pad=n % 3, shift=f % 2)
        dw._base.fill_(7.0)
        mx.weight_grad(kept, dy, out=dw)
        assert torch.equal(dw.cpu(), torch.from_numpy(xv.T @ dyv).to(TYPES[out]))
        dw.fill_(7.0)
        assert bool((dw._base == 7.0).all()), "wrote outside the matrix"


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("t, f, n", GRADS)
def test_gradient_of_general_values(t, f, n, kind):
    """dY in its whole precision: a binary16 or FP32 gradient is not rounded
    to bfloat16 (that would be 2^-9 of each product, far over this bound)."""
    r = rng(t, f, n, 2)
    x, _ = dense(values(r, t, f), "f32")
    kept = mx.checkpoint(x)
    xv = oracle.values(kept.codes.cpu().numpy(), kept.scales.cpu().numpy(), t, "e4m3")
    dy, dyv = dense(r.standard_normal((t, n)) * 1e-3, kind, pad=8 * (n % 2))
    terms = {"bf16": 1, "f16": 2, "f32": 3}[kind]
    got = mx.weight_grad(kept, dy).double().cpu().numpy()
    want, size = xv @ dyv, np.abs(xv) @ np.abs(dyv)
    assert np.all(near(got, want, size, terms * t, "f32"))
    acc = torch.full((f, n), 0.5, device="cuda")
    mx.weight_grad(kept, dy, out=acc, alpha=2.0, beta=-1.0)
    assert np.all(near(acc.double().cpu().numpy(), 2 * want - 0.5, 2 * size + 0.5, terms * t + 2, "f32"))


def test_gradient_matches_differences():
    """Central differences of sum(dY * (x^ W)) in 64 bits at the checkpoint's
    values: the sum is linear in W, so they are exact up to rounding."""
    r = rng(11)
    t, f, n = 65, 24, 20
    kept = mx.checkpoint(torch.from_numpy(r.standard_normal((t, f))).float().cuda())
    xv = oracle.values(kept.codes.cpu().numpy(), kept.scales.cpu().numpy(), t, "e4m3")
    dy, dyv = dense(r.standard_normal((t, n)), "f32")
    w = r.standard_normal((f, n))
    got = mx.weight_grad(kept, dy).double().cpu().numpy()
    x8 = xv.T
    for i, j in [(0, 0), (3, 7), (23, 19), (11, 0)]:
        d = np.zeros((f, n))
        d[i, j] = 1e-3
        diff = (np.sum(dyv * (x8 @ (w + d))) - np.sum(dyv * (x8 @ (w - d)))) / 2e-3
        assert abs(got[i, j] - diff) <= (3 * t + 8) * 2.0 ** -23 * (np.abs(xv) @ np.abs(dyv))[i, j] + 1e-9


def test_gradient_of_infinite_and_nan_values():
    """A NaN block or a non-finite dY element reaches exactly its feature or
    column; FP32 and binary16 terms keep infinities infinite."""
    r = rng(12)
    x = r.standard_normal((100, 40)) + 3.0  # nowhere zero
    x = np.where(np.abs(x) < 0.5, 0.5, x)
    x[50, 7] = np.inf
    kept = mx.checkpoint(torch.from_numpy(x).float().cuda())
    for kind in TYPES:
        dy = r.standard_normal((100, 30))
        dy[10, 3] = np.inf
        dy[20, 5] = np.nan
        t, _ = dense(dy, kind)
        g = mx.weight_grad(kept, t).cpu().numpy()
        assert np.isnan(g[7]).all() and np.isnan(g[:, 5]).all()
        rest = np.delete(np.delete(g, 7, 0), [3, 5], 1)
        assert np.isfinite(rest).all()
        assert np.isinf(np.delete(g[:, 3], 7)).all()


def test_other_streams_give_the_same():
    """Work and allocations on a stream of the caller's, given or current."""
    r = rng(13)
    x = torch.from_numpy(r.standard_normal((300, 512))).to(torch.bfloat16).cuda()
    w = torch.from_numpy(r.standard_normal((512, 264))).to(torch.bfloat16).cuda()
    dy = torch.from_numpy(r.standard_normal((300, 264))).to(torch.bfloat16).cuda()
    wq = mx.quantize(w, transposed=True)
    want = mx.matmul(x, wq), mx.weight_grad(mx.checkpoint(x), dy), mx.restore(mx.checkpoint(x))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = (mx.matmul(x, wq, stream=s), mx.weight_grad(mx.checkpoint(x, stream=s), dy, stream=s),
           mx.restore(mx.checkpoint(x, stream=s), stream=s))
    with torch.cuda.stream(s):
        got2 = mx.matmul(x, wq), mx.weight_grad(mx.checkpoint(x), dy), mx.restore(mx.checkpoint(x))
    s.synchronize()
    for a, b, c in zip(want, got, got2):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_graph_replays_match_eager():
    """The whole layer captured once and replayed over changed inputs, with
    eager work in between."""
    r = rng(14)
    shape = (160, 512)
    x = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    w = torch.from_numpy(r.standard_normal((512, 256)) / 20).to(torch.bfloat16).cuda()
    dy = torch.zeros(160, 256, dtype=torch.bfloat16, device="cuda")

    def step():
        wq = mx.quantize(w, transposed=True)
        kept = mx.checkpoint(x)
        return mx.matmul(x, wq), mx.weight_grad(kept, dy), mx.restore(kept)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for k in range(4):
        x.copy_(torch.from_numpy(r.standard_normal(shape)))
        dy.copy_(torch.from_numpy(r.standard_normal((160, 256))))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, step()):
            assert torch.equal(a, b), k


@pytest.mark.parametrize("kind", TYPES)
def test_linear_layer_trains(kind):
    """mx.linear's output and gradients against the formulas in 64 bits."""
    r = rng(15)
    t, k, n = 96, 128, 64
    x, xe = dense(r.standard_normal((t, k)), kind)
    w, we = dense(r.standard_normal((k, n)) / 8, kind)
    x.requires_grad_(True)
    w.requires_grad_(True)
    wq = mx.quantize(w.detach(), transposed=True)
    y = mx.linear(x, w, wq)
    q = lambda v, fmt: oracle.round_trip(v, fmt)  # noqa: E731
    xq, wv = q(xe, "e2m1"), q(we.T, "e2m1").T
    assert np.all(near(y.detach().double().cpu().numpy(), xq @ wv, np.abs(xq) @ np.abs(wv), k, kind))
    dy, dye = dense(r.standard_normal((t, n)), kind)
    y.backward(dy)
    x8 = q(xe.T, "e4m3").T
    assert np.all(near(w.grad.double().cpu().numpy(), x8.T @ dye, np.abs(x8).T @ np.abs(dye), 3 * t, kind))
    assert np.all(near(x.grad.double().cpu().numpy(), dye @ we.T, np.abs(dye) @ np.abs(we).T, n, kind))
    # An expanded gradient (of a sum) and a weight that needs none.
    x2 = x.detach().clone().requires_grad_(True)
    mx.linear(x2, w.detach(), wq).sum().backward()
    assert np.all(near(x2.grad.double().cpu().numpy(), np.ones((t, n)) @ we.T, np.abs(np.ones((t, n)) @ np.abs(we.T)), n, kind))


def test_offsets_past_32_bits():
    """Rows that lie past 2^31 and 2^32 bytes of their buffer."""
    big = torch.empty(5 << 30, dtype=torch.uint8, device="cuda")
    r = rng(16)
    x, exact = dense(r.standard_normal((3, 64)), "bf16")
    codes = big.view(5 << 10, 1 << 20)[::2048][:3, :32]  # rows 2 GiB apart
    q = mx.MxTensor(codes, torch.empty(3, 2, dtype=torch.uint8, device="cuda"), 64)
    mx.quantize(x, out=q)
    check_codes(q, exact, "e2m1")
    b = mx.quantize(dense(r.standard_normal((20, 64)), "bf16")[0])
    near_q = mx.quantize(x)
    assert torch.equal(mx.matmul(q, b), mx.matmul(near_q, b))
    assert torch.equal(mx.matmul(b, q), mx.matmul(b, near_q))
    assert torch.equal(mx.dequantize(q), mx.dequantize(near_q))
    wide = big.view(torch.bfloat16)[: (5 << 29)].view(5, 1 << 29)[:, :64]  # rows 1 GiB apart
    wide.copy_(torch.from_numpy(r.standard_normal((5, 64))))
    dense5 = wide.contiguous()
    assert torch.equal(mx.checkpoint(wide).codes, mx.checkpoint(dense5).codes)
    kept = mx.checkpoint(torch.from_numpy(r.standard_normal((5, 16))).float().cuda())
    assert torch.equal(mx.weight_grad(kept, wide), mx.weight_grad(kept, dense5))
