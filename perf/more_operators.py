"""Measured cases of the expert layers' operators: products grouped by expert
with ragged sizes, their weight gradient, 4-bit weights with group scales and
the few-row products with them, dense and grouped by expert.

Groups.  Rows of x are sorted by group (expert); ``offsets`` (groups + 1 whole
numbers on the GPU) says that rows offsets[g] .. offsets[g + 1] - 1 are group
g's.  A group may be empty, and rows before the first and behind the last
offset belong to none (a padded batch): their results are zeros.

* product: y[t] = x[t] @ w[g of t], w groups x K x N (or, transposed,
  groups x N x K: the product that gives the input's gradient).
* gradient: dw[g] = x_g.T @ dy_g, groups x K x N.

4-bit weights.  An N x K matrix (outputs x inputs) is held in groups of
``block`` consecutive k: codes q of 0 .. 15, two a byte, the even k in the low
half; a row is filled up to whole 32 k (16 bytes).  A group has a scale s and,
where it has one, a zero point z (a byte; otherwise z = 8): w = s * (q - z).

* With zero points, lo = min(0, group), hi = max(0, group): s = (hi - lo) / 15
  rounded to 32 bits after either operation and then to its type, z = -lo / s
  and q = w / s + z, both ratios rounded to the nearest whole number (ties to
  even) and the results kept within 0 .. 15.
* Without: s = max|group| / 7, rounded the same, q = w / s + 8.

``own`` False runs the operators in elementary torch operations in 32 bits;
``own`` True calls ``dense_gemm_row_amd.grouped`` and ``dense_gemm_row_amd.w4``.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # Decoding one token: the eight experts that its router picked.
        dict(name="experts_token", op="product", rows=8, groups=64, k=2048, n=1024, dtype="bf16", out="bf16",
             transposed=False, pad=0),
        # A short padded prompt through a layer of odd widths, 32-bit results.
        dict(name="experts_ragged", op="product", rows=1531, groups=16, k=1000, n=1337, dtype="f16", out="f32",
             transposed=True, pad=19),
        # A training batch through a few wide experts.
        dict(name="experts_batch", op="product", rows=16384, groups=8, k=4096, n=4096, dtype="bf16", out="bf16",
             transposed=False, pad=0),
        # The input's gradient of many narrow experts.
        dict(name="experts_input_grad", op="product", rows=16384, groups=64, k=1024, n=2048, dtype="bf16", out="bf16",
             transposed=True, pad=0),
        # Weight gradients of a small odd layer, some experts without a token.
        dict(name="gradient_ragged", op="gradient", rows=777, groups=8, k=520, n=263, dtype="f16", out="f16", pad=5),
        # Weight gradients of the training batch, in 32 bits.
        dict(name="gradient_batch", op="gradient", rows=16384, groups=8, k=4096, n=4096, dtype="bf16", out="f32", pad=0),
        # A small odd layer's weights to 4 bits, short groups without zero points, and read back.
        dict(name="weights4_ragged", op="quantize", n=520, k=1000, dtype="f16", scale="f16", transposed=False, block=32,
             zeros=False),
        # A wide layer's K x N weights to 4 bits with zero points, and read back.
        dict(name="weights4_layer", op="quantize", n=11008, k=4096, dtype="bf16", scale="bf16", transposed=True,
             block=128, zeros=True),
        # Decoding: one token through a layer of 4-bit weights.
        dict(name="token4", op="product4", rows=1, n=4096, k=4096, dtype="bf16", block=128, zeros=True),
        # Decoding an odd batch of requests through a wide layer.
        dict(name="batch4", op="product4", rows=33, n=11008, k=4096, dtype="f16", block=64, zeros=False),
        # Decoding one token through eight experts of 4-bit weights.
        dict(name="experts4_token", op="experts4", rows=8, groups=64, n=1024, k=2048, dtype="bf16", block=128, zeros=True,
             pad=0),
        # Decoding a padded batch of requests, short groups.
        dict(name="experts4_batch", op="experts4", rows=512, groups=64, n=2048, k=2048, dtype="bf16", block=32, zeros=True,
             pad=3),
    ]


def _size(rng, low, high):
    """Spread over the logarithm; every third or so moved off the even sizes."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return max(low, min(high, v | 1 if rng.random() < 0.3 else (v + 31) // 32 * 32 if v >= 48 else v))


def draw(rng):
    op = rng.choice(["product", "gradient", "quantize", "product4", "experts4"])
    half = rng.choice(["f16", "bf16", "bf16"])
    if op in ("product", "gradient"):
        dtype = rng.choice([half, half, half, "f32"])
        groups = _size(rng, 1, 64)
        most = 8 * 4096 * 4096 // groups  # (the weights of the largest listed case)
        k = _size(rng, 16, 4096)
        case = dict(op=op, rows=_size(rng, 1, 16384 if dtype != "f32" else 2048), groups=groups, k=k,
                    n=_size(rng, 16, min(4096, most // k)), dtype=dtype, out=rng.choice([dtype, "f32"]),
                    pad=rng.choice([0, 0, 7]))
        if op == "product":
            case["transposed"] = rng.random() < 0.5
        return case
    block, zeros = rng.choice([32, 64, 128, 128]), rng.random() < 0.6
    if op == "quantize":
        dtype = rng.choice([half, half, "f32"])
        return dict(op=op, n=_size(rng, 1, 8192), k=_size(rng, 1, 4096), dtype=dtype,
                    scale=half if dtype == "f32" else dtype, transposed=rng.random() < 0.5, block=block, zeros=zeros)
    if op == "product4":
        return dict(op=op, rows=_size(rng, 1, 512), n=_size(rng, 16, 11008), k=_size(rng, 16, 8192), dtype=half,
                    block=block, zeros=zeros)
    return dict(op=op, rows=_size(rng, 1, 1024), groups=_size(rng, 1, 64), n=_size(rng, 16, 2048), k=_size(rng, 16, 2048),
                dtype=half, block=block, zeros=zeros, pad=rng.choice([0, 0, 7]))


def _coded_bytes(case):
    groups = -(-case["k"] // case["block"])
    size = BYTES[case.get("scale", case["dtype"])] + (1 if case["zeros"] else 0)
    return case["n"] * (-(-case["k"] // 32) * 16 + groups * size)


def work(case):
    k, n, size = case["k"], case["n"], BYTES[case["dtype"]]
    if case["op"] == "quantize":  # the values, their codes, and the values they stand for
        return {"bytes": 2 * n * k * size + _coded_bytes(case), "flops": 4 * n * k}
    rows = case["rows"]
    if case["op"] == "product4":
        return {"bytes": rows * (k + n) * size + _coded_bytes(case), "flops": 2 * rows * n * k}
    used = min(rows, case["groups"])  # groups that can have a row
    if case["op"] == "experts4":
        return {"bytes": (rows + case["pad"]) * (k + n) * size + used * _coded_bytes(case), "flops": 2 * rows * n * k}
    out = BYTES[case["out"]]
    if case["op"] == "product":
        moved = rows * k * size + used * k * n * size + (rows + case["pad"]) * n * out
    else:
        moved = rows * (k + n) * size + case["groups"] * k * n * out
    return {"bytes": moved, "flops": 2 * rows * n * k}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bounds(g, rows, groups):
    """The router's offsets on the host: popular and unpopular experts, so
    that some have many rows and some none."""
    liking = torch.softmax(torch.randn(groups, generator=g, device="cuda"), dim=0)
    pick = torch.multinomial(liking, rows, replacement=True, generator=g)
    counts = torch.bincount(pick, minlength=groups)
    return [0] + torch.cumsum(counts, dim=0).tolist()


def _activations(g, rows, cols, dtype):
    """Hidden states: near normal, rows of different size, a few outlier channels."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    x *= torch.where(torch.rand(1, cols, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return x.to(DTYPES[dtype])


def _weights(g, shape, k, dtype):
    w = torch.empty(shape, dtype=DTYPES[dtype], device="cuda")
    for part in w if w.dim() == 3 else [w]:
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") / math.sqrt(k))
    return w


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    k, n = case["k"], case["n"]
    if case["op"] == "quantize":
        s["w"] = _weights(g, (k, n) if case["transposed"] else (n, k), k, case["dtype"])
        return s
    rows = case["rows"]
    total = rows + case.get("pad", 0)
    s["x"] = _activations(g, total, k, case["dtype"])
    if case["op"] == "product4":
        s["coded"] = _encode(_weights(g, (n, k), k, "f32"), case["block"], case["zeros"], DTYPES[case["dtype"]])
        return s
    s["bounds"] = _bounds(g, rows, case["groups"])
    s["offsets"] = torch.tensor(s["bounds"], dtype=torch.int32, device="cuda")
    if case["op"] == "experts4":
        w = _weights(g, (case["groups"] * n, k), k, "f32")
        coded = _encode(w, case["block"], case["zeros"], DTYPES[case["dtype"]])
        s["coded"] = tuple(t if t is None else t.view(case["groups"], n, -1) for t in coded)
    elif case["op"] == "product":
        shape = (case["groups"], n, k) if case["transposed"] else (case["groups"], k, n)
        s["w"] = _weights(g, shape, k, case["dtype"])
    else:
        dy = 1e-2 * torch.randn(total, n, generator=g, device="cuda")
        dy *= (torch.rand(total, 1, generator=g, device="cuda") > 0.1).float()  # masked tokens
        s["dy"] = dy.to(DTYPES[case["dtype"]])
    return s


def _encode(w, block, zeros, scale_dtype):
    """(codes, scales, zero points or None) of an N x K matrix, packed."""
    q, s, z = _to_codes(w, block, zeros, scale_dtype)
    rows, k = w.shape
    codes = torch.zeros(rows, -(-k // 32) * 32, dtype=torch.uint8, device=w.device)
    codes[:, :k] = q.view(rows, -1)[:, :k].to(torch.uint8)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), s, z.to(torch.uint8) if zeros else None


# ---------------------------------------------------------------------------
# The plain form: elementary operations in 32 bits (the ratios that decide a
# code in 64, where a quotient in 32 could fall on a border that it is next to)
# ---------------------------------------------------------------------------
def _to_codes(w, block, zeros, scale_dtype):
    """Codes (rows x groups x block), scales and zero points (rows x groups)."""
    rows, k = w.shape
    groups = -(-k // block)
    v = torch.zeros(rows, groups * block, dtype=torch.float32, device=w.device)
    v[:, :k] = w
    v = v.view(rows, groups, block)
    if zeros:
        lo, hi = v.amin(dim=2).clamp(max=0), v.amax(dim=2).clamp(min=0)
        s = ((hi - lo).double() / 15).float().to(scale_dtype)
    else:
        s = (v.abs().amax(dim=2).double() / 7).float().to(scale_dtype)
    by = torch.where(s > 0, s.double(), 1.0)
    if zeros:
        z = torch.where(s > 0, torch.round(-lo.double() / by).clamp(0, 15), 0.0)
    else:
        z = torch.full_like(by, 8.0)
    q = torch.round(v.double() / by[:, :, None]) + z[:, :, None]
    q = torch.where(s[:, :, None] > 0, q.clamp(0, 15), z[:, :, None])
    return q.to(torch.int32), s, z.to(torch.int32)


def _decode(coded, block, k):
    """The values of packed codes, in 32 bits."""
    codes, s, z = coded
    q = torch.stack((codes & 15, codes >> 4), dim=2).view(codes.shape[0], -1)[:, :k].float()
    zero = torch.full_like(s, 8, dtype=torch.float32) if z is None else z.float()
    return (q - zero.repeat_interleave(block, dim=1)[:, :k]) * s.float().repeat_interleave(block, dim=1)[:, :k]


def _plain(s):
    k = s["k"]
    if s["op"] == "quantize":
        w = s["w"].t() if s["transposed"] else s["w"]
        q, scale, z = _to_codes(w, s["block"], s["zeros"], DTYPES[s["scale"]])
        value = (q - z[:, :, None]).float() * scale.float()[:, :, None]
        return value.view(w.shape[0], -1)[:, :k].to(s["w"].dtype)
    if s["op"] == "product4":
        return (s["x"].float() @ _decode(s["coded"], s["block"], k).t()).to(s["x"].dtype)
    out = DTYPES[s.get("out", s["dtype"])]
    x, bounds = s["x"], s["bounds"]
    if s["op"] == "gradient":
        y = torch.zeros(s["groups"], k, s["n"], dtype=out, device=x.device)
    else:
        y = torch.zeros(x.shape[0], s["n"], dtype=out, device=x.device)
    for g in range(s["groups"]):
        a, b = bounds[g], bounds[g + 1]
        if a == b:
            continue
        if s["op"] == "gradient":
            y[g] = x[a:b].float().t() @ s["dy"][a:b].float()
        elif s["op"] == "experts4":
            w = _decode(tuple(t if t is None else t[g] for t in s["coded"]), s["block"], k)
            y[a:b] = x[a:b].float() @ w.t()
        else:
            w = s["w"][g].float()
            y[a:b] = x[a:b].float() @ (w.t() if s["transposed"] else w)
    return y


# ---------------------------------------------------------------------------
# The framework's operators
# ---------------------------------------------------------------------------
def _framework(s):
    from dense_gemm_row_amd import grouped, w4
    if s["op"] == "quantize":
        q = w4.quantize(s["w"], group=s["block"], zeros=s["zeros"], transposed=s["transposed"],
                        scale_dtype=DTYPES[s["scale"]])
        return w4.dequantize(q, dtype=s["w"].dtype)
    if s["op"] == "product4":
        return w4.matmul(s["x"], w4.W4Tensor(*s["coded"], cols=s["k"], group=s["block"]))
    if s["op"] == "experts4":
        return w4.grouped_matmul(s["x"], w4.W4Tensor(*s["coded"], cols=s["k"], group=s["block"]), s["offsets"])
    if s["op"] == "product":
        return grouped.matmul(s["x"], s["w"], s["offsets"], transposed=s["transposed"], out_dtype=DTYPES[s["out"]])
    return grouped.weight_grad(s["x"], s["dy"], s["offsets"], out_dtype=DTYPES[s["out"]])


def run(state):
    return _framework(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def _nearest(a, s):
    """The whole number nearest to a / s (s > 0), ties to even, found from
    exact products: floor first, then which half of the step a is in."""
    low = torch.floor(a / s)
    low = low - (low * s > a).double() + ((low + 1) * s <= a).double()
    middle = (low + 0.5) * s
    odd = torch.remainder(low, 2)
    return low + (a > middle).double() + (a == middle).double() * odd


def _exact_weights(w, block, zeros, scale_dtype):
    """The values that w's 4-bit codes stand for, one group after another."""
    values = torch.empty(w.shape, dtype=torch.float64, device=w.device)
    for begin in range(0, w.shape[1], block):
        part = w[:, begin:begin + block].double()
        low = torch.minimum(part.min(dim=1, keepdim=True).values, torch.zeros((), dtype=torch.float64, device=w.device))
        high = torch.maximum(part.max(dim=1, keepdim=True).values, torch.zeros((), dtype=torch.float64, device=w.device))
        span = (high - low).float().double() / 15 if zeros else torch.maximum(high, -low) / 7
        scale = span.float().to(scale_dtype).double()
        step = torch.where(scale > 0, scale, torch.ones_like(scale))
        zero = _nearest(-low, step).clamp(0, 15) if zeros else torch.full_like(step, 8.0)
        code = (_nearest(part, step) + zero).clamp(0, 15)
        values[:, begin:begin + block] = torch.where(scale > 0, scale * (code - zero), torch.zeros_like(code))
    return values


def _exact_decode(coded, block, k):
    codes, scales, zero_points = coded
    column = torch.arange(k, device=codes.device)
    q = (codes[:, column // 2].to(torch.int64) >> (4 * (column % 2))) % 16
    z = 8 if zero_points is None else zero_points[:, column // block].to(torch.int64)
    return scales[:, column // block].double() * (q - z).double()


def exact(case, seed):
    s = prepare(case, seed)
    k, n = case["k"], case["n"]
    if case["op"] == "quantize":
        return _exact_weights(s["w"].t() if case["transposed"] else s["w"], case["block"], case["zeros"],
                              DTYPES[case["scale"]])
    x = s["x"].double()
    if case["op"] == "product4":
        return torch.mm(x, _exact_decode(s["coded"], case["block"], k).t())
    shape = (case["groups"], k, n) if case["op"] == "gradient" else (x.shape[0], n)
    result = torch.zeros(shape, dtype=torch.float64, device=x.device)
    edge = s["offsets"].tolist()
    for g, (a, b) in enumerate(zip(edge[:-1], edge[1:])):
        if case["op"] == "gradient":
            result[g] = torch.mm(x[a:b].t(), s["dy"][a:b].double())
        elif case["op"] == "experts4":
            one = [None if t is None else t[g] for t in s["coded"]]
            result[a:b] = torch.mm(x[a:b], _exact_decode(one, case["block"], k).t())
        else:
            w = s["w"][g].double()
            result[a:b] = torch.mm(x[a:b], w.t() if case["transposed"] else w)
    return result
