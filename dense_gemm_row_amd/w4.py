"""Integer 4-bit weights with a scale (and zero point) for every group of
inputs: binding of include/gemm_w4.h and its torch forms.

The functions with the C names only marshal arguments.  The torch forms
(`quantize`, `dequantize`, `matmul`, `grouped_matmul`) take GPU tensors,
allocate results and workspaces with torch on the launch stream, and run the
HIP kernels of ``libgemm.so``; there is no fallback.

A decoding step through a layer, and through a layer of experts, in these
terms (w is K x N, we experts x K x N)::

    wq = w4.quantize(w, transposed=True)         # once
    y = w4.matmul(x, wq)
    weq = w4.quantize(we, transposed=True)
    y = w4.grouped_matmul(x, weq, offsets)       # rows of x sorted by expert
"""
from __future__ import annotations

import ctypes

from . import gemm, grouped, mx

GROUPS = (32, 64, 128)  # values per scale
ROWS = 128              # GEMM_W4_ROWS
EXPORTS = ["gemm_w4_quantize", "gemm_w4_dequantize", "gemm_w4_matmul", "gemm_w4_matmul_workspace_bytes", "gemm_w4_grouped",
           "gemm_w4_grouped_workspace_bytes"]

_declared = None


class GemmW4(ctypes.Structure):
    """gemm_w4_t: a coded weight operand."""
    _fields_ = [("codes", ctypes.c_void_p), ("ldq", ctypes.c_int64), ("stride_q", ctypes.c_int64),
                ("scales", ctypes.c_void_p), ("lds", ctypes.c_int64), ("stride_s", ctypes.c_int64),
                ("zeros", ctypes.c_void_p), ("ldz", ctypes.c_int64), ("stride_z", ctypes.c_int64), ("group", ctypes.c_int32)]


def lib():
    """The loaded libgemm with the signatures of gemm_w4.h."""
    global _declared
    if _declared is None:
        L = gemm.lib()
        i64, i32, p, q = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.POINTER(GemmW4)
        L.gemm_w4_quantize.argtypes = [i32, i32, i32, i64, i64, p, i64, q, p]
        L.gemm_w4_dequantize.argtypes = [i32, i32, i64, i64, q, p, i64, p]
        L.gemm_w4_matmul.argtypes = [i32, i64, i64, i64, p, i64, q, p, i64, p, i64, p]
        L.gemm_w4_matmul_workspace_bytes.argtypes = [i64, i64, i64]
        L.gemm_w4_grouped.argtypes = [i32, i64, i64, i64, i64, p, p, i64, q, p, i64, i32, p, i64, p]
        L.gemm_w4_grouped_workspace_bytes.argtypes = [i64, i64, i64, i64]
        for name in EXPORTS:
            getattr(L, name).restype = i64 if name.endswith("_bytes") else ctypes.c_int
        _declared = L
    return _declared


def gemm_w4_quantize(dtype, s_dtype, trans, N, K, X, ldx, q: GemmW4, stream=None) -> int:
    return lib().gemm_w4_quantize(dtype, s_dtype, trans, N, K, X, ldx, gemm._ref(q), stream)


def gemm_w4_dequantize(dtype, s_dtype, N, K, q: GemmW4, X, ldx, stream=None) -> int:
    return lib().gemm_w4_dequantize(dtype, s_dtype, N, K, gemm._ref(q), X, ldx, stream)


def gemm_w4_matmul(dtype, M, N, K, X, ldx, q: GemmW4, Y, ldy, workspace=None, workspace_bytes=0, stream=None) -> int:
    return lib().gemm_w4_matmul(dtype, M, N, K, X, ldx, gemm._ref(q), Y, ldy, workspace, workspace_bytes, stream)


def gemm_w4_matmul_workspace_bytes(M, N, K) -> int:
    return lib().gemm_w4_matmul_workspace_bytes(M, N, K)


def gemm_w4_grouped(dtype, G, T, N, K, offsets, X, ldx, q: GemmW4, Y, ldy, fill=0, workspace=None, workspace_bytes=0,
                    stream=None) -> int:
    return lib().gemm_w4_grouped(dtype, G, T, N, K, offsets, X, ldx, gemm._ref(q), Y, ldy, fill, workspace, workspace_bytes,
                                 stream)


def gemm_w4_grouped_workspace_bytes(G, T, N, K) -> int:
    return lib().gemm_w4_grouped_workspace_bytes(G, T, N, K)


# --------------------------------------------------------------------------
# Torch forms (see mx.py for the launch stream and allocations).
# --------------------------------------------------------------------------
class W4Tensor:
    """4-bit weights (the format of include/gemm_w4.h): ``codes`` (uint8, N x
    16 bytes for every 32 of K), ``scales`` (float16 or bfloat16, N x groups)
    and ``zeros`` (uint8, N x groups; None: every zero point is 8) of ``cols``
    = K values a row, ``group`` (32, 64 or 128) of them to a scale.  With a
    leading dimension more they are a stack of matrices, one an expert.  All
    may be views with larger strides, rows contiguous; codes need 16-byte
    alignment and strides of multiples of 16.  (Products of few rows are
    fastest where K is whole 256 k and rows of x, scales and zero points begin
    aligned to 16 bytes and to 256 k's; with an odd K, or rows of x that begin
    on 2 bytes, some take three times as long: see include/gemm_w4.h.)"""
    __slots__ = ("codes", "scales", "zeros", "cols", "group")

    def __init__(self, codes, scales, zeros, cols: int, group: int = 128):
        if group not in GROUPS:
            raise ValueError(f"groups of {group}: 32, 64 or 128")
        if mx._torch is None:
            mx._load()
        torch = mx._torch
        cs, width, count = codes.shape, -(-cols // 32) * 16, -(-cols // group)
        if len(cs) not in (2, 3) or codes.dtype is not torch.uint8 or cs[-1] != width:
            raise ValueError(f"codes must be uint8 with rows of {width} bytes for {cols} columns")
        if scales.dtype not in (torch.float16, torch.bfloat16):
            raise TypeError("scales must be float16 or bfloat16")
        shape = (*cs[:-1], count)
        if scales.shape != shape:
            raise ValueError(f"scales must have shape {shape}, not {tuple(scales.shape)}")
        if (width > 1 and codes.stride(-1) != 1) or (count > 1 and scales.stride(-1) != 1):
            raise ValueError("rows must be contiguous (unit column stride)")
        at = codes.get_device()
        if scales.get_device() != at:
            raise ValueError("codes and scales are on different devices")
        if zeros is not None:
            if zeros.dtype is not torch.uint8:
                raise TypeError("zeros must be uint8")
            if zeros.shape != shape:
                raise ValueError(f"zeros must have shape {shape}, not {tuple(zeros.shape)}")
            if count > 1 and zeros.stride(-1) != 1:
                raise ValueError("rows must be contiguous (unit column stride)")
            if zeros.get_device() != at:
                raise ValueError("codes and zeros are on different devices")
        self.codes, self.scales, self.zeros, self.cols, self.group = codes, scales, zeros, cols, group

    @property
    def shape(self):
        """(N, K), or (experts, N, K)."""
        return (*self.codes.shape[:-1], self.cols)

    @property
    def device(self):
        return self.codes.device

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.codes, self.scales, self.zeros) if t is not None)

    def __getitem__(self, expert: int) -> "W4Tensor":
        """One matrix of a stack."""
        if self.codes.dim() != 3:
            raise TypeError("not a stack of matrices")
        return W4Tensor(self.codes[expert], self.scales[expert], None if self.zeros is None else self.zeros[expert],
                        self.cols, self.group)

    def _desc(self):
        """The C-ABI's description of these tensors."""
        c, s, z = self.codes, self.scales, self.zeros
        cs, width, cd, sd = c.shape, s.shape[-1], c.stride(), s.stride()
        # (A single row's or matrix's stride means nothing.)
        rows, apart = cs[-2] > 1, len(cs) == 3 and cs[0] > 1
        if z is None:
            zp, zl, za = None, 0, 0
        else:
            zd = z.stride()
            zp, zl, za = z.data_ptr(), zd[-2] if rows else width, zd[0] if apart else 0
        return GemmW4(c.data_ptr(), cd[-2] if rows else cs[-1], cd[0] if apart else 0,
                      s.data_ptr(), sd[-2] if rows else width, sd[0] if apart else 0, zp, zl, za, self.group)

    def __repr__(self) -> str:
        return f"W4Tensor({' x '.join(map(str, self.shape))}, groups of {self.group}, {self.device})"


def _coded(q, name, dims):
    if not isinstance(q, W4Tensor):
        raise TypeError(f"{name} must be a W4Tensor")
    if not q.codes.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if q.codes.dim() != dims:
        raise ValueError(f"{name} must be " + ("one matrix (N x K)" if dims == 2 else "a stack of matrices (experts x N x K)"))


def _apart(t, name):
    """Refuses a stack of results two of which share memory (an expanded one)."""
    groups, rows, cols = t.shape
    (near, n), (far, m) = sorted(((t.stride(0), groups), (t.stride(1), rows)))
    if t.numel() > 0 and ((n > 1 and near < cols) or (m > 1 and far < (n - 1) * near + cols)):
        raise ValueError(f"{name}: results of two experts or rows overlap")


def empty(shape, group: int, device, scale_dtype=None, zeros: bool = True) -> W4Tensor:
    """Uninitialised 4-bit weights of shape (N, K) or (experts, N, K), scale
    rows of whole 256 k."""
    if mx._torch is None:
        mx._load()
    torch = mx._torch
    if group not in GROUPS:
        raise ValueError(f"groups of {group}: 32, 64 or 128")
    lead, K = tuple(shape[:-1]), shape[-1]
    count = -(-K // group)
    wide = -(-K // 256) * (256 // group)

    def whole(n, dtype):
        if len(lead) == 1:  # (`empty` takes 0.4 us longer to read its arguments)
            return torch.empty_strided((lead[0], n), (max(n, 1), 1), dtype=dtype, device=device)
        return torch.empty((*lead, n), dtype=dtype, device=device)

    def rows(n, dtype):
        t = whole(n, dtype)
        return t if n == count else t[..., :count]
    q = W4Tensor.__new__(W4Tensor)  # (as the checks of __init__ would have it)
    q.codes = whole(-(-K // 32) * 16, torch.uint8)
    q.scales = rows(wide, scale_dtype or torch.bfloat16)
    q.zeros = rows(wide, torch.uint8) if zeros else None
    q.cols, q.group = K, group
    return q


def quantize(w, group: int = 128, zeros: bool = True, transposed: bool = False, scale_dtype=None, out: W4Tensor | None = None,
             stream=None) -> W4Tensor:
    """The 4-bit form of w: N x K (outputs x inputs), or with ``transposed`` K
    x N as the other products take weights; a leading dimension more is a
    stack of experts.  Scales are of ``scale_dtype`` (default: w's type,
    bfloat16 for float32): the type of the activations to come.  zeros False:
    no zero points.  An ``out`` is written in its own group, scale type and
    zero points."""
    stack = w.dim() == 3
    first = w[0] if stack and w.shape[0] > 0 else w
    if stack and w.shape[0] == 0:
        raise ValueError("an empty stack")
    dtype, rows, cols, ldx = mx._dense(first, "w")
    torch = mx._torch
    N, K = (cols, rows) if transposed else (rows, cols)
    shape = (w.shape[0], N, K) if stack else (N, K)
    given = out is not None
    if not given:
        kind = scale_dtype or (torch.bfloat16 if w.dtype == torch.float32 else w.dtype)
        if kind not in (torch.float16, torch.bfloat16):
            raise TypeError("scale_dtype must be float16 or bfloat16")
        on = mx._Launch(first, stream)
        if on.other:
            with torch.cuda.stream(torch.cuda.ExternalStream(on.handle, device=w.device)):
                out = empty(shape, group, w.device, kind, zeros)
        else:
            out = empty(shape, group, w.device, kind, zeros)
    else:
        _coded(out, "out", len(shape))
        mx._same_device(w, out)
        if out.shape != shape:
            raise ValueError(f"out has shape {out.shape}, not {shape}")
        if stack:
            for part in (out.codes, out.scales, out.zeros):
                if part is not None:
                    _apart(part, "out")
        on = mx._Launch(first, stream)
    for e in range(shape[0] if stack else 1):
        m, q = (w[e], out[e]) if stack else (w, out)
        grouped._call(lib(), "gemm_w4_quantize", w.get_device(), dtype, mx._DTYPES[q.scales.dtype], 1 if transposed else 0, N, K,
                      m.data_ptr(), ldx, ctypes.byref(q._desc()), on.handle)
    if given:
        grouped._written(*(t for t in (out.codes, out.scales, out.zeros) if t is not None))
    return out


def dequantize(q: W4Tensor, dtype=None, out=None, stream=None):
    """The values of 4-bit weights as a tensor of q's shape, of ``dtype``
    (default: the scales' type)."""
    _coded(q, "q", 3 if isinstance(q, W4Tensor) and q.codes.dim() == 3 else 2)
    torch = mx._torch
    stack = q.codes.dim() == 3
    on = mx._Launch(q.codes, stream)
    given = out is not None
    if not given:
        out = on.empty(q.shape, mx._out_dtype(dtype, q.scales.dtype, "dtype"))
    elif tuple(out.shape) != q.shape or (dtype is not None and out.dtype != dtype):
        raise ValueError("out has the wrong shape or dtype")
    if not isinstance(out, torch.Tensor) or not out.is_cuda:
        raise ValueError("out must be a GPU tensor")
    mx._same_device(q, out)
    if stack and given:
        _apart(out, "out")
    for e in range(q.shape[0] if stack else 1):
        one, x = (q[e], out[e]) if stack else (q, out)
        x_dtype, N, K, ldx = mx._dense(x, "out")
        grouped._call(lib(), "gemm_w4_dequantize", q.codes.get_device(), x_dtype, mx._DTYPES[q.scales.dtype], N, K,
                      ctypes.byref(one._desc()), x.data_ptr(), ldx, on.handle)
    if given:
        grouped._written(out)
    return out


def _operands(name, x, q, dims, out, stream):
    """The checks that both products share: (library dtype, rows, K, ldx, N,
    launch, out, ldy)."""
    if isinstance(q, W4Tensor) and (x.requires_grad or q.scales.requires_grad):
        grouped._no_graph(name, "")
    _coded(q, "q", dims)
    dtype, rows, K, ldx = mx._dense(x, "x")
    if x.dtype != q.scales.dtype:
        raise TypeError(f"x must have the scales' type, {q.scales.dtype}")
    mx._same_device(x, q)
    if q.cols != K:
        raise ValueError(f"inner dimensions differ: {K} vs {q.cols}")
    N = q.codes.shape[-2]
    on = mx._Launch(x, stream)
    if out is None:
        out = on.empty((rows, N), x.dtype)
        return dtype, rows, K, ldx, N, on, out, max(N, 1)
    if tuple(out.shape) != (rows, N) or out.dtype != x.dtype:
        raise ValueError("out has the wrong shape or dtype")
    _, _, _, ldy = mx._dense(out, "out")
    mx._same_device(out, x)
    return dtype, rows, K, ldx, N, on, out, ldy


def matmul(x, q: W4Tensor, out=None, stream=None):
    """x @ w.T for 4-bit weights q (N x K) and x (M x K) of the scales' type,
    which is the result's.  Up to 128 rows the codes are multiplied as they
    are; more rows multiply dequantised weights, rounded to that type (results
    are off by about a third more), through a workspace of 2 N K bytes.  (For serving: no graph is recorded, and the
    call is refused where one would be, as by ``grouped.matmul``.)"""
    given = out is not None
    dtype, M, K, ldx, N, on, out, ldy = _operands("w4.matmul", x, q, 2, out, stream)
    need = 0 if M <= ROWS else lib().gemm_w4_matmul_workspace_bytes(M, N, K)
    ws = on.empty(need, mx._torch.uint8) if need > 0 else None
    grouped._call(lib(), "gemm_w4_matmul", x.get_device(), dtype, M, N, K, x.data_ptr(), ldx, ctypes.byref(q._desc()),
                  out.data_ptr(), ldy, ws.data_ptr() if ws is not None else None, max(need, 0), on.handle)
    if given:
        grouped._written(out)
    return out


def grouped_matmul(x, q: W4Tensor, offsets, out=None, stream=None):
    """y[t] = x[t] @ w[g].T for the rows t of every group g, rows offsets[g] to
    offsets[g + 1] - 1 of x (T x K), and a stack q of 4-bit weights (experts x
    N x K).  Rows of no group are zero in a new result; in ``out`` they stay as
    they are.  (Above 128 rows an expert on average all experts' weights are
    dequantised first, rounded to that type as in `matmul`.  For serving: no graph is recorded, and the call is
    refused where one would be, as by ``grouped.matmul``.)"""
    fill = out is None
    dtype, T, K, ldx, N, on, out, ldy = _operands("w4.grouped_matmul", x, q, 3, out, stream)
    G = q.codes.shape[0]
    at = grouped._offsets(offsets, G, x)
    need = 0 if T <= ROWS * G else lib().gemm_w4_grouped_workspace_bytes(G, T, N, K)
    ws = on.empty(need, mx._torch.uint8) if need > 0 else None
    grouped._call(lib(), "gemm_w4_grouped", x.get_device(), dtype, G, T, N, K, at, x.data_ptr(), ldx, ctypes.byref(q._desc()),
                  out.data_ptr(), ldy, 1 if fill else 0, ws.data_ptr() if ws is not None else None, max(need, 0), on.handle)
    if not fill:
        grouped._written(out)
    return out
