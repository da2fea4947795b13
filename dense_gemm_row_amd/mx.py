"""Microscaled operands: binding of include/gemm_mx.h and its torch forms.

The functions with the C names only marshal arguments.  The torch forms
(`quantize`, `dequantize`, `matmul`, `checkpoint`, `restore`, `weight_grad`)
take GPU tensors, allocate outputs and workspaces with torch on the launch
stream, and run the HIP kernels of ``libgemm.so``; there is no fallback.

A linear layer y = x W in these terms (W is K x N, row-major)::

    wq = mx.quantize(w, mx.E2M1, transposed=True)   # once per weight update
    y = mx.matmul(x, wq)                            # x is quantised on the way
    kept = mx.checkpoint(x)                         # 8 bits, for the backward pass
    dx = gemm.matmul(dy, w, b_transposed=True)
    dw = mx.weight_grad(kept, dy)

`linear` is that layer as a torch autograd function.
"""
from __future__ import annotations

import ctypes

from . import gemm

E2M1 = "e2m1"  # 4-bit elements
E4M3 = "e4m3"  # 8-bit elements
BLOCK = 32     # values per scale

FORMATS = {E2M1: 0, E4M3: 1}
BLOCK_BYTES = {E2M1: 16, E4M3: 32}
EXPORTS = ["gemm_mx_quantize", "gemm_mx_dequantize", "gemm_mx_matmul", "gemm_mx_matmul_values",
           "gemm_mx_matmul_values_workspace_bytes", "gemm_mx_wgrad", "gemm_mx_wgrad_workspace_bytes"]

_declared = None


def lib():
    """The loaded libgemm with the signatures of gemm_mx.h."""
    global _declared
    if _declared is None:
        L = gemm.lib()
        i64, i32, p, f = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float
        L.gemm_mx_quantize.argtypes = [i32, i32, i32, i64, i64, p, i64, p, i64, p, i64, p]
        L.gemm_mx_dequantize.argtypes = [i32, i32, i32, i64, i64, p, i64, p, i64, p, i64, p]
        L.gemm_mx_matmul.argtypes = [i32, i64, i64, i64, p, i64, p, i64, p, i64, p, i64, p, i64, p,
                                     ctypes.POINTER(gemm.GemmEpilogue)]
        L.gemm_mx_wgrad.argtypes = [i32, i32, i64, i64, i64, p, i64, p, i64, p, i64, p, i64, f, f,
                                    p, i64, p]
        L.gemm_mx_matmul_values.argtypes = [i32, i32, i64, i64, i64, p, i64, p, i64, p, i64, p, i64, p, i64, p,
                                            ctypes.POINTER(gemm.GemmEpilogue)]
        L.gemm_mx_matmul_values_workspace_bytes.argtypes = [i64, i64]
        L.gemm_mx_matmul_values_workspace_bytes.restype = i64
        for name in ("gemm_mx_quantize", "gemm_mx_dequantize", "gemm_mx_matmul", "gemm_mx_matmul_values",
                     "gemm_mx_wgrad"):
            getattr(L, name).restype = ctypes.c_int
        L.gemm_mx_wgrad_workspace_bytes.argtypes = [i32, i64, i64, i64]
        L.gemm_mx_wgrad_workspace_bytes.restype = i64
        _declared = L
    return _declared


def gemm_mx_quantize(dtype, fmt, trans, rows, cols, X, ldx, codes, ldq, scales, lds, stream=None) -> int:
    return lib().gemm_mx_quantize(dtype, fmt, trans, rows, cols, X, ldx, codes, ldq, scales, lds, stream)


def gemm_mx_dequantize(dtype, fmt, trans, rows, cols, codes, ldq, scales, lds, X, ldx, stream=None) -> int:
    return lib().gemm_mx_dequantize(dtype, fmt, trans, rows, cols, codes, ldq, scales, lds, X, ldx, stream)


def gemm_mx_matmul(c_dtype, M, N, K, A, lda, As, ldas, Bt, ldbt, Bs, ldbs, C, ldc, stream=None,
                   epi: gemm.GemmEpilogue | None = None) -> int:
    return lib().gemm_mx_matmul(c_dtype, M, N, K, A, lda, As, ldas, Bt, ldbt, Bs, ldbs, C, ldc, stream,
                                ctypes.byref(epi) if epi is not None else None)


def gemm_mx_matmul_values(a_dtype, c_dtype, M, N, K, X, ldx, Bt, ldbt, Bs, ldbs, C, ldc, workspace=None,
                          workspace_bytes=0, stream=None, epi: gemm.GemmEpilogue | None = None) -> int:
    return lib().gemm_mx_matmul_values(a_dtype, c_dtype, M, N, K, X, ldx, Bt, ldbt, Bs, ldbs, C, ldc, workspace,
                                       workspace_bytes, stream, ctypes.byref(epi) if epi is not None else None)


def gemm_mx_matmul_values_workspace_bytes(M, K) -> int:
    return lib().gemm_mx_matmul_values_workspace_bytes(M, K)


def gemm_mx_wgrad(y_dtype, c_dtype, T, F, N, codes, ldq, scales, lds, dY, ldy, dW, ldw, alpha=1.0, beta=0.0,
                  workspace=None, workspace_bytes=0, stream=None) -> int:
    return lib().gemm_mx_wgrad(y_dtype, c_dtype, T, F, N, codes, ldq, scales, lds, dY, ldy, dW, ldw,
                               alpha, beta, workspace, workspace_bytes, stream)


def gemm_mx_wgrad_workspace_bytes(y_dtype, T, F, N) -> int:
    return lib().gemm_mx_wgrad_workspace_bytes(y_dtype, T, F, N)


# --------------------------------------------------------------------------
# Torch forms.  A small call takes about as long as the host needs to make it,
# so these look at every tensor once and ask torch for little: the current
# stream's handle without a Stream object, one allocation a result.
# --------------------------------------------------------------------------
_FAR = 1 << 26  # strides from here on, in bytes, take the workspace in gemm_mx_matmul_values
_torch = None
_DTYPES = {}       # torch dtype -> library dtype
_raw_stream = None  # device index -> handle of torch's current stream


def _load():
    global _torch, _raw_stream
    import torch
    _DTYPES.update({torch.float32: gemm.DTYPE_F32, torch.float16: gemm.DTYPE_F16,
                    torch.bfloat16: gemm.DTYPE_BF16})
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    _torch = torch


class MxTensor:
    """A coded matrix (the format of include/gemm_mx.h): ``codes`` (uint8,
    rows x 16 or 32 bytes a block) and ``scales`` (uint8, rows x blocks), for
    ``cols`` values a row.  Both may be views with a larger row stride; codes
    need 16-byte alignment and a row stride of a multiple of 16.  Products are
    several times faster where the scales' row stride is a multiple of 4 bytes
    too (`empty` and `quantize` make it so; a contiguous copy may not be)."""
    __slots__ = ("codes", "scales", "cols", "fmt")

    def __init__(self, codes, scales, cols: int, fmt: str = E2M1):
        if fmt not in FORMATS:
            raise ValueError(f"unknown format {fmt!r}: {E2M1!r} or {E4M3!r}")
        blocks = -(-cols // BLOCK)
        cs, ss = codes.shape, scales.shape
        if len(cs) != 2 or len(ss) != 2 or codes.element_size() != 1 or scales.element_size() != 1:
            raise ValueError("codes and scales must be 2-D tensors of bytes")
        if cs[0] != ss[0]:
            raise ValueError("codes and scales differ in rows")
        if cs[1] != blocks * BLOCK_BYTES[fmt] or ss[1] != blocks:
            raise ValueError(f"{cols} columns need {blocks * BLOCK_BYTES[fmt]} code bytes and {blocks} scales a row")
        if (cs[1] > 1 and codes.stride(1) != 1) or (blocks > 1 and scales.stride(1) != 1):
            raise ValueError("rows must be contiguous (unit column stride)")
        if codes.device != scales.device:
            raise ValueError("codes and scales are on different devices")
        self.codes, self.scales, self.cols, self.fmt = codes, scales, cols, fmt

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    @property
    def shape(self) -> tuple[int, int]:
        return self.codes.shape[0], self.cols

    @property
    def device(self):
        return self.codes.device

    def nbytes(self) -> int:
        return self.codes.shape[0] * (self.codes.shape[1] + self.scales.shape[1])

    def _args(self):
        c, s = self.codes, self.scales
        rows, width = c.shape
        if rows > 1:
            return c.data_ptr(), c.stride(0), s.data_ptr(), s.stride(0)
        # A single row's stride means nothing: its length, in whole words.
        return c.data_ptr(), -(-width // 16) * 16, s.data_ptr(), -(-s.shape[1] // 4) * 4

    def __repr__(self) -> str:
        return f"MxTensor({self.rows} x {self.cols}, {self.fmt}, {self.device})"


class _Launch:
    """The launch stream of a call on `index`, and allocations on it, so that
    torch's allocator orders their reuse after the kernels (the current stream
    is left as it is)."""
    __slots__ = ("handle", "other", "device")

    def __init__(self, t, stream):
        if _torch is None:
            _load()
        self.device = t.device
        current = _raw_stream(t.get_device())
        if stream is None:
            self.handle, self.other = current, False
        else:
            self.handle = stream.cuda_stream if isinstance(stream, _torch.cuda.Stream) else int(stream)
            self.other = self.handle != current

    def empty(self, shape, dtype):
        if not self.other:
            return _torch.empty(shape, dtype=dtype, device=self.device)
        with _torch.cuda.stream(_torch.cuda.ExternalStream(self.handle, device=self.device)):
            return _torch.empty(shape, dtype=dtype, device=self.device)

    def coded(self, rows, cols, fmt):
        if not self.other:
            return empty(rows, cols, fmt, self.device)
        with _torch.cuda.stream(_torch.cuda.ExternalStream(self.handle, device=self.device)):
            return empty(rows, cols, fmt, self.device)


def _dense(t, name):
    """(library dtype, rows, columns, leading dimension) of a GPU matrix."""
    if _torch is None:
        _load()
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D tensor")
    dtype = _DTYPES.get(t.dtype)
    if dtype is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    rows, cols = t.shape
    sr, sc = t.stride()
    if cols > 1 and sc != 1:
        raise ValueError("rows must be contiguous (unit column stride)")
    return dtype, rows, cols, max(sr if rows > 1 else cols, 1)


def _coded(q, name, fmt):
    if not isinstance(q, MxTensor):
        raise TypeError(f"{name} must be an MxTensor")
    if q.fmt != fmt:
        raise ValueError(f"{name} must have {fmt} elements")
    if not q.codes.is_cuda:
        raise ValueError(f"{name} must be on the GPU")


def _same_device(a, b):
    if a.device != b.device:
        raise ValueError(f"operands on different devices: {a.device} and {b.device}")


def _check(st, name):
    if st != gemm.GEMM_OK:
        raise gemm.GemmError(st, name)


def _out_dtype(dtype, default, name):
    dtype = dtype or default
    if dtype not in _DTYPES:
        raise TypeError(f"{name} must be float32, float16 or bfloat16")
    return dtype


def _scale_row(blocks: int) -> int:
    unit = 4 if blocks < 16 else 16
    return -(-blocks // unit) * unit


def empty(rows: int, cols: int, fmt: str, device) -> MxTensor:
    """An uninitialised coded matrix; scale rows are a multiple of 4 bytes, or
    of 16 where they are that long (the widest pieces the kernels copy)."""
    if _torch is None:
        _load()
    if fmt not in FORMATS:
        raise ValueError(f"unknown format {fmt!r}: {E2M1!r} or {E4M3!r}")
    blocks = -(-cols // BLOCK)
    q = MxTensor.__new__(MxTensor)  # (as the checks of __init__ would have it)
    q.codes = _torch.empty((rows, blocks * BLOCK_BYTES[fmt]), dtype=_torch.uint8, device=device)
    width = _scale_row(blocks)
    if width == blocks:
        q.scales = _torch.empty((rows, blocks), dtype=_torch.uint8, device=device)
    else:
        q.scales = _torch.empty_strided((rows, blocks), (width, 1), dtype=_torch.uint8, device=device)
    q.cols, q.fmt = cols, fmt
    return q


def quantize(x, fmt: str = E2M1, transposed: bool = False, out: MxTensor | None = None, stream=None) -> MxTensor:
    """The coded form of the 2-D tensor x (blocks along its rows), or with
    ``transposed`` of x.T (blocks down its columns)."""
    dtype, rows, cols, ldx = _dense(x, "x")
    shape = (cols, rows) if transposed else (rows, cols)
    on = _Launch(x, stream)
    if out is None:
        out = on.coded(*shape, fmt)
    else:
        _coded(out, "out", fmt)
        _same_device(x, out)
        if out.shape != shape:
            raise ValueError(f"out has shape {out.shape}, not {shape}")
    _check(lib().gemm_mx_quantize(dtype, FORMATS[fmt], 1 if transposed else 0, rows, cols, x.data_ptr(), ldx,
                                  *out._args(), on.handle), "gemm_mx_quantize")
    return out


def dequantize(q: MxTensor, dtype=None, transposed: bool = False, out=None, stream=None):
    """The values of a coded matrix (transposed: of its transpose) as a
    tensor of ``dtype`` (default bfloat16)."""
    if not isinstance(q, MxTensor):
        raise TypeError("q must be an MxTensor")
    if not q.codes.is_cuda:
        raise ValueError("q must be on the GPU")
    rows, cols = (q.cols, q.rows) if transposed else q.shape
    on = _Launch(q.codes, stream)
    if out is None:
        out = on.empty((rows, cols), _out_dtype(dtype, _torch.bfloat16, "dtype"))
    elif tuple(out.shape) != (rows, cols) or (dtype is not None and out.dtype != dtype):
        raise ValueError("out has the wrong shape or dtype")
    x_dtype, _, _, ldx = _dense(out, "out")
    _same_device(q, out)
    _check(lib().gemm_mx_dequantize(x_dtype, FORMATS[q.fmt], 1 if transposed else 0, rows, cols, *q._args(),
                                    out.data_ptr(), ldx, on.handle), "gemm_mx_dequantize")
    return out


def matmul(a, b: MxTensor, out=None, out_dtype=None, alpha: float = 1.0, beta: float = 0.0, bias=None,
           act: int = gemm.ACT_NONE, stream=None):
    """act(alpha * a @ b.T + beta * out + bias): a (M x K) an E2M1 MxTensor,
    or a tensor that is quantised to E2M1 on the way; b (N x K) an E2M1
    MxTensor (of a K x N weight: ``quantize(w, transposed=True)``).  The
    result is bfloat16 unless out or out_dtype says otherwise.  bias: N
    float32 values."""
    _coded(b, "b", E2M1)
    values = not isinstance(a, MxTensor)
    if values:
        a_dtype, M, K, lda = _dense(a, "a")
    else:
        _coded(a, "a", E2M1)
        M, K = a.shape
    _same_device(a, b)
    N = b.rows
    if b.cols != K:
        raise ValueError(f"inner dimensions differ: {K} vs {b.cols}")
    on = _Launch(b.codes, stream)
    if out is None:
        if beta != 0.0:
            raise ValueError("beta needs out")
        out = on.empty((M, N), _out_dtype(out_dtype, _torch.bfloat16, "out_dtype"))
    elif tuple(out.shape) != (M, N) or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out has the wrong shape or dtype")
    c_dtype, _, _, ldc = _dense(out, "out")
    _same_device(out, b)
    epi = None
    if alpha != 1.0 or beta != 0.0 or bias is not None or act != gemm.ACT_NONE:
        if bias is not None and (bias.dtype != _torch.float32 or bias.numel() != N or not bias.is_contiguous()
                                 or bias.device != b.device):
            raise ValueError("bias must be a contiguous float32 GPU tensor of N values")
        epi = ctypes.byref(gemm.GemmEpilogue(float(alpha), float(beta),
                                             bias.data_ptr() if bias is not None else None, int(act)))
    if not values:
        _check(lib().gemm_mx_matmul(c_dtype, M, N, K, *a._args(), *b._args(), out.data_ptr(), ldc, on.handle, epi),
               "gemm_mx_matmul")
        return out
    x, coded, row = a.data_ptr(), b._args(), lda * a.element_size()
    # A decoding step's few rows need no workspace (the header's conditions).
    inside = (M <= 16 and (x | row) % 16 == 0 and (coded[2] | coded[3]) % 4 == 0 and N <= _FAR - 16
              and max(row, coded[1], coded[3]) < _FAR)
    need = 0 if inside else lib().gemm_mx_matmul_values_workspace_bytes(M, K)
    ws = on.empty(need, _torch.uint8) if need > 0 else None
    _check(lib().gemm_mx_matmul_values(a_dtype, c_dtype, M, N, K, x, lda, *coded, out.data_ptr(), ldc,
                                       ws.data_ptr() if ws is not None else None, need, on.handle, epi),
           "gemm_mx_matmul_values")
    return out


def checkpoint(x, out: MxTensor | None = None, stream=None) -> MxTensor:
    """The 8-bit checkpoint of activations x (tokens x features): E4M3 codes
    of x.T, in blocks of 32 tokens of one feature, about half of bfloat16's
    bytes.  `weight_grad` takes it as it is; `restore` gives the values."""
    return quantize(x, E4M3, transposed=True, out=out, stream=stream)


def restore(kept: MxTensor, dtype=None, out=None, stream=None):
    """The activations (tokens x features) that a checkpoint stands for."""
    _coded(kept, "kept", E4M3)
    return dequantize(kept, dtype=dtype, transposed=True, out=out, stream=stream)


def weight_grad(kept: MxTensor, dy, out=None, out_dtype=None, alpha: float = 1.0, beta: float = 0.0, stream=None):
    """dW = alpha * x.T @ dy + beta * out from x's checkpoint (features x
    tokens) and dy (tokens x N): features x N, float32 unless out or
    out_dtype says otherwise.  beta = 1 accumulates over micro-batches.  (A
    bfloat16 dy with N a multiple of 8 should have rows on 16 bytes; a slice
    that has not is up to nine times slower than its contiguous copy.)"""
    _coded(kept, "kept", E4M3)
    y_dtype, rows, N, ldy = _dense(dy, "dy")
    _same_device(kept, dy)
    F, T = kept.shape
    if rows != T:
        raise ValueError(f"tokens differ: {T} vs {rows}")
    on = _Launch(dy, stream)
    if out is None:
        if beta != 0.0:
            raise ValueError("beta needs out")
        out = on.empty((F, N), _out_dtype(out_dtype, _torch.float32, "out_dtype"))
    elif tuple(out.shape) != (F, N) or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out has the wrong shape or dtype")
    c_dtype, _, _, ldw = _dense(out, "out")
    _same_device(out, dy)
    need = lib().gemm_mx_wgrad_workspace_bytes(y_dtype, T, F, N)
    ws = on.empty(need, _torch.uint8) if need > 0 else None
    _check(lib().gemm_mx_wgrad(y_dtype, c_dtype, T, F, N, *kept._args(), dy.data_ptr(), ldy, out.data_ptr(), ldw,
                               alpha, beta, ws.data_ptr() if ws is not None else None, max(need, 0), on.handle),
           "gemm_mx_wgrad")
    return out


def _row_major(t) -> bool:
    rows, cols = t.shape
    return (cols <= 1 or t.stride(1) == 1) and (rows <= 1 or t.stride(0) >= cols)


_Linear = None


def linear(x, w, wq: MxTensor):
    """y = x @ w for training: the forward product in 4 bits, the backward
    pass from 8-bit activations.  x is tokens x K, w the K x N weight (any of
    float32, float16, bfloat16; x of the same type; row-major or the transpose
    of a row-major N x K parameter), wq its coded form
    ``quantize(w, transposed=True)`` (of such a parameter:
    ``quantize(parameter)``), remade by the caller after each weight update.
    Saved for backward are w and the 8-bit checkpoint of x, not x.
    Gradients: dx = dy @ w.T with w itself, not its 4-bit values, and dw =
    x^.T @ dy with x^ the 8-bit checkpoint's values, not the 4-bit ones that
    the product took; both in w's type.  There is no second derivative."""
    global _Linear
    if _Linear is None:
        _Linear = _make_linear()
    return _Linear.apply(x, w, wq)


def _make_linear():
    import torch

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, wq):
            if x.dtype != w.dtype:
                raise TypeError("x and w must have one type")
            if wq.shape != (w.shape[1], w.shape[0]):
                raise ValueError("wq is not the coded form of w.T")
            if not (_row_major(w) or _row_major(w.t())):
                raise ValueError("w must be row-major or the transpose of a row-major tensor")
            _same_device(x, w)
            y = matmul(x, wq, out_dtype=x.dtype)
            codes = scales = None
            if ctx.needs_input_grad[1]:
                # (The scales' rows with their padding: a hook that copies a
                # saved tensor keeps its shape, but no padding in strides.)
                T, F = x.shape
                blocks = -(-T // BLOCK)
                codes = torch.empty((F, blocks * BLOCK_BYTES[E4M3]), dtype=torch.uint8, device=x.device)
                scales = torch.empty((F, _scale_row(blocks)), dtype=torch.uint8, device=x.device)
                checkpoint(x, out=MxTensor(codes, scales[:, :blocks], T, E4M3))
            ctx.save_for_backward(w, codes, scales)
            return y

        @staticmethod
        @torch.autograd.function.once_differentiable  # (the kernels record no graph)
        def backward(ctx, dy):
            w, codes, scales = ctx.saved_tensors
            if not _row_major(dy):
                dy = dy.contiguous()  # an expanded or transposed gradient
            dx = dw = None
            if ctx.needs_input_grad[0]:
                dx = gemm.matmul(dy, w, b_transposed=True) if _row_major(w) else gemm.matmul(dy, w.t())
            if ctx.needs_input_grad[1]:
                T = dy.shape[0]
                dw = weight_grad(MxTensor(codes, scales[:, :-(-T // BLOCK)], T, E4M3), dy, out_dtype=w.dtype)
            return dx, dw, None

    return Linear
