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
EXPORTS = ["gemm_mx_quantize", "gemm_mx_dequantize", "gemm_mx_matmul", "gemm_mx_wgrad",
           "gemm_mx_wgrad_workspace_bytes"]

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
        for name in ("gemm_mx_quantize", "gemm_mx_dequantize", "gemm_mx_matmul", "gemm_mx_wgrad"):
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


def gemm_mx_wgrad(y_dtype, c_dtype, T, F, N, codes, ldq, scales, lds, dY, ldy, dW, ldw, alpha=1.0, beta=0.0,
                  workspace=None, workspace_bytes=0, stream=None) -> int:
    return lib().gemm_mx_wgrad(y_dtype, c_dtype, T, F, N, codes, ldq, scales, lds, dY, ldy, dW, ldw,
                               alpha, beta, workspace, workspace_bytes, stream)


def gemm_mx_wgrad_workspace_bytes(y_dtype, T, F, N) -> int:
    return lib().gemm_mx_wgrad_workspace_bytes(y_dtype, T, F, N)


# --------------------------------------------------------------------------
# Torch forms.
# --------------------------------------------------------------------------
_DTYPES = None


def _dtypes():
    global _DTYPES
    if _DTYPES is None:
        import torch
        _DTYPES = {torch.float32: gemm.DTYPE_F32, torch.float16: gemm.DTYPE_F16,
                   torch.bfloat16: gemm.DTYPE_BF16}
    return _DTYPES


class MxTensor:
    """A coded matrix (the format of include/gemm_mx.h): ``codes`` (uint8,
    rows x 16 or 32 bytes a block) and ``scales`` (uint8, rows x blocks), for
    ``cols`` values a row.  Both may be views with a larger row stride; codes
    need 16-byte alignment and a row stride of a multiple of 16."""
    __slots__ = ("codes", "scales", "cols", "fmt")

    def __init__(self, codes, scales, cols: int, fmt: str = E2M1):
        if fmt not in FORMATS:
            raise ValueError(f"unknown format {fmt!r}: {E2M1!r} or {E4M3!r}")
        blocks = -(-cols // BLOCK)
        if codes.dim() != 2 or scales.dim() != 2 or codes.element_size() != 1 or scales.element_size() != 1:
            raise ValueError("codes and scales must be 2-D tensors of bytes")
        if codes.shape[0] != scales.shape[0]:
            raise ValueError("codes and scales differ in rows")
        if codes.shape[1] != blocks * BLOCK_BYTES[fmt] or scales.shape[1] != blocks:
            raise ValueError(f"{cols} columns need {blocks * BLOCK_BYTES[fmt]} code bytes and {blocks} scales a row")
        if (codes.shape[1] > 1 and codes.stride(1) != 1) or (scales.shape[1] > 1 and scales.stride(1) != 1):
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
        many = c.shape[0] > 1
        return (c.data_ptr(), c.stride(0) if many else -(-c.shape[1] // 16) * 16,
                s.data_ptr(), s.stride(0) if many else s.shape[1])

    def __repr__(self) -> str:
        return f"MxTensor({self.rows} x {self.cols}, {self.fmt}, {self.device})"


def _stream(t, stream):
    import torch
    if stream is None:
        return torch.cuda.current_stream(t.device).cuda_stream
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


class _On:
    """Allocations on the launch stream, so that torch's allocator orders
    their reuse after the kernels (the current stream is left as it is)."""

    def __init__(self, device, stream):
        import torch
        self.ctx = None
        if stream != torch.cuda.current_stream(device).cuda_stream:
            self.ctx = torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device))

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _dense(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name}: expected a 2-D tensor")
    if t.dtype not in _dtypes():
        raise TypeError(f"{name} must be float32, float16 or bfloat16")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    return gemm._ld(t)


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


def empty(rows: int, cols: int, fmt: str, device) -> MxTensor:
    """An uninitialised coded matrix; scale rows are a multiple of 4 bytes."""
    import torch
    if fmt not in FORMATS:
        raise ValueError(f"unknown format {fmt!r}: {E2M1!r} or {E4M3!r}")
    blocks = -(-cols // BLOCK)
    codes = torch.empty((rows, blocks * BLOCK_BYTES[fmt]), dtype=torch.uint8, device=device)
    scales = torch.empty((rows, -(-blocks // 4) * 4), dtype=torch.uint8, device=device)
    return MxTensor(codes, scales[:, :blocks], cols, fmt)


def quantize(x, fmt: str = E2M1, transposed: bool = False, out: MxTensor | None = None, stream=None) -> MxTensor:
    """The coded form of the 2-D tensor x (blocks along its rows), or with
    ``transposed`` of x.T (blocks down its columns)."""
    ldx = _dense(x, "x")
    rows, cols = x.shape
    shape = (cols, rows) if transposed else (rows, cols)
    s = _stream(x, stream)
    if out is None:
        with _On(x.device, s):
            out = empty(*shape, fmt, x.device)
    else:
        _coded(out, "out", fmt)
        _same_device(x, out)
        if out.shape != shape:
            raise ValueError(f"out has shape {out.shape}, not {shape}")
    c, ldq, sc, lds = out._args()
    _check(lib().gemm_mx_quantize(_dtypes()[x.dtype], FORMATS[fmt], int(transposed), rows, cols, x.data_ptr(), ldx,
                                  c, ldq, sc, lds, s), "gemm_mx_quantize")
    return out


def dequantize(q: MxTensor, dtype=None, transposed: bool = False, out=None, stream=None):
    """The values of a coded matrix (transposed: of its transpose) as a
    tensor of ``dtype`` (default bfloat16)."""
    import torch
    if not isinstance(q, MxTensor):
        raise TypeError("q must be an MxTensor")
    if not q.codes.is_cuda:
        raise ValueError("q must be on the GPU")
    shape = (q.cols, q.rows) if transposed else (q.rows, q.cols)
    s = _stream(q, stream)
    if out is None:
        dtype = dtype or torch.bfloat16
        if dtype not in _dtypes():
            raise TypeError("dtype must be float32, float16 or bfloat16")
        with _On(q.device, s):
            out = torch.empty(shape, dtype=dtype, device=q.device)
    elif tuple(out.shape) != shape or (dtype is not None and out.dtype != dtype):
        raise ValueError("out has the wrong shape or dtype")
    ldx = _dense(out, "out")
    _same_device(q, out)
    c, ldq, sc, lds = q._args()
    _check(lib().gemm_mx_dequantize(_dtypes()[out.dtype], FORMATS[q.fmt], int(transposed), shape[0], shape[1],
                                    c, ldq, sc, lds, out.data_ptr(), ldx, s), "gemm_mx_dequantize")
    return out


def matmul(a, b: MxTensor, out=None, out_dtype=None, alpha: float = 1.0, beta: float = 0.0, bias=None,
           act: int = gemm.ACT_NONE, stream=None):
    """act(alpha * a @ b.T + beta * out + bias): a (M x K) an E2M1 MxTensor,
    or a tensor that is quantised to E2M1 on the way; b (N x K) an E2M1
    MxTensor (of a K x N weight: ``quantize(w, transposed=True)``).  The
    result is bfloat16 unless out or out_dtype says otherwise.  bias: N
    float32 values."""
    import torch
    _coded(b, "b", E2M1)
    if not isinstance(a, MxTensor):
        _dense(a, "a")
    else:
        _coded(a, "a", E2M1)
    _same_device(a, b)
    M, K = a.shape
    N = b.rows
    if b.cols != K:
        raise ValueError(f"inner dimensions differ: {K} vs {b.cols}")
    s = _stream(b, stream)
    if not isinstance(a, MxTensor):
        a = quantize(a, E2M1, stream=s)
    if out is None:
        if beta != 0.0:
            raise ValueError("beta needs out")
        out_dtype = out_dtype or torch.bfloat16
        if out_dtype not in _dtypes():
            raise TypeError("out_dtype must be float32, float16 or bfloat16")
        with _On(b.device, s):
            out = torch.empty((M, N), dtype=out_dtype, device=b.device)
    elif tuple(out.shape) != (M, N) or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out has the wrong shape or dtype")
    ldc = _dense(out, "out")
    _same_device(out, b)
    epi = None
    if alpha != 1.0 or beta != 0.0 or bias is not None or act != gemm.ACT_NONE:
        if bias is not None and (bias.dtype != torch.float32 or bias.numel() != N or not bias.is_contiguous()
                                 or bias.device != b.device):
            raise ValueError("bias must be a contiguous float32 GPU tensor of N values")
        epi = ctypes.byref(gemm.GemmEpilogue(float(alpha), float(beta),
                                             bias.data_ptr() if bias is not None else None, int(act)))
    _check(lib().gemm_mx_matmul(_dtypes()[out.dtype], M, N, K, *a._args(), *b._args(), out.data_ptr(), ldc, s, epi),
           "gemm_mx_matmul")
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
    out_dtype says otherwise.  beta = 1 accumulates over micro-batches."""
    import torch
    _coded(kept, "kept", E4M3)
    ldy = _dense(dy, "dy")
    _same_device(kept, dy)
    F, T = kept.shape
    N = dy.shape[1]
    if dy.shape[0] != T:
        raise ValueError(f"tokens differ: {T} vs {dy.shape[0]}")
    s = _stream(dy, stream)
    y_dtype = _dtypes()[dy.dtype]
    need = lib().gemm_mx_wgrad_workspace_bytes(y_dtype, T, F, N)
    ws = None
    if out is not None and (tuple(out.shape) != (F, N) or (out_dtype is not None and out.dtype != out_dtype)):
        raise ValueError("out has the wrong shape or dtype")
    if out is None:
        if beta != 0.0:
            raise ValueError("beta needs out")
        out_dtype = out_dtype or torch.float32
        if out_dtype not in _dtypes():
            raise TypeError("out_dtype must be float32, float16 or bfloat16")
    with _On(dy.device, s):
        if out is None:
            out = torch.empty((F, N), dtype=out_dtype, device=dy.device)
        if need > 0:
            ws = torch.empty(need, dtype=torch.uint8, device=dy.device)
    ldw = _dense(out, "out")
    _same_device(out, dy)
    _check(lib().gemm_mx_wgrad(y_dtype, _dtypes()[out.dtype], T, F, N, *kept._args(), dy.data_ptr(), ldy,
                               out.data_ptr(), ldw, float(alpha), float(beta),
                               ws.data_ptr() if ws is not None else None, need if ws is not None else 0, s),
           "gemm_mx_wgrad")
    return out


_Linear = None


def linear(x, w, wq: MxTensor):
    """y = x @ w for training: the forward product in 4 bits, the backward
    pass from 8-bit activations.  x is tokens x K, w the K x N weight (any of
    float32, float16, bfloat16; x of the same type), wq its coded form
    ``quantize(w, transposed=True)``, remade by the caller after each weight
    update.  Saved for backward are w and the 8-bit checkpoint of x, not x.
    Gradients (straight through the quantisation): dx = dy @ w.T and dw =
    x^.T @ dy with x^ the checkpoint's values, both in w's type."""
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
            ctx.kept = checkpoint(x) if ctx.needs_input_grad[1] else None
            ctx.save_for_backward(w)
            return matmul(x, wq, out_dtype=x.dtype)

        @staticmethod
        def backward(ctx, dy):
            w, = ctx.saved_tensors
            if dy.dim() == 2 and dy.shape[1] > 1 and dy.stride(1) != 1 or (dy.shape[0] > 1 and dy.stride(0) < dy.shape[1]):
                dy = dy.contiguous()  # an expanded or transposed gradient
            dx = gemm.matmul(dy, w, b_transposed=True) if ctx.needs_input_grad[0] else None
            dw = weight_grad(ctx.kept, dy, out_dtype=w.dtype) if ctx.needs_input_grad[1] else None
            return dx, dw, None

    return Linear
