"""Grouped products, a layer of experts: binding of include/gemm_grouped.h and
its torch forms.

The functions with the C names only marshal arguments.  The torch forms
(`matmul`, `weight_grad`) take GPU tensors, allocate results with torch on the
launch stream, and run the HIP kernels of ``libgemm.so``; there is no fallback.
Nothing of a call waits for the GPU: the groups' sizes stay there.

A layer of experts in these terms (rows of x sorted by expert, w experts x K x
N, ``offsets`` an int32 GPU tensor of experts + 1 values)::

    y = grouped.matmul(x, w, offsets)
    dx = grouped.matmul(dy, w, offsets, transposed=True)
    dw = grouped.weight_grad(x, dy, offsets)

`linear` is that layer as a torch autograd function.  Its weights in 4 bits,
for decoding: ``w4.grouped_matmul``.
"""
from __future__ import annotations

import ctypes

from . import gemm, mx

EXPORTS = ["gemm_grouped_matmul", "gemm_grouped_wgrad"]

_declared = None


def lib():
    """The loaded libgemm with the signatures of gemm_grouped.h."""
    global _declared
    if _declared is None:
        L = gemm.lib()
        i64, i32, p, f = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float
        L.gemm_grouped_matmul.argtypes = [i32, i32, i32, i64, i64, i64, i64, p, p, i64, p, i64, i64, p, i64, i32, p]
        L.gemm_grouped_wgrad.argtypes = [i32, i32, i64, i64, i64, i64, p, p, i64, p, i64, p, i64, i64, f, f, p]
        for name in EXPORTS:
            getattr(L, name).restype = ctypes.c_int
        _declared = L
    return _declared


def gemm_grouped_matmul(dtype, c_dtype, trans_w, G, T, N, K, offsets, X, ldx, W, ldw, stride_w, Y, ldy, fill=0,
                        stream=None) -> int:
    return lib().gemm_grouped_matmul(dtype, c_dtype, trans_w, G, T, N, K, offsets, X, ldx, W, ldw, stride_w, Y, ldy, fill,
                                     stream)


def gemm_grouped_wgrad(dtype, c_dtype, G, T, K, N, offsets, X, ldx, dY, ldy, dW, ldw, stride_w, alpha=1.0, beta=0.0,
                       stream=None) -> int:
    return lib().gemm_grouped_wgrad(dtype, c_dtype, G, T, K, N, offsets, X, ldx, dY, ldy, dW, ldw, stride_w, alpha, beta,
                                    stream)


# --------------------------------------------------------------------------
# Torch forms (see mx.py for the launch stream and allocations).
# --------------------------------------------------------------------------
def _call(L, name, index, *args):
    """The C-ABI call with the operands' device as the current one."""
    if index == mx._torch._C._cuda_getDevice():
        status = getattr(L, name)(*args)
    else:
        with mx._torch.cuda.device(index):
            status = getattr(L, name)(*args)
    if status != gemm.GEMM_OK:
        raise gemm.GemmError(status, name)


def _stack(w, name):
    """(library dtype, groups, rows, columns, leading dimension, stride) of a
    GPU tensor of matrices."""
    if w.dim() != 3:
        raise ValueError(f"{name}: expected a 3-D tensor (groups x rows x columns)")
    if mx._torch is None:
        mx._load()
    dtype = mx._DTYPES.get(w.dtype)
    if dtype is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16")
    if not w.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    groups, rows, cols = w.shape
    sg, sr, sc = w.stride()
    if cols > 1 and sc != 1:
        raise ValueError(f"{name}: rows must be contiguous (unit column stride)")
    # (As mx._dense.)
    return dtype, groups, rows, cols, sr if rows > 1 and cols > 0 else max(cols, 1), sg if groups > 1 else rows * max(cols, 1)


def _offsets(offsets, groups, like):
    torch = mx._torch
    if not isinstance(offsets, torch.Tensor) or offsets.dtype != torch.int32 or offsets.dim() != 1:
        raise TypeError("offsets must be a 1-D int32 tensor")
    if offsets.shape[0] != groups + 1:
        raise ValueError(f"{groups} groups need {groups + 1} offsets, not {offsets.shape[0]}")
    if groups > 0 and offsets.stride(0) != 1:
        raise ValueError("offsets must be contiguous")
    mx._same_device(like, offsets)
    return offsets.data_ptr()


def _result_dtype(dtype, operand):
    if dtype not in (operand, mx._torch.float32):
        raise TypeError("the result has the operands' type or float32")
    return dtype


def _no_graph(name, instead):
    """Refuses an operand whose gradient the result would lose."""
    if mx._torch is None:
        mx._load()
    if mx._torch.is_grad_enabled():
        raise RuntimeError(f"{name} records no graph, so an operand that requires a gradient would get none: {instead}call it "
                           "under torch.no_grad() or with detached operands")


def _written(*tensors):
    """Tells autograd that a caller's tensors were written, as torch's own
    operators do: a graph that has saved one of them refuses its backward pass."""
    mx._torch.autograd.graph.increment_version(tensors)


def matmul(x, w, offsets, transposed: bool = False, out=None, out_dtype=None, stream=None):
    """y[t] = x[t] @ w[g] for the rows t of every group g, rows offsets[g] to
    offsets[g + 1] - 1 of x (T x K).  w is groups x K x N, or with
    ``transposed`` groups x N x K (y[t] = x[t] @ w[g].T), of x's type.  The
    result (T x N) has x's type or float32 (out_dtype).  Rows of no group are
    zero in a new result; in ``out`` they stay as they are.  No graph is
    recorded: where one would be (an operand requires a gradient and grad mode
    is on) the call is refused; `linear` records one."""
    if x.requires_grad or w.requires_grad:
        _no_graph("grouped.matmul", "use grouped.linear, or ")
    dtype, T, K, ldx = mx._dense(x, "x")
    w_dtype, G, rows, cols, ldw, stride_w = _stack(w, "w")
    N, inner = (rows, cols) if transposed else (cols, rows)
    if w_dtype != dtype:
        raise TypeError("x and w must have one type")
    if inner != K:
        raise ValueError(f"inner dimensions differ: {K} vs {inner}")
    mx._same_device(x, w)
    at = _offsets(offsets, G, x)
    on = mx._Launch(x, stream)
    fill = out is None
    if fill:
        out = on.empty((T, N), _result_dtype(out_dtype or x.dtype, x.dtype))
    elif tuple(out.shape) != (T, N) or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out has the wrong shape or dtype")
    c_dtype, _, _, ldy = mx._dense(out, "out")
    _result_dtype(out.dtype, x.dtype)
    mx._same_device(out, x)
    _call(lib(), "gemm_grouped_matmul", x.get_device(), dtype, c_dtype, 1 if transposed else 0, G, T, N, K, at, x.data_ptr(),
          ldx, w.data_ptr(), ldw, stride_w, out.data_ptr(), ldy, 1 if fill else 0, on.handle)
    if not fill:
        _written(out)
    return out


def weight_grad(x, dy, offsets, out=None, out_dtype=None, alpha: float = 1.0, beta: float = 0.0, stream=None):
    """dw[g] = alpha * x_g.T @ dy_g + beta * out[g] for every group's rows of
    x (T x K) and dy (T x N), of one type: groups x K x N, float32 unless out
    or out_dtype says x's type.  A group without rows has zeros (beta = 1: out
    as it is); beta = 1 accumulates over micro-batches.  The matrices of out lie
    one behind another (out.stride(0) at least a matrix's extent)."""
    dtype, T, K, ldx = mx._dense(x, "x")
    y_dtype, rows, N, ldy = mx._dense(dy, "dy")
    if y_dtype != dtype:
        raise TypeError("x and dy must have one type")
    if rows != T:
        raise ValueError(f"rows differ: {T} vs {rows}")
    mx._same_device(x, dy)
    if not isinstance(offsets, mx._torch.Tensor) or offsets.dim() != 1 or offsets.shape[0] < 1:
        raise TypeError("offsets must be a 1-D int32 tensor")
    G = offsets.shape[0] - 1
    at = _offsets(offsets, G, x)
    on = mx._Launch(x, stream)
    given = out is not None
    if not given:
        if beta != 0.0:
            raise ValueError("beta needs out")
        out = on.empty((G, K, N), _result_dtype(out_dtype or mx._torch.float32, x.dtype))
    elif tuple(out.shape) != (G, K, N) or (out_dtype is not None and out.dtype != out_dtype):
        raise ValueError("out has the wrong shape or dtype")
    c_dtype, _, _, _, ldw, stride_w = _stack(out, "out")
    _result_dtype(out.dtype, x.dtype)
    mx._same_device(out, x)
    _call(lib(), "gemm_grouped_wgrad", x.get_device(), dtype, c_dtype, G, T, K, N, at, x.data_ptr(), ldx, dy.data_ptr(),
          ldy, out.data_ptr(), ldw, stride_w, alpha, beta, on.handle)
    if given:
        _written(out)
    return out


_Linear = None


def linear(x, w, offsets, transposed: bool = False):
    """`matmul` for training: x is T x K, w groups x K x N (``transposed``:
    groups x N x K), of one type.  Gradients have that type too: dx = dy @
    w[g].T (zero for rows of no group) and dw[g] = x_g.T @ dy_g, summed in 32
    bits and rounded once.  There is no second derivative.

    A step captured into a graph: warm it up on the capturing stream, and let go
    of every result of an earlier step over the same leaves before the capture
    (torch's backward pass would end the process where a leaf's gradient
    belongs to another stream; `linear` refuses leaves of its own steps, it
    cannot see those of other operators)."""
    global _Linear
    if _Linear is None:
        _Linear = _make_linear()
    held = None  # (until the new graph holds it)
    if mx._torch.is_grad_enabled():
        held = [_accumulation(t) for t in (x, w)
                if isinstance(t, mx._torch.Tensor) and t.requires_grad and t.is_leaf and t.is_cuda]
    y = _Linear.apply(x, w, offsets, transposed)
    del held
    return y


def _accumulation(leaf):
    """The node that accumulates a leaf's gradient.  It lives as long as any
    graph with the leaf and belongs to the stream of the first of them: in a
    capture on another stream the leaf is refused."""
    node = leaf.view_as(leaf).grad_fn.next_functions[0][0]
    here = mx._raw_stream(leaf.get_device())
    first = node.metadata.setdefault("grouped.linear", here)
    if first != here and mx._torch.cuda.is_current_stream_capturing():
        raise RuntimeError("capture: results of an earlier step on another stream over the same leaf are alive")
    return node


def _make_linear():
    if mx._torch is None:
        mx._load()
    import torch

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, offsets, transposed):
            y = matmul(x, w, offsets, transposed)
            # (What a gradient does not need is not kept.)
            ctx.save_for_backward(x if ctx.needs_input_grad[1] else None, w if ctx.needs_input_grad[0] else None, offsets)
            ctx.transposed = transposed
            return y

        @staticmethod
        @torch.autograd.function.once_differentiable  # (the kernels record no graph)
        def backward(ctx, dy):
            x, w, offsets = ctx.saved_tensors
            if not mx._row_major(dy):
                dy = dy.contiguous()  # an expanded or transposed gradient
            dx = dw = None
            if ctx.needs_input_grad[0]:
                dx = matmul(dy, w, offsets, not ctx.transposed)
            if ctx.needs_input_grad[1]:
                a, b = (dy, x) if ctx.transposed else (x, dy)
                dw = weight_grad(a, b, offsets, out_dtype=x.dtype)
            return dx, dw, None, None

    return Linear
