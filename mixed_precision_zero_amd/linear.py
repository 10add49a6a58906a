"""Binding of the linear layer's operators of libneox_zero1.so (include/neox_linear.h): the
product with bias, activation, dropout and residual, its gradients, dropout by itself, and
the layer on MXFP4 copies.

As in the package itself, the functions with C names take addresses and only marshal
arguments; below them are the conveniences that take torch tensors.  Those run on the
current stream of their tensors' device, take their workspace from torch's allocator on
that stream, and reject what the operators do not cover; nothing falls back to torch.
They are no part of torch's autograd: results carry no graph, even of inputs that require
gradients; those are for the backward functions to make.
"""
from __future__ import annotations

import ctypes as C

import mixed_precision_zero_amd as Z
from mixed_precision_zero_amd import NEOX_BF16, NEOX_F16, NeoxError, _check  # noqa: F401
from mixed_precision_zero_amd.matrix import (MXFP4, NEOX_F32, _code, _on, _rows_of,  # noqa: F401
                                             mxfp4_quantize)

NEOX_ACT_NONE, NEOX_ACT_RELU, NEOX_ACT_GELU, NEOX_ACT_GELU_TANH, NEOX_ACT_SILU = range(5)
ACTS = {"none": NEOX_ACT_NONE, "relu": NEOX_ACT_RELU, "gelu": NEOX_ACT_GELU,
        "gelu_tanh": NEOX_ACT_GELU_TANH, "silu": NEOX_ACT_SILU}

_V, _U, _I = C.c_void_p, C.c_uint64, C.c_int32


class neox_drop(C.Structure):
    _fields_ = [("p", C.c_double), ("seed", _U), ("offset", _U), ("counter", _V)]


class neox_epilogue(C.Structure):
    _fields_ = [("dtype", _I), ("act", _I), ("bias", _V), ("residual", _V), ("residual_ld", _U),
                ("pre", _V), ("pre_ld", _U), ("drop", neox_drop)]


class neox_linear_args(C.Structure):
    _fields_ = [("x", _V), ("w", _V), ("y", _V), ("x_ld", _U), ("w_ld", _U), ("y_ld", _U),
                ("m", _U), ("n", _U), ("k", _U), ("y_dtype", _I), ("reserved", _I),
                ("epi", neox_epilogue)]


class neox_linear_grads(C.Structure):
    _fields_ = [("dy", _V), ("pre", _V), ("x", _V), ("w", _V), ("dx", _V), ("dw", _V),
                ("dbias", _V), ("dy_ld", _U), ("pre_ld", _U), ("x_ld", _U), ("w_ld", _U),
                ("dx_ld", _U), ("dw_ld", _U), ("m", _U), ("n", _U), ("k", _U), ("dtype", _I),
                ("act", _I), ("accumulate", _I), ("reserved", _I), ("drop", neox_drop)]


# Every symbol include/neox_linear.h declares.
EXPORTS = ("neox_linear_workspace", "neox_linear", "neox_linear_backward_workspace",
           "neox_linear_backward", "neox_mxfp4_linear", "neox_dropout",
           "neox_dropout_backward_workspace", "neox_dropout_backward")

_lib = None
_byref = C.byref


def lib():
    """The loaded library with these functions' signatures; raises if it is not built."""
    global _lib
    L = Z.lib()
    if _lib is not L:
        P = C.POINTER
        L.neox_linear_workspace.argtypes = [P(neox_linear_args), P(_U)]
        L.neox_linear.argtypes = [P(neox_linear_args), _V, _U, _V]
        L.neox_linear_backward_workspace.argtypes = [P(neox_linear_grads), P(_U)]
        L.neox_linear_backward.argtypes = [P(neox_linear_grads), _V, _U, _V]
        L.neox_mxfp4_linear.argtypes = [_V, _V, _U, _V, _V, _U, _U, _V, _I, _U, P(neox_epilogue), _V]
        L.neox_dropout.argtypes = [_V, _U, _V, _V, _U, _V, _U, _U, _U, _I, P(neox_drop), _V]
        L.neox_dropout_backward_workspace.argtypes = [_U, _U, P(_U)]
        L.neox_dropout_backward.argtypes = [_V, _U, _V, _U, _V, _I, _U, _U, _I, P(neox_drop), _V, _U, _V]
        for name in EXPORTS:
            getattr(L, name).restype = C.c_int
        _lib = L
    return L


# --------------------------------------------------------------------------------------
# C names
# --------------------------------------------------------------------------------------

def neox_linear_workspace(args: neox_linear_args) -> int:
    n = _U()
    _check(lib().neox_linear_workspace(_byref(args), _byref(n)))
    return n.value


def neox_linear(args: neox_linear_args, workspace=0, workspace_bytes=0, stream_ptr=0):
    _check(lib().neox_linear(C.byref(args), workspace, workspace_bytes, stream_ptr))


def neox_linear_backward_workspace(args: neox_linear_grads) -> int:
    n = _U()
    _check(lib().neox_linear_backward_workspace(C.byref(args), C.byref(n)))
    return n.value


def neox_linear_backward(args: neox_linear_grads, workspace=0, workspace_bytes=0, stream_ptr=0):
    _check(lib().neox_linear_backward(C.byref(args), workspace, workspace_bytes, stream_ptr))


def neox_mxfp4_linear(a_codes, a_scales, m, b_codes, b_scales, n, k, c, dtype, ldc,
                      epi: neox_epilogue, stream_ptr=0):
    _check(lib().neox_mxfp4_linear(a_codes, a_scales, m, b_codes, b_scales, n, k, c, dtype, ldc,
                                   C.byref(epi), stream_ptr))


def neox_dropout(x, x_ld, bias, residual, residual_ld, y, y_ld, rows, cols, dtype,
                 drop: neox_drop | None, stream_ptr=0):
    _check(lib().neox_dropout(x, x_ld, bias, residual, residual_ld, y, y_ld, rows, cols, dtype,
                              None if drop is None else C.byref(drop), stream_ptr))


def neox_dropout_backward_workspace(rows: int, cols: int) -> int:
    n = _U()
    _check(lib().neox_dropout_backward_workspace(rows, cols, C.byref(n)))
    return n.value


def neox_dropout_backward(dy, dy_ld, dx, dx_ld, dbias, accumulate, rows, cols, dtype,
                          drop: neox_drop | None, workspace=0, workspace_bytes=0, stream_ptr=0):
    _check(lib().neox_dropout_backward(dy, dy_ld, dx, dx_ld, dbias, accumulate, rows, cols, dtype,
                                       None if drop is None else C.byref(drop), workspace,
                                       workspace_bytes, stream_ptr))


# --------------------------------------------------------------------------------------
# torch-facing conveniences
# --------------------------------------------------------------------------------------

class Dropout:
    """A mask: probability p, seed and offset of the counter-based generator (64 bits each).
    counter: an int64 CUDA tensor of one element that is added to the offset when the work
    runs, so that replays of a captured graph draw masks of their own."""

    __slots__ = ("c", "counter")

    def __init__(self, p: float, seed: int, offset: int = 0, counter=None):
        if not 0.0 <= p <= 1.0:
            raise ValueError("p must be in [0, 1]")
        for v, name in ((seed, "seed"), (offset, "offset")):
            if not 0 <= v < 1 << 64:
                raise ValueError(f"{name} must be in [0, 2^64)")
        if counter is not None:
            import torch
            if not counter.is_cuda or counter.dtype != torch.int64 or counter.numel() != 1:
                raise ValueError("counter must be an int64 CUDA tensor of one element")
        self.counter = counter
        self.c = neox_drop(p, seed, offset, None if counter is None else counter.data_ptr())

    def __repr__(self):
        return f"Dropout(p={self.c.p}, seed={self.c.seed}, offset={self.c.offset})"


def _act(name) -> int:
    if name not in ACTS:
        raise ValueError(f"act {name!r}: one of {', '.join(ACTS)}")
    return ACTS[name]


def _half(t, name) -> int:
    code = _code(t.dtype)
    if code == NEOX_F32:
        raise ValueError(f"{name} must be float16 or bfloat16")
    return code


def _vector(t, name, n, dtype, device):
    if t.shape != (n,) or t.dtype != dtype or t.device != device or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must hold {n} adjacent elements of {dtype} on {device}")
    return t.data_ptr()


def _matrix(t, name, m, n, dtype, device):
    """(address, row stride) of an m x n matrix of that type and (CUDA) device."""
    if t.dtype != dtype or t.device != device or t.shape != (m, n):
        raise ValueError(f"{name} must be {m} x {n} of {dtype} on {device}")
    return t.data_ptr(), n if t.is_contiguous() else _rows_of(t, name)


def _drop_of(drop, device):
    if drop is not None and drop.counter is not None and drop.counter.device != device:
        raise ValueError("the dropout's counter is on another device")
    return drop


def _epilogue(epi, half, device, m, n, y, bias, act, dropout, residual, pre):
    """Fills epi; returns pre's tensor or None."""
    import torch
    epi.dtype = _code(half)
    epi.act = _act(act)
    if bias is not None:
        epi.bias = _vector(bias, "bias", n, half, device)
    if residual is not None:
        epi.residual, epi.residual_ld = _matrix(residual, "residual", m, n, y.dtype, device)
    if pre is True:
        pre = torch.empty((m, n), dtype=half, device=device)
        epi.pre, epi.pre_ld = pre.data_ptr(), n
    elif pre is False or pre is None:
        pre = None
    else:
        epi.pre, epi.pre_ld = _matrix(pre, "pre", m, n, half, device)
    if _drop_of(dropout, device) is not None:
        epi.drop = dropout.c
    return pre


def _result(out, m, n, dtype, device):
    """(tensor, row stride) of the result."""
    import torch
    if out is None:
        return torch.empty((m, n), dtype=dtype, device=device), n
    if out.shape != (m, n) or out.device != device or (dtype is not None and out.dtype != dtype):
        raise ValueError("out must have the result's shape and device, and the type asked for")
    return out, _rows_of(out, "out")


def _space(need, device):
    """(tensor, address) of a workspace."""
    import torch
    if not need:
        return None, 0
    t = torch.empty(need, dtype=torch.uint8, device=device)
    return t, t.data_ptr()


def linear(x, w, bias=None, act: str = "none", dropout: Dropout | None = None, residual=None,
           dtype=None, out=None, pre=False):
    """residual + dropout(act(x w^T + bias)) of x (m, k) and w (n, k), both float16 or bfloat16,
    as a new (m, n) matrix of type `dtype` (x's by default, or float32) or in out, which may be
    the residual.  Returns (result, pre): pre is x w^T + bias in x's type if it is asked for
    (True, or a tensor for it), as linear_backward needs it for an act; else None."""
    half, device = x.dtype, x.device
    _half(x, "x")
    x_ld = _rows_of(x, "x")
    m, k = x.shape
    if w.dim() != 2 or w.shape[1] != k:
        raise ValueError("x and w must have the same number of columns")
    n = w.shape[0]
    a = neox_linear_args()
    a.w, a.w_ld = _matrix(w, "w", n, k, half, device)
    guard, stream = _on(x)
    with guard:
        y, a.y_ld = _result(out, m, n, dtype if out is not None else dtype or half, device)
        pre = _epilogue(a.epi, half, device, m, n, y, bias, act, dropout, residual, pre)
        a.x, a.x_ld, a.y = x.data_ptr(), x_ld, y.data_ptr()
        a.m, a.n, a.k, a.y_dtype = m, n, k, _code(y.dtype)
        need = neox_linear_workspace(a)
        work, at = _space(need, device)
        neox_linear(a, at, need, stream)
    return y, pre


def linear_backward(dy, x=None, w=None, pre=None, act: str = "none", dropout: Dropout | None = None,
                    dx=True, dw=True, dbias=False, accumulate: bool = False):
    """The gradients of linear's result for dy: (dx, dw, dbias), each made where it is True, a
    tensor for it, or False (None comes back).  x is needed for dw, w for dx, pre for an act.
    accumulate: dw and dbias, given as tensors, are added to."""
    import torch
    half, device = dy.dtype, dy.device
    a = neox_linear_grads()
    a.dtype = _half(dy, "dy")
    a.act = _act(act)
    a.dy_ld = _rows_of(dy, "dy")
    m, n = dy.shape
    want = [t is not None and t is not False for t in (dx, dw, dbias)]
    if want[1] and x is None or want[0] and w is None:
        raise ValueError("dw needs x, and dx needs w")
    if accumulate and (dw is True or dbias is True):
        raise ValueError("accumulate adds to tensors that are given")
    if want[0]:
        k = w.shape[1]
    elif want[1]:
        k = x.shape[1]
    else:
        k = 1
    if want[1]:
        a.x, a.x_ld = _matrix(x, "x", m, k, half, device)
    if want[0]:
        a.w, a.w_ld = _matrix(w, "w", n, k, half, device)
    if a.act:
        if pre is None:
            raise ValueError("an act's gradient needs pre")
        a.pre, a.pre_ld = _matrix(pre, "pre", m, n, half, device)
    if _drop_of(dropout, device) is not None:
        a.drop = dropout.c
    guard, stream = _on(dy)
    with guard:
        if dx is True:
            dx = torch.empty((m, k), dtype=half, device=device)
            a.dx, a.dx_ld = dx.data_ptr(), k
        elif want[0]:
            a.dx, a.dx_ld = _matrix(dx, "dx", m, k, half, device)
        if dw is True:
            dw = torch.empty((n, k), dtype=half, device=device)
            a.dw, a.dw_ld = dw.data_ptr(), k
        elif want[1]:
            a.dw, a.dw_ld = _matrix(dw, "dw", n, k, half, device)
        if dbias is True:
            dbias = torch.empty(n, dtype=half, device=device)
            a.dbias = dbias.data_ptr()
        elif want[2]:
            a.dbias = _vector(dbias, "dbias", n, half, device)
        a.dy, a.m, a.n, a.k, a.accumulate = dy.data_ptr(), m, n, k, int(accumulate)
        need = neox_linear_backward_workspace(a)
        work, at = _space(need, device)
        neox_linear_backward(a, at, need, stream)
    return dx if want[0] else None, dw if want[1] else None, dbias if want[2] else None


def mxfp4_linear(x, w: MXFP4, bias=None, act: str = "none", dropout: Dropout | None = None,
                 residual=None, dtype=None, out=None, pre=False, half=None):
    """linear on the MXFP4 copy w of an n x k weight, by the MXFP4 copy of x: x is one, or a
    matrix (of one row or more) of which one is made.  half: the type of bias and pre (x's where
    x is a float16 or bfloat16 matrix, else bfloat16).  dtype: the result's, `half` by default,
    float16, bfloat16 or float32; of the half types only `half`."""
    import torch
    if not isinstance(x, MXFP4):
        if half is None and x.dtype != torch.float32:
            half = x.dtype
        x = mxfp4_quantize(x)
    half = half or torch.bfloat16
    if _code(half) == NEOX_F32:
        raise ValueError("half must be float16 or bfloat16")
    if x.cols != w.cols or x.device != w.device:
        raise ValueError("x and w must have the same number of columns, on one device")
    m, n, device = x.rows, w.rows, x.device
    epi = neox_epilogue()
    y, ldc = _result(out, m, n, dtype if out is not None else dtype or half, device)
    pre = _epilogue(epi, half, device, m, n, y, bias, act, dropout, residual, pre)
    guard, stream = _on(y)
    with guard:
        neox_mxfp4_linear(*x._at, m, *w._at, n, x.cols, y.data_ptr(), _code(y.dtype), ldc, epi, stream)
    return y, pre


def dropout(x, drop: Dropout | None, bias=None, residual=None, out=None):
    """residual + drop(x + bias) of a matrix x, in a new matrix or in out, which may be x or the
    residual.  drop None: no dropout."""
    m, n = x.shape
    x_ld = _rows_of(x, "x")
    y, y_ld = _result(out, m, n, x.dtype, x.device)
    b = None if bias is None else _vector(bias, "bias", n, x.dtype, x.device)
    r, r_ld = (None, 0) if residual is None else _matrix(residual, "residual", m, n, x.dtype, x.device)
    _drop_of(drop, x.device)
    guard, stream = _on(x)
    with guard:
        neox_dropout(x.data_ptr(), x_ld, b, r, r_ld, y.data_ptr(), y_ld, m, n, _code(x.dtype),
                     None if drop is None else drop.c, stream)
    return y


def dropout_backward(dy, drop: Dropout | None, dx=True, dbias=False, accumulate: bool = False):
    """The gradients of dropout's result for dy: (dx, dbias), each made where it is True, a tensor
    for it (dx may be dy), or False.  accumulate: dbias, given as a tensor, is added to."""
    import torch
    m, n = dy.shape
    dy_ld = _rows_of(dy, "dy")
    has_bias = dbias is not None and dbias is not False
    if accumulate and dbias is True:
        raise ValueError("accumulate adds to a tensor that is given")
    _drop_of(drop, dy.device)
    guard, stream = _on(dy)
    with guard:
        if dx is None or dx is False:
            dx, at, dx_ld = None, None, 0
        else:
            dx, dx_ld = _result(None if dx is True else dx, m, n, dy.dtype, dy.device)
            at = dx.data_ptr()
        if dbias is True:
            dbias = torch.empty(n, dtype=dy.dtype, device=dy.device)
        b = _vector(dbias, "dbias", n, dy.dtype, dy.device) if has_bias else None
        need = neox_dropout_backward_workspace(m, n) if has_bias else 0
        work, w_at = _space(need, dy.device)
        neox_dropout_backward(dy.data_ptr(), dy_ld, at, dx_ld, b, int(accumulate), m, n,
                              _code(dy.dtype), None if drop is None else drop.c, w_at, need, stream)
    return dx, dbias if has_bias else None
