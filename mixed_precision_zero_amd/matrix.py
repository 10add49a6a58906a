"""Binding of the matrix operators of libneox_zero1.so (include/neox_matrix.h): the
Newton-Schulz orthogonalisation, the Muon step, and the MXFP4 copy of a matrix with its
product.

As in the package itself, the functions with C names take addresses and only marshal
arguments; below them are the conveniences that take torch tensors.  Those run on the
current stream of their tensors' device, take their workspace from torch's allocator on
that stream, and reject what the operators do not cover; nothing falls back to torch.
"""
from __future__ import annotations

import contextlib
import ctypes as C

import mixed_precision_zero_amd as Z
from mixed_precision_zero_amd import (NEOX_BF16, NEOX_F16, NeoxError, _check,  # noqa: F401
                                      neox_scaler_state_t, neox_zero1_config)

NEOX_F32 = 3
NEOX_NS_MAX_STEPS = 16
NEOX_MUON_SCALE_SHAPE, NEOX_MUON_SCALE_RMS = 0, 1


class neox_ns_config(C.Structure):
    _fields_ = [("steps", C.c_int32), ("reserved", C.c_int32), ("eps", C.c_double),
                ("coef", (C.c_double * 3) * NEOX_NS_MAX_STEPS)]


class neox_muon_config(C.Structure):
    _fields_ = [("ns", neox_ns_config), ("nesterov", C.c_int32), ("scale_mode", C.c_int32),
                ("workspace_bytes", C.c_uint64)]


class neox_muon_matrix(C.Structure):
    _fields_ = [("grad", C.c_void_p), ("half", C.c_void_p), ("master", C.c_void_p),
                ("momentum", C.c_void_p), ("rows", C.c_uint64), ("cols", C.c_uint64),
                ("flags", C.c_uint32), ("reserved", C.c_uint32), ("mx_codes", C.c_void_p),
                ("mx_scales", C.c_void_p), ("mx_codes_t", C.c_void_p), ("mx_scales_t", C.c_void_p)]


# Every symbol include/neox_matrix.h declares.
EXPORTS = ("neox_ns_default_config", "neox_orthogonalize_workspace", "neox_orthogonalize",
           "neox_muon_default_config", "neox_muon_create", "neox_muon_step",
           "neox_muon_step_local", "neox_muon_step_apply", "neox_muon_state",
           "neox_muon_scaler_set", "neox_muon_destroy", "neox_mxfp4_layout",
           "neox_mxfp4_quantize", "neox_mxfp4_dequantize", "neox_mxfp4_product")

_lib = None


def lib():
    """The loaded library with these functions' signatures; raises if it is not built."""
    global _lib
    L = Z.lib()
    if _lib is not L:
        P, V, U, I = C.POINTER, C.c_void_p, C.c_uint64, C.c_int32
        L.neox_ns_default_config.argtypes = [P(neox_ns_config)]
        L.neox_orthogonalize_workspace.argtypes = [U, U, U, P(U)]
        L.neox_orthogonalize.argtypes = [P(neox_ns_config), V, I, U, U, V, I, U, U, U, U, U,
                                         C.c_double, V, U, V]
        L.neox_muon_default_config.argtypes = [P(neox_muon_config)]
        L.neox_muon_create.argtypes = [P(neox_zero1_config), P(neox_muon_config),
                                       P(neox_muon_matrix), U, V, P(V)]
        L.neox_muon_step.argtypes = [V, C.c_float, V]
        L.neox_muon_step_local.argtypes = [V, V, V]
        L.neox_muon_step_apply.argtypes = [V, V, C.c_uint32, C.c_float, V]
        L.neox_muon_state.argtypes = [V, P(neox_scaler_state_t)]
        L.neox_muon_scaler_set.argtypes = [V, P(neox_scaler_state_t), V]
        L.neox_muon_destroy.argtypes = [V]
        L.neox_mxfp4_layout.argtypes = [U, U, P(U), P(U)]
        L.neox_mxfp4_quantize.argtypes = [V, I, U, U, U, I, V, V, V]
        L.neox_mxfp4_dequantize.argtypes = [V, V, U, U, V, I, U, V]
        L.neox_mxfp4_product.argtypes = [V, V, U, V, V, U, U, V, I, U, V]
        for name in EXPORTS:
            getattr(L, name).restype = C.c_int
        _lib = L
    return L


# --------------------------------------------------------------------------------------
# C names
# --------------------------------------------------------------------------------------

def neox_ns_default_config(steps=None, eps=None, coef=None) -> neox_ns_config:
    """coef: one (a, b, c) for every step, or a list of one for each (which sets steps)."""
    cfg = neox_ns_config()
    _check(lib().neox_ns_default_config(C.byref(cfg)))
    if coef is not None:
        if len(coef) == 3 and not hasattr(coef[0], "__len__"):
            coef = [coef] * (cfg.steps if steps is None else steps)
        if len(coef) > NEOX_NS_MAX_STEPS or any(len(c) != 3 for c in coef):
            raise ValueError(f"coef: (a, b, c) of at most {NEOX_NS_MAX_STEPS} steps")
        for k, abc in enumerate(coef):
            cfg.coef[k][:] = abc
        cfg.steps = len(coef)
    if steps is not None:
        if coef is not None and steps != len(coef):
            raise ValueError("steps and the length of coef differ")
        cfg.steps = steps
    if eps is not None:
        cfg.eps = eps
    return cfg


def neox_orthogonalize_workspace(count: int, rows: int, cols: int) -> int:
    n = C.c_uint64()
    _check(lib().neox_orthogonalize_workspace(count, rows, cols, C.byref(n)))
    return n.value


def neox_orthogonalize(cfg, src, src_dtype, src_ld, src_stride, dst, dst_dtype, dst_ld, dst_stride,
                       count, rows, cols, scale, workspace, workspace_bytes, stream_ptr=0):
    _check(lib().neox_orthogonalize(C.byref(cfg), src, src_dtype, src_ld, src_stride, dst, dst_dtype,
                                    dst_ld, dst_stride, count, rows, cols, scale, workspace,
                                    workspace_bytes, stream_ptr))


def neox_muon_default_config(**overrides) -> neox_muon_config:
    cfg = neox_muon_config()
    _check(lib().neox_muon_default_config(C.byref(cfg)))
    for k, v in overrides.items():
        if not hasattr(cfg, k):
            raise AttributeError(k)
        setattr(cfg, k, v)
    return cfg


def neox_muon_create(cfg, mcfg, mats, stream_ptr: int = 0) -> int:
    arr = (neox_muon_matrix * max(1, len(mats)))(*mats)
    h = C.c_void_p()
    _check(lib().neox_muon_create(C.byref(cfg), C.byref(mcfg), arr, len(mats),
                                  C.c_void_p(stream_ptr), C.byref(h)))
    return h.value


def neox_muon_step(h: int, lr: float, stream_ptr: int = 0):
    _check(lib().neox_muon_step(C.c_void_p(h), C.c_float(lr), C.c_void_p(stream_ptr)))


def neox_muon_step_local(h: int, local_sumsq_ptr: int, stream_ptr: int = 0):
    _check(lib().neox_muon_step_local(C.c_void_p(h), C.c_void_p(local_sumsq_ptr),
                                      C.c_void_p(stream_ptr)))


def neox_muon_step_apply(h: int, rank_sumsq_ptr: int, lr: float, stream_ptr: int = 0,
                         nranks: int = 1):
    _check(lib().neox_muon_step_apply(C.c_void_p(h), C.c_void_p(rank_sumsq_ptr), nranks,
                                      C.c_float(lr), C.c_void_p(stream_ptr)))


def neox_muon_state(h: int) -> neox_scaler_state_t:
    st = neox_scaler_state_t()
    _check(lib().neox_muon_state(C.c_void_p(h), C.byref(st)))
    return st


def neox_muon_scaler_set(h: int, loss_scale: float, good_steps=0, step=0, skipped_total=0,
                         consecutive_overflows=0, stream_ptr: int = 0):
    st = neox_scaler_state_t()
    st.loss_scale = loss_scale
    st.good_steps = good_steps
    st.step = step
    st.skipped_total = skipped_total
    st.consecutive_overflows = consecutive_overflows
    _check(lib().neox_muon_scaler_set(C.c_void_p(h), C.byref(st), C.c_void_p(stream_ptr)))


def neox_muon_destroy(h: int):
    _check(lib().neox_muon_destroy(C.c_void_p(h)))


def neox_mxfp4_layout(rows: int, cols: int):
    """-> (bytes of the codes, bytes of the scales)."""
    a, b = C.c_uint64(), C.c_uint64()
    _check(lib().neox_mxfp4_layout(rows, cols, C.byref(a), C.byref(b)))
    return a.value, b.value


def neox_mxfp4_quantize(src, dtype, rows, cols, ld, transpose, codes, scales, stream_ptr=0):
    _check(lib().neox_mxfp4_quantize(src, dtype, rows, cols, ld, transpose, codes, scales, stream_ptr))


def neox_mxfp4_dequantize(codes, scales, rows, cols, dst, dtype, ld, stream_ptr=0):
    _check(lib().neox_mxfp4_dequantize(codes, scales, rows, cols, dst, dtype, ld, stream_ptr))


def neox_mxfp4_product(a_codes, a_scales, m, b_codes, b_scales, n, k, c, dtype, ldc, stream_ptr=0):
    _check(lib().neox_mxfp4_product(a_codes, a_scales, m, b_codes, b_scales, n, k, c, dtype, ldc,
                                    stream_ptr))


# --------------------------------------------------------------------------------------
# torch-facing conveniences
# --------------------------------------------------------------------------------------

_CODE = {}


def _code(dtype) -> int:
    if not _CODE:
        import torch
        _CODE.update({torch.float16: NEOX_F16, torch.bfloat16: NEOX_BF16, torch.float32: NEOX_F32})
    if dtype not in _CODE:
        raise ValueError(f"{dtype}: float16, bfloat16 or float32 needed")
    return _CODE[dtype]


def _rows_of(t, name):
    """The row stride of a 2-D CUDA tensor whose columns are adjacent."""
    if not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: elements of a row must be adjacent")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


_HERE = contextlib.nullcontext()
_stream_of = None


def _on(t):
    """(device guard, stream address) for work on t.  The guard does nothing where t's device is
    the current one already: entering one costs more than a small launch.  torch's accessor of
    the bare stream address, where it has it, saves making a Stream object (2 us)."""
    import torch
    global _stream_of
    if _stream_of is None:
        _stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
            (lambda i: torch.cuda.current_stream(i).cuda_stream)
    d = t.device
    guard = _HERE if torch.cuda.current_device() == d.index else torch.cuda.device(d)
    return guard, _stream_of(d.index)


def _batch(t, name, rows, cols):
    """t's matrices as one run: (elements from one to the next, elements from row to row)."""
    if t.is_contiguous():
        return rows * cols, cols
    if cols > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: elements of a row must be adjacent")
    ld = t.stride(-2) if rows > 1 else cols
    step, n = rows * ld, 1
    for size, stride in reversed(list(zip(t.shape[:-2], t.stride()[:-2]))):
        if size == 1:
            continue
        if n > 1 and stride != step * n:
            raise ValueError(f"{name}: the matrices must lie at one distance from each other")
        if n == 1:
            step = stride
        n *= size
    return step, ld


_default_ns = None

def orthogonalize(x, out=None, dtype=None, scale: float = 1.0, cfg: neox_ns_config | None = None):
    """scale * (the orthogonal factor of each matrix of x, approximately).  x: a matrix or a
    batch of them (..., rows, cols) with adjacent columns; out: the result's tensor (it may
    be x), else a new one of type `dtype` (x's by default)."""
    import torch
    if not x.is_cuda or x.dim() < 2:
        raise ValueError("x must be a CUDA tensor of at least two dimensions")
    if out is None:
        out = torch.empty(x.shape, dtype=dtype or x.dtype, device=x.device)
    elif out.shape != x.shape or out.device != x.device or (dtype is not None and out.dtype != dtype):
        raise ValueError("out must have x's shape and device, and the type asked for")
    global _default_ns
    if cfg is None:
        if _default_ns is None:
            _default_ns = neox_ns_default_config()
        cfg = _default_ns
    rows, cols = x.shape[-2:]
    count = 1
    for size in x.shape[:-2]:
        count *= size
    (xs, xld), (os_, old) = _batch(x, "x", rows, cols), _batch(out, "out", rows, cols)
    guard, stream = _on(x)
    with guard:
        need = neox_orthogonalize_workspace(count, rows, cols)
        work = torch.empty(need, dtype=torch.uint8, device=x.device)
        neox_orthogonalize(cfg, x.data_ptr(), _code(x.dtype), xld, xs, out.data_ptr(),
                           _code(out.dtype), old, os_, count, rows, cols, scale, work.data_ptr(),
                           need, stream)
    return out


class MXFP4:
    """A rows x cols matrix in MXFP4: codes (rows, K/2) and scales (rows, K/32), uint8, K
    being cols rounded up to a multiple of 128.  Copies that the operators make are one
    allocation; its two tensors are made when they are asked for."""

    __slots__ = ("rows", "cols", "device", "_memory", "_codes", "_scales", "_at")

    def __init__(self, codes, scales, rows: int, cols: int):
        import torch
        k = -(-cols // 128) * 128
        for t, width, name in ((codes, k // 2, "codes"), (scales, k // 32, "scales")):
            if not t.is_cuda or t.dtype != torch.uint8 or not t.is_contiguous() or \
                    tuple(t.shape) != (rows, width):
                raise ValueError(f"{name} must be a contiguous uint8 CUDA tensor of "
                                 f"({rows}, {width})")
        if codes.device != scales.device:
            raise ValueError("codes and scales are on different devices")
        self.rows, self.cols, self.device = rows, cols, codes.device
        self._codes, self._scales = codes, scales
        self._at = codes.data_ptr(), scales.data_ptr()

    @staticmethod
    def empty(rows: int, cols: int, device) -> "MXFP4":
        import torch
        k = -(-cols // 128) * 128
        q = object.__new__(MXFP4)          # right by construction: nothing to check
        q._memory = torch.empty(rows * (k // 2 + k // 32), dtype=torch.uint8, device=device)
        q.rows, q.cols, q.device = rows, cols, q._memory.device
        q._codes = q._scales = None
        at = q._memory.data_ptr()
        q._at = at, at + rows * (k // 2)
        return q

    @property
    def codes(self):
        if self._codes is None:
            k = -(-self.cols // 128) * 128
            self._codes = self._memory[:self.rows * (k // 2)].view(self.rows, k // 2)
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            k = -(-self.cols // 128) * 128
            self._scales = self._memory[self.rows * (k // 2):].view(self.rows, k // 32)
        return self._scales

    def __repr__(self):
        return f"MXFP4({self.rows} x {self.cols}, {self.device})"


def mxfp4_quantize(x, transpose: bool = False, out: MXFP4 | None = None) -> MXFP4:
    """The MXFP4 copy of matrix x, or of its transpose."""
    ld = _rows_of(x, "x")
    rows, cols = x.shape
    want = (cols, rows) if transpose else (rows, cols)
    if out is None:
        out = MXFP4.empty(*want, x.device)
    elif (out.rows, out.cols) != want or out.device != x.device:
        raise ValueError(f"out must be a {want[0]} x {want[1]} copy on x's device")
    guard, stream = _on(x)
    with guard:
        neox_mxfp4_quantize(x.data_ptr(), _code(x.dtype), rows, cols, ld, int(transpose),
                            *out._at, stream)
    return out


def mxfp4_dequantize(q: MXFP4, dtype=None, out=None):
    """The values of a copy, as a new matrix of type `dtype` (bfloat16 by default) or in out."""
    import torch
    if out is None:
        out, ld = torch.empty((q.rows, q.cols), dtype=dtype or torch.bfloat16, device=q.device), q.cols
    elif tuple(out.shape) != (q.rows, q.cols) or out.device != q.device or \
            (dtype is not None and out.dtype != dtype):
        raise ValueError("out must have the copy's shape and device, and the type asked for")
    else:
        ld = _rows_of(out, "out")
    guard, stream = _on(out)
    with guard:
        neox_mxfp4_dequantize(*q._at, q.rows, q.cols,
                              out.data_ptr(), _code(out.dtype), ld, stream)
    return out


def mxfp4_product(a: MXFP4, b: MXFP4, dtype=None, out=None):
    """a b^T of an m x k and an n x k copy, as an m x n matrix of type `dtype` (bfloat16 by
    default) or in out."""
    import torch
    if a.cols != b.cols or a.device != b.device:
        raise ValueError("a and b must have the same number of columns, on one device")
    if out is None:
        out, ld = torch.empty((a.rows, b.rows), dtype=dtype or torch.bfloat16, device=a.device), b.rows
    elif tuple(out.shape) != (a.rows, b.rows) or out.device != a.device or \
            (dtype is not None and out.dtype != dtype):
        raise ValueError("out must have the product's shape and device, and the type asked for")
    else:
        ld = _rows_of(out, "out")
    guard, stream = _on(out)
    with guard:
        neox_mxfp4_product(*a._at, a.rows, *b._at, b.rows, a.cols, out.data_ptr(),
                           _code(out.dtype), ld, stream)
    return out


def muon_matrix(grad, half, master, momentum, decay: bool, copy: MXFP4 | None = None,
                copy_t: MXFP4 | None = None) -> neox_muon_matrix:
    """neox_muon_matrix over four contiguous CUDA matrices of one shape on one device (no copies
    made).
    copy / copy_t: MXFP4 copies of the weights / of their transpose that each applied step
    rewrites."""
    import torch
    shape = tuple(grad.shape)
    for t, dt in ((grad, None), (half, None), (master, torch.float32), (momentum, torch.float32)):
        if not t.is_cuda or t.dim() != 2 or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError("arrays must be contiguous 2-D CUDA tensors of one shape")
        if t.device != grad.device:
            raise ValueError("the arrays must be on one device")
        if dt is not None and t.dtype != dt:
            raise ValueError("master / momentum must be float32")
    if grad.dtype not in (torch.float16, torch.bfloat16) or half.dtype != grad.dtype:
        raise ValueError("grad and half must share float16 or bfloat16")
    for q, want in ((copy, shape), (copy_t, shape[::-1])):
        if q is not None and (q.rows, q.cols) != want:
            raise ValueError(f"the copy must be {want[0]} x {want[1]}")
        if q is not None and q.device != grad.device:
            raise ValueError("the copies must be on the arrays' device")
    return neox_muon_matrix(grad.data_ptr(), half.data_ptr(), master.data_ptr(), momentum.data_ptr(),
                            shape[0], shape[1], Z.NEOX_SEG_DECAY if decay else 0, 0,
                            *((None, None) if copy is None else copy._at),
                            *((None, None) if copy_t is None else copy_t._at))


class Muon:
    """Owner of one step handle.  The tensors behind the matrices must outlive it."""

    def __init__(self, cfg: neox_zero1_config, mats, mcfg: neox_muon_config | None = None,
                 stream_ptr: int | None = None):
        self.handle = 0
        self._mats = list(mats)
        self.handle = neox_muon_create(cfg, neox_muon_default_config() if mcfg is None else mcfg,
                                       self._mats,
                                       Z.current_stream_ptr() if stream_ptr is None else stream_ptr)

    def step(self, lr: float, stream_ptr: int | None = None):
        neox_muon_step(self.handle, lr, Z.current_stream_ptr() if stream_ptr is None else stream_ptr)

    def state(self) -> neox_scaler_state_t:
        return neox_muon_state(self.handle)

    def close(self):
        if self.handle:
            h, self.handle = self.handle, 0
            neox_muon_destroy(h)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
