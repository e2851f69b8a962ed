"""The row operators of the library (include/rows.h): layer norm, dropout, rows
in 8 bits and the linear layer on them.

``conv_norm_*``, ``conv_dropout_*``, ``conv_quantize_rows`` and ``conv_int8_*``
keep the C names and only marshal arguments; ``layer_norm``,
``layer_norm_backward``, ``dropout``, ``dropout_backward``, ``quantize_rows`` and
``linear_int8`` take CUDA tensors and allocate outputs and scratch with torch."""
from __future__ import annotations

import ctypes
from operator import index as _whole

from . import DTYPES, _check, _dtype_name, _ptr, load
from .dense import (FLAG_LINEAR_RESIDUAL_LAST, LINEAR_ACTIVATIONS, _dense_out, _rows_dense, _run, _same, _scratch,
                    _stream_handle, _torch, _turn)

__all__ = [
    "NormProblem", "DropoutProblem", "QuantizeProblem", "Int8Problem", "FLAG_NORM_STREAM", "FLAG_INT8_FEW", "FLAG_INT8_MID",
    "FLAG_INT8_MANY", "make_norm_problem", "make_dropout_problem", "make_quantize_problem", "make_int8_problem",
    "conv_norm_forward", "conv_norm_backward_scratch_bytes", "conv_norm_backward", "conv_dropout_forward",
    "conv_dropout_backward", "conv_quantize_rows", "conv_int8_scratch_bytes", "conv_int8_describe_plan",
    "conv_int8_forward", "layer_norm", "layer_norm_backward", "dropout", "dropout_backward", "quantize_rows",
    "linear_int8",
]

FLAG_NORM_STREAM = 0x1
FLAG_INT8_FEW = 0x10
FLAG_INT8_MID = 0x20
FLAG_INT8_MANY = 0x40


class NormProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "width", "x_stride", "y_stride")] + [
        ("eps", ctypes.c_float), ("dtype", ctypes.c_int32), ("has_weight", ctypes.c_int32),
        ("has_bias", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class DropoutProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "width", "x_stride", "residual_stride", "y_stride")] + [
        ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64), ("p", ctypes.c_double), ("dtype", ctypes.c_int32),
        ("has_residual", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class QuantizeProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("rows", "width", "x_stride", "q_stride")] + [
        ("dtype", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class Int8Problem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "rows", "c_in", "c_out", "x_stride", "w_stride", "residual_stride", "y_stride")] + [
        ("act", ctypes.c_int32), ("act_alpha", ctypes.c_float), ("act_beta", ctypes.c_float),
        ("dtype", ctypes.c_int32), ("x_quantized", ctypes.c_int32), ("has_bias", ctypes.c_int32),
        ("has_residual", ctypes.c_int32), ("flags", ctypes.c_uint32)]


_lib = None


def _load() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        lib = load()
        P, vp, sz, i32 = ctypes.POINTER, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
        np, dp, qp, ip = P(NormProblem), P(DropoutProblem), P(QuantizeProblem), P(Int8Problem)
        for name, args in {
            "conv_norm_forward": [np] + [vp] * 6,
            "conv_norm_backward_scratch_bytes": [np, P(sz)],
            "conv_norm_backward": [np] + [vp] * 8 + [sz, vp],
            "conv_dropout_forward": [dp] + [vp] * 5,
            "conv_dropout_backward": [dp] + [vp] * 4,
            "conv_quantize_rows": [qp] + [vp] * 4,
            "conv_int8_scratch_bytes": [ip, P(sz)],
            "conv_int8_describe_plan": [ip, i32, ctypes.c_char_p, sz],
            "conv_int8_forward": [ip] + [vp] * 8 + [sz, vp],
        }.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        _lib = lib
    return _lib


def make_norm_problem(rows, width, *, dtype="f32", x_stride=0, y_stride=0, eps=1e-5, has_weight=True, has_bias=True,
                      flags=0) -> NormProblem:
    return NormProblem(int(rows), int(width), int(x_stride), int(y_stride), float(eps), DTYPES[dtype],
                       1 if has_weight else 0, 1 if has_bias else 0, int(flags))


def make_dropout_problem(rows, width, p, seed, offset=0, *, dtype="f32", x_stride=0, residual_stride=0, y_stride=0,
                         has_residual=False, flags=0) -> DropoutProblem:
    return DropoutProblem(int(rows), int(width), int(x_stride), int(residual_stride), int(y_stride), int(seed),
                          int(offset), float(p), DTYPES[dtype], 1 if has_residual else 0, int(flags))


def make_quantize_problem(rows, width, *, dtype="f32", x_stride=0, q_stride=0, flags=0) -> QuantizeProblem:
    return QuantizeProblem(int(rows), int(width), int(x_stride), int(q_stride), DTYPES[dtype], int(flags))


def make_int8_problem(rows, c_in, c_out, *, dtype="f32", x_quantized=True, x_stride=0, w_stride=0, residual_stride=0,
                      y_stride=0, act="identity", alpha=0.0, beta=0.0, has_bias=False, has_residual=False,
                      flags=0) -> Int8Problem:
    return Int8Problem(int(rows), int(c_in), int(c_out), int(x_stride), int(w_stride), int(residual_stride),
                       int(y_stride), LINEAR_ACTIVATIONS[act], float(alpha), float(beta), DTYPES[dtype],
                       1 if x_quantized else 0, 1 if has_bias else 0, 1 if has_residual else 0, int(flags))


# ---- the C functions, same names --------------------------------------------
def _call(name, p, *args) -> None:
    _check(getattr(_load(), name)(ctypes.byref(p), *args), name)


def _bytes(name, p) -> int:
    n = ctypes.c_size_t()
    _call(name, p, ctypes.byref(n))
    return n.value


def conv_norm_forward(p: NormProblem, x, weight, bias, y, stats=None, stream=None) -> None:
    _call("conv_norm_forward", p, _ptr(x), _ptr(weight), _ptr(bias), _ptr(y), _ptr(stats), _stream_handle(stream))


def conv_norm_backward_scratch_bytes(p: NormProblem) -> int:
    return _bytes("conv_norm_backward_scratch_bytes", p)


def conv_norm_backward(p: NormProblem, x, weight, stats, dy, dx, dweight, dbias, scratch=None, scratch_bytes: int = 0,
                       stream=None) -> None:
    _call("conv_norm_backward", p, _ptr(x), _ptr(weight), _ptr(stats), _ptr(dy), _ptr(dx), _ptr(dweight), _ptr(dbias),
          _ptr(scratch), scratch_bytes, _stream_handle(stream))


def conv_dropout_forward(p: DropoutProblem, x, residual, y, state=None, stream=None) -> None:
    _call("conv_dropout_forward", p, _ptr(x), _ptr(residual), _ptr(y), _ptr(state), _stream_handle(stream))


def conv_dropout_backward(p: DropoutProblem, dy, dx, state=None, stream=None) -> None:
    _call("conv_dropout_backward", p, _ptr(dy), _ptr(dx), _ptr(state), _stream_handle(stream))


def conv_quantize_rows(p: QuantizeProblem, x, q, scale, stream=None) -> None:
    _call("conv_quantize_rows", p, _ptr(x), _ptr(q), _ptr(scale), _stream_handle(stream))


def conv_int8_scratch_bytes(p: Int8Problem) -> int:
    return _bytes("conv_int8_scratch_bytes", p)


def conv_int8_describe_plan(p: Int8Problem, sm_count: int) -> str:
    buf = ctypes.create_string_buffer(512)
    _call("conv_int8_describe_plan", p, int(sm_count), buf, len(buf))
    return buf.value.decode()


def conv_int8_forward(p: Int8Problem, x, x_scale, w, w_scale, bias, residual, y, scratch=None, scratch_bytes: int = 0,
                      stream=None) -> None:
    _call("conv_int8_forward", p, _ptr(x), _ptr(x_scale), _ptr(w), _ptr(w_scale), _ptr(bias), _ptr(residual), _ptr(y),
          _ptr(scratch), scratch_bytes, _stream_handle(stream))


# ---- conveniences -----------------------------------------------------------
# What the checks of a call's operands gave, by the operands' shapes, types and devices: a call like one before, on dense
# operands, checks and marshals nothing anew.  (Scratch sizes go by the device's SM count, so by the device.)
_seen: dict = {}


def _remember(key, found):
    if len(_seen) >= 4096:
        _seen.clear()
    _seen[key] = found
    return found


def _tag(t):
    """What _seen goes by for an operand."""
    return t.shape, t.dtype, t.get_device(), t.is_contiguous()


def _dense_key(key, tensors):
    """key if every operand is dense, else None: strides are no part of it."""
    return key if all(t is None or t.is_contiguous() for t in tensors) else None


def _vector(t, width, what):
    if t is not None and (t.dim() != 1 or t.shape[0] != width or not t.is_contiguous()):
        raise ValueError(f"{what} must be a contiguous [{width}]")


def _like(t, x, what):
    """t's row stride; ValueError unless it has x's shape."""
    if t.shape != x.shape:
        raise ValueError(f"{what} must have x's shape")
    return _rows_dense(t, x.shape[-1], what)[1]


def _width(x, what="x"):
    if x.dim() == 0:
        raise ValueError(f"{what} must be [..., width]")
    return x.shape[-1]


def _empty(shape, like, dtype=None):
    # (a device's number in place of the device takes 3 us more)
    return torch.empty(shape, dtype=dtype or like.dtype, device=like.device)


def _with_scratch(call, args, need, scratch, index, handle):
    if need == 0 and scratch is None:
        return call(*args, None, 0, handle or None)
    with _turn(need, scratch, index, handle):
        _, at, n = _scratch(need, scratch, index, handle)
        return call(*args, at, n, handle or None)


torch = None  # imported by the first call that takes tensors


def _begin():
    global torch
    if torch is None:
        torch = _torch()


def _norm_plan(x, weight, bias, out, eps, flags):
    dt = DTYPES[_dtype_name(x)]
    index = _same(x, (weight, bias, out))
    width = _width(x)
    rows, ldx = _rows_dense(x, width, "x")
    _vector(weight, width, "weight")
    _vector(bias, width, "bias")
    ldy = 0 if out is None else _like(out, x, "out")
    p = NormProblem(rows, width, ldx, ldy, eps, dt, 0 if weight is None else 1, 0 if bias is None else 1, flags)
    return ctypes.byref(p), index, (*x.shape[:-1], 2)


def layer_norm(x, weight=None, bias=None, *, eps=1e-5, save=False, out=None, flags=0, stream=None):
    """y = (x - mean) / sqrt(var + eps) * weight + bias over the last dimension
    of a CUDA tensor x [..., width]; weight and bias [width], or None, of x's
    element type.  Rows may be strided.  With ``save``, returns (y, stats): stats
    is float32 [..., 2], the mean and 1 / sqrt(var + eps) of each row, for
    ``layer_norm_backward``."""
    key = ("norm", x.shape, x.dtype, x.get_device(), x.is_contiguous(), weight if weight is None else _tag(weight),
           bias if bias is None else _tag(bias), out if out is None else _tag(out), eps, flags)
    found = _seen.get(key)
    if found is None:
        _begin()
        found = _norm_plan(x, weight, bias, out, eps, flags)
        if _dense_key(key, (x, weight, bias, out)):
            _remember(key, found)
    return _run(_norm_call, found[1], stream, found, x, weight, bias, save, out)


def _norm_call(handle, found, x, weight, bias, save, out):
    ref, index, stats_shape = found
    if out is None:
        out = _empty(x.shape, x)
    stats = _empty(stats_shape, x, torch.float32) if save else None
    status = _load().conv_norm_forward(ref, x.data_ptr(), _ptr(weight), _ptr(bias), out.data_ptr(), _ptr(stats), handle or None)
    if status:
        _check(status, "conv_norm_forward")
    return (out, stats) if save else out


def _norm_back_plan(dy, x, weight, stats, dx, flags):
    dt = DTYPES[_dtype_name(x)]
    index = _same(x, (weight, dy))
    width = _width(x)
    rows, ldx = _rows_dense(x, width, "x")
    ldy = _like(dy, x, "dy")
    _vector(weight, width, "weight")
    if stats.shape != (*x.shape[:-1], 2) or stats.dtype != torch.float32 or stats.get_device() != index or \
            not stats.is_contiguous():
        raise ValueError("stats must be what layer_norm(..., save=True) returned for x")
    if dx is not None:
        _dense_out(dx, x.shape, x, "dx")
    # (eps plays no part: the statistics have it)
    p = NormProblem(rows, width, ldx, ldy, 0.0, dt, 0 if weight is None else 1, 0, flags)
    with torch.cuda.device(index):
        need = conv_norm_backward_scratch_bytes(p)
    return ctypes.byref(p), index, need, (width,)


def layer_norm_backward(dy, x, weight, stats, *, need_dx=True, need_dweight=True, need_dbias=True, dx=None, scratch=None,
                        flags=0, stream=None):
    """The gradients of ``layer_norm`` for dy [..., width]: (dx, dweight, dbias),
    None where not wanted.  ``stats`` is what layer_norm(..., save=True) returned;
    weight is that call's (None: none)."""
    key = ("norm back", x.shape, x.dtype, x.get_device(), x.is_contiguous(), _tag(dy),
           weight if weight is None else _tag(weight), _tag(stats), dx if dx is None else _tag(dx), flags)
    found = _seen.get(key)
    if found is None:
        _begin()
        found = _norm_back_plan(dy, x, weight, stats, dx, flags)
        if _dense_key(key, (dy, x, weight, stats, dx)):
            _remember(key, found)
    return _run(_norm_back_call, found[1], stream, found, dy, x, weight, stats, need_dx, need_dweight, need_dbias, dx, scratch)


def _norm_back_call(handle, found, dy, x, weight, stats, need_dx, need_dweight, need_dbias, dx, scratch):
    ref, index, need, vector = found
    if not need_dx:
        dx = None
    elif dx is None:
        dx = _empty(x.shape, x)
    dw = _empty(vector, x) if need_dweight else None  # (two allocations are quicker than the halves of one)
    db = _empty(vector, x) if need_dbias else None
    if dw is None and db is None:
        need = 0
    args = (ref, x.data_ptr(), _ptr(weight), stats.data_ptr(), dy.data_ptr(), _ptr(dx), _ptr(dw), _ptr(db))
    status = _with_scratch(_load().conv_norm_backward, args, need, scratch, index, handle)
    if status:
        _check(status, "conv_norm_backward")
    return dx, dw, db


_WORD = (1 << 64) - 1


def _dropout_plan(x, residual, out, seed):
    dt = DTYPES[_dtype_name(x)]
    index = _same(x, (residual, out))
    width = _width(x)
    rows, ldx = _rows_dense(x, width, "x")
    ldr = 0 if residual is None else _like(residual, x, "residual")
    ldy = 0 if out is None else _like(out, x, "out")
    if hasattr(seed, "data_ptr") and (seed.dtype != torch.int64 or seed.numel() != 2 or not seed.is_contiguous() or
                                      seed.get_device() != index):
        raise ValueError("seed must be an int or a contiguous int64 tensor of a seed and an offset on x's device")
    return index, rows, width, ldx, ldr, ldy, dt


def _dropout(back, x, p, seed, offset, residual, out, stream):
    state = hasattr(seed, "data_ptr")
    offset = _whole(offset)  # (numpy's whole numbers refuse 64-bit masks)
    if not state:
        seed = _whole(seed)
    key = ("dropout", x.shape, x.dtype, x.get_device(), x.is_contiguous(),
           residual if residual is None else _tag(residual), out if out is None else _tag(out), _tag(seed) if state else None)
    found = _seen.get(key)
    if found is None:
        _begin()
        found = _dropout_plan(x, residual, out, seed)
        if _dense_key(key, (x, residual, out)):
            _remember(key, found)
    if not -1 << 63 <= offset <= _WORD or not (state or -1 << 63 <= seed <= _WORD):
        raise ValueError("seed and offset must fit 64 bits")
    return _run(_dropout_call, found[0], stream, found, back, x, p, seed, offset, residual, out, state)


def _dropout_call(handle, found, back, x, p, seed, offset, residual, out, state):
    index, rows, width, ldx, ldr, ldy, dt = found
    if out is None:
        out = _empty(x.shape, x)
    if back:
        ldx, ldy = ldy, ldx  # the C function's strides are those of the forward call's x and y
    # (a problem of its own: the offset is another one at every call)
    q = ctypes.byref(DropoutProblem(rows, width, ldx, ldr, ldy, 0 if state else seed & _WORD, offset & _WORD, p, dt,
                                    0 if residual is None else 1, 0))
    at = seed.data_ptr() if state else None
    if back:
        status = _load().conv_dropout_backward(q, x.data_ptr(), out.data_ptr(), at, handle or None)
    else:
        status = _load().conv_dropout_forward(q, x.data_ptr(), _ptr(residual), out.data_ptr(), at, handle or None)
    if status:
        _check(status, "conv_dropout_backward" if back else "conv_dropout_forward")
    return out


def dropout(x, p, seed, offset=0, *, residual=None, out=None, stream=None):
    """y = residual + (x / (1 - p) where kept, else 0) on a CUDA tensor x
    [..., width], each value dropped with probability p (to 2^-16; the scale is
    that of the p taken).  Which ones is a function of seed, offset and the place
    (row, column) alone: ``dropout_backward`` with the same ones drops the same
    values, and nothing is stored.  Calls that are to draw apart take different
    offsets.  ``seed`` may be an int64 CUDA tensor [seed, offset], read when the
    kernel runs (its offset is added to ``offset``): a captured graph then draws
    anew when it changes."""
    return _dropout(False, x, p, seed, offset, residual, out, stream)


def dropout_backward(dy, p, seed, offset=0, *, out=None, stream=None):
    """The gradient of ``dropout`` for dy [..., width]: dy / (1 - p) where that
    call kept the value, else 0.  The residual's gradient is dy."""
    return _dropout(True, dy, p, seed, offset, None, out, stream)


def _quantize_plan(x):
    dt = DTYPES[_dtype_name(x)]
    index = _same(x, ())
    width = _width(x)
    rows, ldx = _rows_dense(x, width, "x")
    return ctypes.byref(QuantizeProblem(rows, width, ldx, 0, dt, 0)), index, x.shape[:-1]


def quantize_rows(x, *, stream=None):
    """(q, scale) of a CUDA tensor x [..., width]: scale [...] float32 is a row's
    largest absolute value * (1 / 127), q [..., width] int8 the rows divided by it,
    rounded to nearest even.  For the rows of activations, and of weights."""
    key = "quantize", x.shape, x.dtype, x.get_device(), x.is_contiguous()
    found = _seen.get(key)
    if found is None:
        _begin()
        found = _quantize_plan(x)
        if _dense_key(key, (x,)):
            _remember(key, found)
    return _run(_quantize_call, found[1], stream, found, x)


def _quantize_call(handle, found, x):
    ref, index, lead = found
    q = _empty(x.shape, x, torch.int8)
    scale = _empty(lead, x, torch.float32)
    status = _load().conv_quantize_rows(ref, x.data_ptr(), q.data_ptr(), scale.data_ptr(), handle or None)
    if status:
        _check(status, "conv_quantize_rows")
    return q, scale


def _int8_plan(x, w, w_scale, bias, residual, x_scale, dtype, act, alpha, beta, residual_last, out, flags):
    if w.dim() != 2 or w.dtype != torch.int8:
        raise ValueError("w must be int8 [c_out, c_in]")
    c_out, c_in = w.shape
    index = x.get_device()
    quantized = x.dtype == torch.int8
    if quantized:
        if x_scale is None or dtype is None:
            raise ValueError("an int8 x needs x_scale and dtype")
        if x_scale.shape != x.shape[:-1] or not x_scale.is_contiguous():
            raise ValueError("x_scale must be contiguous and have x's leading dimensions")
    elif x_scale is not None or dtype not in (None, x.dtype):
        raise ValueError("x_scale and dtype are for an int8 x")
    else:
        dtype = x.dtype
    _same(w, (x,) if quantized else ())
    _same(w_scale, (x_scale,))
    if w_scale.dtype != torch.float32 or w.get_device() != index or w_scale.get_device() != index:
        raise ValueError("scales must be float32 and operands share x's device")
    for t in (bias, residual, out):
        if t is not None and (t.dtype != dtype or t.get_device() != index):
            raise ValueError("bias, residual and out must have y's element type and x's device")
    dt = DTYPES.get({torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}.get(dtype))
    if dt is None:
        raise TypeError(f"unsupported element type {dtype}")
    rows, ldx = _rows_dense(x, c_in, "x")
    ldw = _rows_dense(w, c_in, "w")[1]
    _vector(w_scale, c_out, "w_scale")
    _vector(bias, c_out, "bias")
    y_shape = (*x.shape[:-1], c_out)
    ldr = ldy = 0
    if residual is not None:
        if residual.shape != y_shape:
            raise ValueError("residual must have y's shape")
        ldr = _rows_dense(residual, c_out, "residual")[1]
    if out is not None:
        if out.shape != y_shape:
            raise ValueError("out must have y's shape")
        ldy = _rows_dense(out, c_out, "out")[1]
    if residual_last:
        flags |= FLAG_LINEAR_RESIDUAL_LAST
    p = Int8Problem(rows, c_in, c_out, ldx, ldw, ldr, ldy, LINEAR_ACTIVATIONS[act], alpha, beta, dt, 1 if quantized else 0,
                    0 if bias is None else 1, 0 if residual is None else 1, flags)
    with torch.cuda.device(index):
        need = conv_int8_scratch_bytes(p)
    return ctypes.byref(p), index, need, y_shape, dtype


def linear_int8(x, w, w_scale, bias=None, residual=None, *, x_scale=None, dtype=None, act="identity", alpha=0.0, beta=0.0,
                residual_last=False, out=None, scratch=None, flags=0, stream=None):
    """y = act((q w^T) * x_scale * w_scale + bias + residual) on CUDA tensors: w
    [c_out, c_in] int8 and w_scale [c_out] float32 as ``quantize_rows`` gives them
    for a weight matrix; x [..., c_in] either of an element type, its rows
    quantised by the call, or int8 with its x_scale [...] float32.  bias [c_out],
    residual and y [..., c_out] have x's element type, or ``dtype`` for an int8 x.
    The integer sums are exact.  Activations and ``residual_last`` as in
    ``linear``.  Half the weights' memory; quicker than ``linear`` for up to some
    16 rows, as quick for some tens in a wide layer, slower from some hundreds on
    (2048 rows of 4096 -> 4096 60 us beside 40)."""
    key = ("int8", x.shape, x.dtype, x.get_device(), x.is_contiguous(), _tag(w), _tag(w_scale),
           bias if bias is None else _tag(bias), residual if residual is None else _tag(residual),
           x_scale if x_scale is None else _tag(x_scale), dtype, act, alpha, beta, residual_last,
           out if out is None else _tag(out), flags)
    found = _seen.get(key)
    if found is None:
        _begin()
        found = _int8_plan(x, w, w_scale, bias, residual, x_scale, dtype, act, alpha, beta, residual_last, out, flags)
        if _dense_key(key, (x, w, w_scale, bias, residual, x_scale, out)):
            _remember(key, found)
    return _run(_int8_call, found[1], stream, found, x, w, w_scale, bias, residual, x_scale, out, scratch)


def _int8_call(handle, found, x, w, w_scale, bias, residual, x_scale, out, scratch):
    ref, index, need, y_shape, dtype = found
    if out is None:
        out = _empty(y_shape, x, dtype)
    args = (ref, x.data_ptr(), _ptr(x_scale), w.data_ptr(), w_scale.data_ptr(), _ptr(bias), _ptr(residual), out.data_ptr())
    status = _with_scratch(_load().conv_int8_forward, args, need, scratch, index, handle)
    if status:
        _check(status, "conv_int8_forward")
    return out
