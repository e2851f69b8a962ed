"""The dense operators of the library (include/linear.h): the linear layer, the
gated feed-forward block and the clipping of gradients by their global norm.

``conv_linear_*``, ``conv_gated_*`` and ``conv_clip_*`` keep the C names and
only marshal arguments; ``linear``, ``linear_backward``, ``gated_ffn``,
``gated_ffn_backward`` and ``clip_grad_norm`` take CUDA tensors and allocate
outputs and scratch with torch."""
from __future__ import annotations

import contextlib
import ctypes
import threading
from array import array

from . import ACTIVATIONS, DTYPES, _check, _dtype_name, _ptr, load

__all__ = [
    "LinearProblem", "GatedProblem", "LINEAR_ACTIVATIONS", "FLAG_LINEAR_RESIDUAL_LAST", "FLAG_LINEAR_UNALIGNED",
    "FLAG_LINEAR_FORCE_FFMA", "FLAG_LINEAR_NO_FEW_ROWS", "make_linear_problem", "make_gated_problem",
    "conv_linear_scratch_bytes", "conv_linear_backward_scratch_bytes", "conv_linear_describe_plan",
    "conv_linear_forward", "conv_linear_backward", "conv_gated_scratch_bytes", "conv_gated_backward_scratch_bytes",
    "conv_gated_saved_bytes", "conv_gated_forward", "conv_gated_backward", "conv_clip_scratch_bytes",
    "conv_clip_grads", "conv_linear_device_error", "linear", "linear_backward", "gated_ffn", "gated_ffn_backward",
    "clip_grad_norm",
]

LINEAR_ACTIVATIONS = dict(ACTIVATIONS, gelu=9, gelu_tanh=10)
FLAG_LINEAR_RESIDUAL_LAST = 0x1
FLAG_LINEAR_UNALIGNED = 0x2
FLAG_LINEAR_FORCE_FFMA = 0x4
FLAG_LINEAR_NO_FEW_ROWS = 0x8


class LinearProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "rows", "c_in", "c_out", "x_stride", "w_stride", "residual_stride", "y_stride")] + [
        ("act", ctypes.c_int32), ("act_alpha", ctypes.c_float), ("act_beta", ctypes.c_float),
        ("dtype", ctypes.c_int32), ("has_bias", ctypes.c_int32), ("has_residual", ctypes.c_int32),
        ("flags", ctypes.c_uint32)]


class GatedProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "rows", "c_in", "hidden", "c_out", "x_stride", "residual_stride", "y_stride")] + [
        ("act", ctypes.c_int32), ("act_alpha", ctypes.c_float), ("act_beta", ctypes.c_float),
        ("dtype", ctypes.c_int32), ("has_residual", ctypes.c_int32), ("flags", ctypes.c_uint32)]


torch = None  # imported by the first call that takes tensors


def _torch():
    global torch
    import torch as module
    torch = module
    return module


_lib = None


def _load() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        lib = load()
        P, vp, sz = ctypes.POINTER, ctypes.c_void_p, ctypes.c_size_t
        i64, i32, f = ctypes.c_int64, ctypes.c_int32, ctypes.c_float
        lp, gp = P(LinearProblem), P(GatedProblem)
        for name, args in {
            "conv_linear_scratch_bytes": [lp, P(sz)],
            "conv_linear_backward_scratch_bytes": [lp, P(sz)],
            "conv_linear_describe_plan": [lp, i32, i32, ctypes.c_char_p, sz],
            "conv_linear_forward": [lp] + [vp] * 7 + [sz, vp],
            "conv_linear_backward": [lp] + [vp] * 9 + [sz, vp],
            "conv_gated_scratch_bytes": [gp, P(sz)],
            "conv_gated_backward_scratch_bytes": [gp, P(sz)],
            "conv_gated_saved_bytes": [gp, P(sz)],
            "conv_gated_forward": [gp] + [vp] * 8 + [sz, vp],
            "conv_gated_backward": [gp] + [vp] * 11 + [sz, vp],
            "conv_clip_scratch_bytes": [i64, vp, P(sz)],
            "conv_clip_grads": [i64, vp, vp, vp, vp, f, f, vp, vp, sz, vp],
            "conv_linear_device_error": [P(ctypes.c_uint32), i32],
        }.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        _lib = lib
    return _lib


def make_linear_problem(rows, c_in, c_out, *, dtype="f32", x_stride=0, w_stride=0, residual_stride=0, y_stride=0,
                        act="identity", alpha=0.0, beta=0.0, has_bias=False, has_residual=False,
                        flags=0) -> LinearProblem:
    return LinearProblem(int(rows), int(c_in), int(c_out), int(x_stride), int(w_stride), int(residual_stride),
                         int(y_stride), LINEAR_ACTIVATIONS[act], float(alpha), float(beta), DTYPES[dtype],
                         1 if has_bias else 0, 1 if has_residual else 0, int(flags))


def make_gated_problem(rows, c_in, hidden, c_out, *, dtype="f32", x_stride=0, residual_stride=0, y_stride=0,
                       act="silu", alpha=0.0, beta=0.0, has_residual=False, flags=0) -> GatedProblem:
    return GatedProblem(int(rows), int(c_in), int(hidden), int(c_out), int(x_stride), int(residual_stride),
                        int(y_stride), LINEAR_ACTIVATIONS[act], float(alpha), float(beta), DTYPES[dtype],
                        1 if has_residual else 0, int(flags))


# ---- the C functions, same names --------------------------------------------
def _stream_handle(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream or None
    return (stream.cuda_stream if hasattr(stream, "cuda_stream") else stream) or None


def _bytes(name, p) -> int:
    n = ctypes.c_size_t()
    _check(getattr(_load(), name)(ctypes.byref(p), ctypes.byref(n)), name)
    return n.value


def conv_linear_scratch_bytes(p: LinearProblem) -> int:
    return _bytes("conv_linear_scratch_bytes", p)


def conv_linear_backward_scratch_bytes(p: LinearProblem) -> int:
    return _bytes("conv_linear_backward_scratch_bytes", p)


def conv_linear_describe_plan(p: LinearProblem, which: int, sm_count: int) -> str:
    buf = ctypes.create_string_buffer(512)
    _check(_load().conv_linear_describe_plan(ctypes.byref(p), int(which), int(sm_count), buf, len(buf)),
           "conv_linear_describe_plan")
    return buf.value.decode()


def conv_linear_forward(p: LinearProblem, x, w, bias, residual, y, pre=None, scratch=None, scratch_bytes: int = 0,
                        stream=None) -> None:
    _check(_load().conv_linear_forward(ctypes.byref(p), _ptr(x), _ptr(w), _ptr(bias), _ptr(residual), _ptr(y),
                                       _ptr(pre), _ptr(scratch), scratch_bytes, _stream_handle(stream)),
           "conv_linear_forward")


def conv_linear_backward(p: LinearProblem, x, w, pre, dy, dx, dw, dbias, dresidual, scratch=None,
                         scratch_bytes: int = 0, stream=None) -> None:
    _check(_load().conv_linear_backward(ctypes.byref(p), _ptr(x), _ptr(w), _ptr(pre), _ptr(dy), _ptr(dx), _ptr(dw),
                                        _ptr(dbias), _ptr(dresidual), _ptr(scratch), scratch_bytes,
                                        _stream_handle(stream)), "conv_linear_backward")


def conv_gated_scratch_bytes(p: GatedProblem) -> int:
    return _bytes("conv_gated_scratch_bytes", p)


def conv_gated_backward_scratch_bytes(p: GatedProblem) -> int:
    return _bytes("conv_gated_backward_scratch_bytes", p)


def conv_gated_saved_bytes(p: GatedProblem) -> int:
    return _bytes("conv_gated_saved_bytes", p)


def conv_gated_forward(p: GatedProblem, x, w_gate, w_up, w_down, residual, y, saved=None, scratch=None,
                       scratch_bytes: int = 0, stream=None) -> None:
    _check(_load().conv_gated_forward(ctypes.byref(p), _ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(w_down),
                                      _ptr(residual), _ptr(y), _ptr(saved), _ptr(scratch), scratch_bytes,
                                      _stream_handle(stream)), "conv_gated_forward")


def conv_gated_backward(p: GatedProblem, x, w_gate, w_up, w_down, saved, dy, dx, dw_gate, dw_up, dw_down,
                        scratch=None, scratch_bytes: int = 0, stream=None) -> None:
    _check(_load().conv_gated_backward(ctypes.byref(p), _ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(saved),
                                       _ptr(dy), _ptr(dx), _ptr(dw_gate), _ptr(dw_up), _ptr(dw_down), _ptr(scratch),
                                       scratch_bytes, _stream_handle(stream)), "conv_gated_backward")


def conv_clip_scratch_bytes(sizes) -> int:
    n = ctypes.c_size_t()
    sizes = (ctypes.c_int64 * len(sizes))(*sizes)
    _check(_load().conv_clip_scratch_bytes(len(sizes), sizes, ctypes.byref(n)), "conv_clip_scratch_bytes")
    return n.value


def conv_clip_grads(inputs, outputs, sizes, dtypes, max_norm, eps, norm, scratch=None, scratch_bytes: int = 0,
                    stream=None) -> None:
    """``inputs`` / ``outputs`` (or None: the norm alone) are tensors or device
    addresses, ``sizes`` their element counts, ``dtypes`` names of DTYPES."""
    n = len(inputs)
    vps = ctypes.c_void_p * n
    _check(_load().conv_clip_grads(
        n, vps(*[_ptr(t) for t in inputs]), None if outputs is None else vps(*[_ptr(t) for t in outputs]),
        (ctypes.c_int64 * n)(*sizes), (ctypes.c_int32 * n)(*[DTYPES[d] for d in dtypes]), float(max_norm), float(eps),
        _ptr(norm), _ptr(scratch), scratch_bytes, _stream_handle(stream)), "conv_clip_grads")


def conv_linear_device_error(reset: bool = True) -> int:
    word = ctypes.c_uint32()
    _check(_load().conv_linear_device_error(ctypes.byref(word), 1 if reset else 0), "conv_linear_device_error")
    return word.value


# ---- conveniences -----------------------------------------------------------
def _rows(t, width, what):
    """(rows, row stride) of a tensor [..., width] whose rows are evenly spaced
    and whose elements of a row are adjacent; ValueError for any other."""
    shape, strides = t.shape, t.stride()
    n = len(shape)
    if n == 0 or shape[-1] != width:
        raise ValueError(f"{what} must be [..., {width}], not {tuple(shape)}")
    if width > 1 and strides[-1] != 1 and t.numel():
        raise ValueError(f"{what}: the elements of a row must be adjacent")
    if n == 2 and strides[0] >= width:
        rows, stride = shape[0], strides[0]
        return rows, stride if rows > 1 else 0
    if 0 in shape[:-1]:
        return 0, 0  # (the strides of an empty tensor say nothing)
    rows, stride = 1, None
    for i in range(n - 2, -1, -1):
        if shape[i] == 1:
            continue
        if stride is None:  # (0 is a stride: a broadcast dimension, whose rows are one row)
            stride = strides[i]
        elif strides[i] != stride * rows:
            raise ValueError(f"{what}: rows must be evenly spaced")
        rows *= shape[i]
    if rows > 1 and stride < width:
        raise ValueError(f"{what}: rows must not overlap")
    return rows, stride if rows > 1 else 0


def _rows_dense(t, width, what):
    """_rows, quicker for the dense tensors that most calls have."""
    if width and t.is_contiguous() and t.dim() and t.shape[-1] == width:  # (width 0: the C function refuses it)
        return t.numel() // width, 0
    return _rows(t, width, what)


def _same(x, others):
    """The operands' device number; ValueError unless they share x's type and device."""
    dtype, index = x.dtype, x.get_device()
    for t in others:
        if t is not None and (t.dtype != dtype or t.get_device() != index):
            raise ValueError("operands must share x's element type and device")
    if index < 0:
        raise ValueError("operands must be CUDA tensors")
    return index


class _On:
    """A call on another stream than the current one, or another device.  Memory
    that torch allocates for the call belongs to that stream, so that it is not
    handed out again while the call's kernels still run."""

    __slots__ = ("handle", "ctx")

    def __init__(self, index, stream):
        if stream is None:
            self.ctx = torch.cuda.device(index)
            self.handle = torch.cuda.current_stream(index).cuda_stream
        else:
            if hasattr(stream, "cuda_stream"):
                s = stream
            elif int(stream) == 0:  # the legacy default stream (torch takes the address 0 for a stream of its pool)
                s = torch.cuda.default_stream(index)
            else:
                s = torch.cuda.ExternalStream(int(stream), device=index)
            self.ctx = torch.cuda.stream(s)
            self.handle = s.cuda_stream

    def __enter__(self):
        self.ctx.__enter__()
        return self.handle

    def __exit__(self, *exc):
        self.ctx.__exit__(*exc)


_raw_stream = _device = None


def _run(call, index, stream, *args):
    """call(handle, *args) on the call's stream, with that stream and the operands' device current."""
    global _raw_stream, _device
    if _raw_stream is None:
        _torch()
        _device = torch.cuda.current_device
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda i: torch.cuda.current_stream(i).cuda_stream)
    if stream is None and index == _device():
        return call(_raw_stream(index), *args)
    with _On(index, stream) as handle:
        return call(handle, *args)


# Problems and their scratch sizes by device (plans go by its SM count) and shape, so that a call of a shape seen before
# marshals nothing anew.
_linear_cache: dict = {}
_gated_cache: dict = {}


def _linear_problem(index, back, *key):
    found = _linear_cache.get((index, back, key))
    if found is None:
        p = LinearProblem(*key)
        need = (conv_linear_backward_scratch_bytes if back else conv_linear_scratch_bytes)(p)
        if len(_linear_cache) >= 4096:
            _linear_cache.clear()
        found = _linear_cache[(index, back, key)] = (p, ctypes.byref(p), need)
    return found


def _gated_problem(index, back, *key):
    found = _gated_cache.get((index, back, key))
    if found is None:
        p = GatedProblem(*key)
        need = (conv_gated_backward_scratch_bytes if back else conv_gated_scratch_bytes)(p)
        if len(_gated_cache) >= 4096:
            _gated_cache.clear()
        found = _gated_cache[(index, back, key)] = (p, ctypes.byref(p), need, conv_gated_saved_bytes(p))
    return found


# Scratch of up to _KEPT bytes is kept per stream: the calls of a stream run one after another, and an allocation from
# torch's pool takes longer than a small call's own work.  A larger one, and one under graph capture (whose memory belongs to
# the graph), is the call's own.
_KEPT = 32 << 20
_kept: dict = {}
_turns: dict = {}
_no_turn = contextlib.nullcontext()


def _turn(need, given, index, handle):
    """Held from the choice of the scratch to the call's last launch: host threads that share a stream take turns at its
    kept scratch.  Streams have a turn each (a launch waits where a stream's queue is full), and a call whose scratch is
    its own, or the caller's, waits for nobody."""
    if need == 0 or given is not None or need > _KEPT:
        return _no_turn
    turn = _turns.get((index, handle))
    return turn if turn is not None else _turns.setdefault((index, handle), threading.RLock())


def _scratch(need, given, index, handle):
    """(tensor or None, its address, bytes); runs under the call's stream."""
    if given is not None:
        return given, given.data_ptr(), given.numel() * given.element_size()
    if need == 0:
        return None, None, 0
    if need > _KEPT or torch.cuda.is_current_stream_capturing():
        t = torch.empty(need, dtype=torch.uint8, device=index)
        return t, t.data_ptr(), need
    t, at, size = _kept.get((index, handle), (None, 0, 0))
    if size < need:
        size = max(need, 1 << 20)
        t = torch.empty(size, dtype=torch.uint8, device=index)
        at = t.data_ptr()
        if len(_kept) >= 64:
            _kept.clear()
        _kept[(index, handle)] = (t, at, size)
    return t, at, size


def _dense_out(out, shape, like, what):
    if out is None:
        return torch.empty(shape, dtype=like.dtype, device=like.device)
    if tuple(out.shape) != tuple(shape) or out.dtype != like.dtype or out.device != like.device or \
            not out.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {tuple(shape)} tensor of x's element type and device")
    return out


def linear(x, w, bias=None, residual=None, *, act="identity", alpha=0.0, beta=0.0, residual_last=False, save=False,
           out=None, scratch=None, flags=0, stream=None):
    """y = act(x w^T + bias + residual) on CUDA tensors: x [..., c_in], w
    [c_out, c_in], bias [c_out], residual and y [..., c_out], one element type.
    Rows may be strided.  ``residual_last``: y = act(x w^T + bias) + residual.
    With ``save``, returns (y, pre): pre is the activation's argument in float32
    for ``linear_backward`` (None for the identity, which needs none)."""
    dt = DTYPES[_dtype_name(x)]
    if w.dim() != 2:
        raise ValueError("w must be [c_out, c_in]")
    c_out, c_in = w.shape
    index = _same(x, (w, bias, residual, out))
    rows, ldx = _rows_dense(x, c_in, "x")
    ldw = _rows_dense(w, c_in, "w")[1]
    xs = x.shape
    y_shape = (xs[0], c_out) if len(xs) == 2 else (*xs[:-1], c_out)
    ldr = ldy = 0
    xp, wp, bp, rp = x.data_ptr(), w.data_ptr(), None, None
    if bias is not None:
        if bias.dim() != 1 or bias.shape[0] != c_out or not bias.is_contiguous():
            raise ValueError("bias must be a contiguous [c_out]")
        bp = bias.data_ptr()
    if residual is not None:
        if residual.shape != y_shape:
            raise ValueError("residual must have y's shape")
        ldr = _rows_dense(residual, c_out, "residual")[1]
        rp = residual.data_ptr()
    if out is not None:
        if out.shape != y_shape:
            raise ValueError("out must have y's shape")
        ldy = _rows_dense(out, c_out, "out")[1]
    if residual_last:
        flags |= FLAG_LINEAR_RESIDUAL_LAST
    if (xp | wp) & 15 and dt:
        flags |= FLAG_LINEAR_UNALIGNED

    def call(handle, out):
        if out is None:
            # (empty_like is the quicker of the two)
            out = torch.empty_like(residual) if rp is not None and ldr == 0 and residual.is_contiguous() else \
                torch.empty(y_shape, dtype=x.dtype, device=x.device)
        pre = torch.empty(y_shape, dtype=torch.float32, device=x.device) if save and act != "identity" else None
        _, ref, need = _linear_problem(index, False, rows, c_in, c_out, ldx, ldw, ldr, ldy, LINEAR_ACTIVATIONS[act], alpha,
                                       beta, dt, 0 if bp is None else 1, 0 if rp is None else 1, flags)
        args = ref, xp, wp, bp, rp, out.data_ptr(), None if pre is None else pre.data_ptr()
        if need:
            with _turn(need, scratch, index, handle):
                _, at, n = _scratch(need, scratch, index, handle)
                status = _load().conv_linear_forward(*args, at, n, handle or None)
        else:
            status = _load().conv_linear_forward(*args, None, 0, handle or None)
        if status:
            _check(status, "conv_linear_forward")
        return (out, pre) if save else out
    return _run(call, index, stream, out)


def linear_backward(dy, x, w, pre=None, *, act="identity", alpha=0.0, beta=0.0, residual_last=False, need_dx=True,
                    need_dw=True, need_dbias=False, need_dresidual=False, dx=None, dw=None, scratch=None, flags=0,
                    stream=None):
    """The gradients of ``linear`` for dy [..., c_out]: (dx, dw, dbias,
    dresidual), None where not wanted.  ``pre`` is what linear(..., save=True)
    returned; act, alpha, beta and residual_last are that call's."""
    torch = _torch()
    dt = DTYPES[_dtype_name(x)]
    if w.dim() != 2:
        raise ValueError("w must be [c_out, c_in]")
    c_out, c_in = w.shape
    index = _same(x, (w, dy))
    rows, ldx = _rows(x, c_in, "x")
    _, ldw = _rows(w, c_in, "w")
    if dy.shape != x.shape[:-1] + (c_out,):
        raise ValueError("dy must have y's shape")
    ldy = _rows(dy, c_out, "dy")[1]
    if act != "identity":
        if pre is None:
            raise ValueError("this activation's gradient needs pre (linear(..., save=True))")
        if pre.shape != dy.shape or pre.dtype != torch.float32 or pre.device != x.device or not pre.is_contiguous():
            raise ValueError("pre must be a contiguous float32 tensor of y's shape")
    else:
        pre = None
    if residual_last:
        flags |= FLAG_LINEAR_RESIDUAL_LAST
    xp, wp, dyp = x.data_ptr(), w.data_ptr(), dy.data_ptr()
    if dt and ((xp if need_dw else 0) | (wp if need_dx else 0) | (dyp if pre is None else 0)) & 15:
        flags |= FLAG_LINEAR_UNALIGNED

    def call(handle, dx, dw):
        dx = _dense_out(dx, x.shape, x, "dx") if need_dx else None
        dw = _dense_out(dw, w.shape, x, "dw") if need_dw else None
        dbias = torch.empty(c_out, dtype=x.dtype, device=x.device) if need_dbias else None
        dres = torch.empty(dy.shape, dtype=x.dtype, device=x.device) if need_dresidual else None
        _, ref, need = _linear_problem(index, True, rows, c_in, c_out, ldx, ldw, 0, ldy, LINEAR_ACTIVATIONS[act], alpha,
                                       beta, dt, 0, 0, flags)
        with _turn(need, scratch, index, handle):
            buf, at, n = _scratch(need, scratch, index, handle)
            status = _load().conv_linear_backward(ref, xp, wp, _ptr(pre), dyp, _ptr(dx), _ptr(dw), _ptr(dbias), _ptr(dres), at,
                                                  n, handle or None)
        _check(status, "conv_linear_backward")
        return dx, dw, dbias, dres
    return _run(call, index, stream, dx, dw)


def _gated(x, w_gate, w_up, w_down):
    if w_gate.dim() != 2 or w_down.dim() != 2 or w_gate.shape != w_up.shape or w_down.shape[1] != w_gate.shape[0]:
        raise ValueError("w_gate and w_up must be [hidden, c_in], w_down [c_out, hidden]")
    for what, t in (("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down)):
        if not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous")
    hidden, c_in = w_gate.shape
    return c_in, hidden, w_down.shape[0]


def gated_ffn(x, w_gate, w_up, w_down, residual=None, *, act="silu", alpha=0.0, beta=0.0, save=False, out=None,
              scratch=None, flags=0, stream=None):
    """y = (act(x w_gate^T) * (x w_up^T)) w_down^T + residual on CUDA tensors: x
    [..., c_in], w_gate and w_up [hidden, c_in], w_down [c_out, hidden],
    residual and y [..., c_out].  With ``save``, returns (y, saved) for
    ``gated_ffn_backward``."""
    dt = DTYPES[_dtype_name(x)]
    index = _same(x, (w_gate, w_up, w_down, residual, out))
    c_in, hidden, c_out = _gated(x, w_gate, w_up, w_down)
    rows, ldx = _rows_dense(x, c_in, "x")
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
    ptrs = x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr()
    if dt and (ptrs[0] | ptrs[1] | ptrs[2] | ptrs[3]) & 15:
        flags |= FLAG_LINEAR_UNALIGNED

    def call(handle, out):
        if out is None:
            out = torch.empty_like(residual) if residual is not None and residual.is_contiguous() else \
                torch.empty(y_shape, dtype=x.dtype, device=x.device)
        _, ref, need, kept = _gated_problem(index, False, rows, c_in, hidden, c_out, ldx, ldr, ldy, LINEAR_ACTIVATIONS[act],
                                            alpha, beta, dt, 0 if residual is None else 1, flags)
        saved = torch.empty(kept, dtype=torch.uint8, device=x.device) if save else None
        with _turn(need, scratch, index, handle):
            buf, at, n = _scratch(need, scratch, index, handle)
            status = _load().conv_gated_forward(ref, *ptrs, _ptr(residual), out.data_ptr(), _ptr(saved), at, n,
                                                handle or None)
        if status:
            _check(status, "conv_gated_forward")
        return (out, saved) if save else out
    return _run(call, index, stream, out)


def gated_ffn_backward(dy, x, w_gate, w_up, w_down, saved, *, act="silu", alpha=0.0, beta=0.0, need_dx=True,
                       need_dw=True, scratch=None, flags=0, stream=None):
    """The gradients of ``gated_ffn`` for dy [..., c_out]: (dx, dw_gate, dw_up,
    dw_down), None where not wanted.  ``saved`` is what gated_ffn(...,
    save=True) returned; act, alpha and beta are that call's.  The residual's
    gradient is dy."""
    torch = _torch()
    dt = DTYPES[_dtype_name(x)]
    index = _same(x, (w_gate, w_up, w_down, dy))
    c_in, hidden, c_out = _gated(x, w_gate, w_up, w_down)
    rows, ldx = _rows(x, c_in, "x")
    if dy.shape != x.shape[:-1] + (c_out,):
        raise ValueError("dy must have y's shape")
    ldy = _rows(dy, c_out, "dy")[1]
    ptrs = x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr()
    if dt and (ptrs[0] | ptrs[1] | ptrs[2] | ptrs[3] | dy.data_ptr()) & 15:
        flags |= FLAG_LINEAR_UNALIGNED

    def call(handle):
        _, ref, need, kept = _gated_problem(index, True, rows, c_in, hidden, c_out, ldx, 0, ldy, LINEAR_ACTIVATIONS[act], alpha,
                                            beta, dt, 0, flags)
        if saved.dtype != torch.uint8 or saved.get_device() != index or saved.numel() != kept:
            raise ValueError("saved must be what gated_ffn(..., save=True) returned for this problem")
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device) if need_dx else None
        dws = [torch.empty(w.shape, dtype=x.dtype, device=x.device) if need_dw else None
               for w in (w_gate, w_up, w_down)]
        with _turn(need, scratch, index, handle):
            buf, at, n = _scratch(need, scratch, index, handle)
            status = _load().conv_gated_backward(ref, *ptrs, saved.data_ptr(), dy.data_ptr(), _ptr(dx),
                                                 *[_ptr(t) for t in dws], at, n, handle or None)
        _check(status, "conv_gated_backward")
        return (dx, *dws)
    return _run(call, index, stream)


def clip_grad_norm(grads, max_norm, *, eps=1e-6, out=None, scratch=None, stream=None):
    """The 2-norm of all tensors of ``grads`` together (a float32 scalar on the
    device), and the tensors scaled by min(1, max_norm / (norm + eps)): in
    place, or into the tensors of ``out``.  Tensors are contiguous, of any mix
    of the element types."""
    torch = _torch()
    grads = list(grads)
    n = len(grads)
    if n == 0:
        raise ValueError("no gradients")
    # one pass over the list per property (a model has hundreds of tensors; their kernels take microseconds)
    tensor = torch.Tensor
    outs = grads if out is None else list(out)
    if len(outs) != n:
        raise ValueError("out must have one tensor per gradient")
    names = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
    types = [g.dtype for g in grads]
    sizes = list(map(tensor.numel, grads))
    index = grads[0].get_device()
    if index < 0:
        raise ValueError("operands must be CUDA tensors")
    if set(map(tensor.get_device, grads)) != {index} or not all(map(tensor.is_contiguous, grads)):
        raise ValueError("gradients must be contiguous and on one device")
    if out is not None and ([o.dtype for o in outs] != types or list(map(tensor.numel, outs)) != sizes or
                            set(map(tensor.get_device, outs)) != {index} or not all(map(tensor.is_contiguous, outs))):
        raise ValueError("out must be contiguous tensors of the gradients' sizes and element types")
    try:
        types = array("i", [names[t] for t in types])
    except KeyError as e:
        raise TypeError(f"unsupported element type {e}") from None
    sizes = array("q", sizes)
    ins = array("Q", map(tensor.data_ptr, grads))
    to = ins if out is None else array("Q", map(tensor.data_ptr, outs))
    lib = _load()

    def call(handle):
        norm = torch.empty((), dtype=torch.float32, device=index)
        at_sizes = sizes.buffer_info()[0]
        need = ctypes.c_size_t()
        _check(lib.conv_clip_scratch_bytes(n, at_sizes, ctypes.byref(need)), "conv_clip_scratch_bytes")
        with _turn(need.value, scratch, index, handle):
            buf, at, size = _scratch(need.value, scratch, index, handle)
            status = lib.conv_clip_grads(n, ins.buffer_info()[0], to.buffer_info()[0], at_sizes, types.buffer_info()[0],
                                         max_norm, eps, norm.data_ptr(), at, size, handle or None)
        _check(status, "conv_clip_grads")
        return norm
    return _run(call, index, stream)
