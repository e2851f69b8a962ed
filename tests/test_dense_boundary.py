"""The dense operators' C ABI on the host: exports, struct layouts, refusals
before anything touches a device, and the Python checks of arguments."""
import ctypes
import os
import re
import subprocess
import sys
import threading

import pytest
import torch

import implicit_gemm_cnn_gb300 as conv
from implicit_gemm_cnn_gb300 import build as conv_build, dense

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, SHAPE, OVERFLOW, DTYPE, ACT, NULL, SCRATCH, ALIAS, DEVICE, CUDA, ARG = range(11)


@pytest.fixture(scope="module")
def lib():
    conv_build.build()
    return dense._load()


def test_exports_every_declared_symbol(lib):
    text = open(os.path.join(ROOT, "include", "linear.h")).read()
    names = re.findall(r"CONV_API\s+[\w\s\*]+?\b(conv_\w+)\s*\(", text)
    assert len(names) == 13, names
    for name in names:
        assert hasattr(lib, name), name
        assert name in conv.__all__ and callable(getattr(conv, name))


def test_struct_layouts_match_the_header():
    assert ctypes.sizeof(conv.LinearProblem) == 88 and conv.LinearProblem.act.offset == 56
    assert conv.LinearProblem.flags.offset == 80
    assert ctypes.sizeof(conv.GatedProblem) == 80 and conv.GatedProblem.flags.offset == 76


def describe(lib, **kw):
    a = dict(rows=4, c_in=8, c_out=8, dtype="bf16")
    a.update(kw)
    p = conv.make_linear_problem(a.pop("rows"), a.pop("c_in"), a.pop("c_out"), **a)
    buf = ctypes.create_string_buffer(256)
    return lib.conv_linear_describe_plan(ctypes.byref(p), 0, 152, buf, 256)


def test_linear_validation(lib):
    assert describe(lib) == OK and describe(lib, rows=0) == OK
    for kw, want in [(dict(rows=-1), SHAPE), (dict(c_in=0), SHAPE), (dict(c_out=0), SHAPE), (dict(rows=2 ** 31), SHAPE),
                     (dict(x_stride=7), SHAPE), (dict(w_stride=7), SHAPE), (dict(y_stride=7), SHAPE),
                     (dict(residual_stride=-1), SHAPE), (dict(x_stride=2 ** 40), SHAPE),
                     (dict(rows=2 ** 30, c_in=2 ** 20), OVERFLOW), (dict(flags=0x100), ARG)]:
        assert describe(lib, **kw) == want, kw
    p = conv.make_linear_problem(4, 8, 8)
    buf = ctypes.create_string_buffer(256)
    ref = ctypes.byref(p)
    assert lib.conv_linear_describe_plan(ref, 3, 152, buf, 256) == ARG
    assert lib.conv_linear_describe_plan(ref, 0, 0, buf, 256) == ARG
    assert lib.conv_linear_describe_plan(ref, 0, 152, None, 0) == NULL
    assert lib.conv_linear_describe_plan(None, 0, 152, buf, 256) == NULL
    p.dtype = 3
    assert lib.conv_linear_describe_plan(ref, 0, 152, buf, 256) == DTYPE
    p.dtype, p.act = 0, 11
    assert lib.conv_linear_describe_plan(ref, 0, 152, buf, 256) == ACT


def test_convolutions_do_not_take_the_dense_activations(lib):
    p = conv.make_problem((1, 4, 8, 8), (4, 4, 3, 3))
    p.act = 9
    ho = ctypes.c_int64()
    assert lib.conv_output_shape(ctypes.byref(p), ctypes.byref(ho), ctypes.byref(ho)) == ACT


def test_linear_pointer_refusals(lib):
    """Reported before a device is asked for: the addresses are never used."""
    p = conv.make_linear_problem(4, 8, 8, has_bias=True, has_residual=True)
    x, w, b, r, y, pre = (0x10000 * i for i in range(1, 7))
    f = lib.conv_linear_forward

    def call(*a):
        return f(ctypes.byref(p), *a, None, 0, None)
    for missing in range(5):
        args = [x, w, b, r, y, pre]
        args[missing] = None
        assert call(*args) == NULL, missing
    assert f(None, x, w, b, r, y, pre, None, 0, None) == NULL
    for bad in (x + 127, w, b + 4, r + 100):
        assert call(x, w, b, r, bad, None) == ALIAS
    assert call(x, w, b, r, y, y + 64) == ALIAS and call(x, w, b, r, y, x) == ALIAS
    # columns side by side in one wider matrix do not overlap; shifted by a row they still do not, by a value they do
    side = conv.make_linear_problem(4, 8, 8, x_stride=24, y_stride=24)
    for at, want in ((x + 32, None), (x + 64, None), (x + 96 + 32, None), (x - 96 + 64, None), (x + 28, ALIAS),
                     (x + 68, ALIAS), (x + 96 + 28, ALIAS)):
        if torch.cuda.is_available() and want is None:
            continue  # (with a device it would run)
        got = f(ctypes.byref(side), x, w, None, None, at, None, None, 0, None)
        assert (got == ALIAS) == (want == ALIAS), at - x
    p.rows = 0
    assert call(None, None, None, None, None, None) == OK  # nothing to do
    p.rows = 4
    g = lib.conv_linear_backward
    dy, dx, dw, db, dr = (0x100000 * i for i in range(1, 6))

    def back(x, w, pre, dy, dx, dw, db, dr):
        return g(ctypes.byref(p), x, w, pre, dy, dx, dw, db, dr, None, 0, None)
    assert back(x, w, None, None, dx, dw, db, dr) == NULL
    assert back(None, w, None, dy, None, dw, None, None) == NULL
    assert back(x, None, None, dy, dx, None, None, None) == NULL
    assert back(x, w, None, dy, dx, dx, None, None) == ALIAS and back(x, w, None, dy, dy, None, None, None) == ALIAS
    p.act = 2
    assert back(x, w, None, dy, dx, None, None, None) == NULL  # pre
    if not torch.cuda.is_available():
        p.act = 0
        assert call(x, w, b, r, y, None) == DEVICE and back(x, w, None, dy, dx, dw, db, dr) == DEVICE


def test_gated_refusals(lib):
    n = ctypes.c_size_t()
    for kw, want in [(dict(), OK), (dict(hidden=0), SHAPE), (dict(rows=-1), SHAPE), (dict(x_stride=3), SHAPE),
                     (dict(flags=1), ARG)]:
        a = dict(rows=4, c_in=8, hidden=16, c_out=8)
        a.update(kw)
        p = conv.make_gated_problem(a.pop("rows"), a.pop("c_in"), a.pop("hidden"), a.pop("c_out"), **a)
        assert lib.conv_gated_saved_bytes(ctypes.byref(p), ctypes.byref(n)) == want, kw
    p = conv.make_gated_problem(4, 8, 16, 8, has_residual=True)
    x, g, u, d, r, y, s = (0x10000 * i for i in range(1, 8))
    f = lib.conv_gated_forward
    for missing in range(6):
        args = [x, g, u, d, r, y]
        args[missing] = None
        assert f(ctypes.byref(p), *args, None, None, 0, None) == NULL
    assert f(ctypes.byref(p), x, g, u, d, r, x, None, None, 0, None) == ALIAS
    assert f(ctypes.byref(p), x, g, u, d, r, y, s + 16, None, 0, None) == ARG  # saved is 256-byte aligned
    assert f(ctypes.byref(p), x, g, u, d, r, y, x, None, 0, None) == ALIAS
    b = lib.conv_gated_backward
    dy, dx, dg, du, dd = (0x100000 * i for i in range(1, 6))
    assert b(ctypes.byref(p), x, g, u, d, None, dy, dx, dg, du, dd, None, 0, None) == NULL
    assert b(ctypes.byref(p), x, g, u, d, s, None, dx, dg, du, dd, None, 0, None) == NULL
    assert b(ctypes.byref(p), None, g, u, d, s, dy, None, dg, None, None, None, 0, None) == NULL
    assert b(ctypes.byref(p), x, g, u, d, s, dy, dx, dg, dg, dd, None, 0, None) == ALIAS
    # the block's saved state: g and u in float32 and h, rows of a multiple of 64 elements
    p = conv.make_gated_problem(10, 8, 13, 8, dtype="f16")
    assert conv.conv_gated_saved_bytes(p) == 2 * 10 * 64 * 4 + 10 * 64 * 2


def test_clip_refusals(lib):
    a, b, norm, scratch = 0x10000, 0x20000, 0x30000, 0x40000
    need = conv.conv_clip_scratch_bytes([100, 50])

    def call(ins=(a, b), outs=None, sizes=(100, 50), types=(0, 2), max_norm=1.0, eps=1e-6, norm=norm, scratch=scratch,
             n=need):
        k = len(ins)
        vp = ctypes.c_void_p * k
        return lib.conv_clip_grads(k, vp(*ins), vp(*(outs or ins)), (ctypes.c_int64 * k)(*sizes),
                                   (ctypes.c_int32 * k)(*types), max_norm, eps, norm, scratch, n, None)
    assert call(ins=(a, None)) == NULL and call(norm=None) == NULL and call(outs=(a, None)) == NULL
    assert call(sizes=(100, -1)) == SHAPE and call(types=(0, 3)) == DTYPE
    assert call(max_norm=-1.0) == ARG and call(max_norm=float("nan")) == ARG and call(eps=-1.0) == ARG
    assert call(ins=(a + 2, b)) == ARG and call(ins=(a, b + 1)) == ARG
    assert call(scratch=None) == SCRATCH and call(n=need - 1) == SCRATCH and call(scratch=scratch + 8) == SCRATCH
    assert call(ins=(a, a + 64)) == ALIAS                      # two tensors over each other, in place
    assert call(outs=(a + 4, b + 0x8000)) == ALIAS             # an output shifted over its input
    assert call(outs=(0x50000, 0x50000 + 64)) == ALIAS         # outputs over each other
    assert call(norm=a + 8) == ALIAS and call(scratch=0x10000, ins=(0x10000, b)) == ALIAS
    assert lib.conv_clip_scratch_bytes(-1, None, ctypes.byref(ctypes.c_size_t())) == SHAPE
    if not torch.cuda.is_available():
        assert call() == DEVICE


def test_python_argument_checks():
    x, w = torch.zeros(4, 8), torch.zeros(6, 8)
    with pytest.raises(ValueError, match="CUDA"):
        conv.linear(x, w)
    with pytest.raises(TypeError):
        conv.linear(x.double(), w.double())
    for rows, want in [(torch.zeros(3, 8), (3, 8)), (torch.zeros(2, 3, 8), (6, 8)), (torch.zeros(8), (1, 0)),
                       (torch.zeros(3, 20)[:, 4:12], (3, 20)), (torch.zeros(0, 8), (0, 0)),
                       (torch.zeros(2, 3, 20)[:, :, :8], (6, 20)), (torch.zeros(1, 1, 8), (1, 0))]:
        assert dense._rows(rows, 8, "x") == want
    for bad in (torch.zeros(3, 7), torch.zeros(8, 3).t(), torch.zeros(2, 4, 20)[:, :3, :8], torch.zeros(1, 8).expand(3, 8),
                torch.zeros(3, 16)[:, ::2], torch.zeros(())):
        with pytest.raises(ValueError):
            dense._rows(bad, 8, "x")


def test_plans(lib):
    """Which kernel runs is a function of the shape and the SM count."""
    def plan(rows, c_in, c_out, which=0, **kw):
        return conv.conv_linear_describe_plan(conv.make_linear_problem(rows, c_in, c_out, **kw), which, 152)
    assert plan(0, 8, 8) == "nothing launches=0"
    for dtype in ("f32", "f16", "bf16"):
        assert plan(1, 1024, 1024, dtype=dtype).startswith("few_rows")
        assert plan(16, 1024, 1024, dtype=dtype).startswith("few_rows")
        assert "launches=1" in plan(16, 1024, 1024, dtype=dtype)
        for flags in (conv.FLAG_LINEAR_NO_FEW_ROWS, 0):
            assert plan(17 if not flags else 1, 1024, 1024, dtype=dtype, flags=flags).startswith("tcgen05")
        assert plan(500, 1024, 1024, dtype=dtype, flags=conv.FLAG_LINEAR_FORCE_FFMA).startswith("ffma")
    assert plan(500, 1024, 1024, dtype="f32").startswith("tcgen05_bf16x3")
    assert "tile=256x256 sms_per_tile=2" in plan(8192, 4096, 8192, dtype="bf16")
    # 256 tiles on 76 pairs: three rounds whole, the last 28 tiles as two ranges each
    d = plan(8192, 2048, 8192, 1, dtype="bf16")
    assert "tiles=256 whole=228 split=2" in d and "launches=2" in d
    # few tiles: all of them in ranges
    assert "whole=0 split=" in plan(64, 8192, 256, dtype="bf16")
    for a in ((3, 5, 7), (100, 1000, 3), (5000, 70, 900), (64, 30000, 64)):
        assert plan(*a, dtype="f16") == plan(*a, dtype="f16")


def test_plans_of_few_rows(lib):
    """Up to 8 rows one kernel; to 16 it, unless the tensor cores are the quicker."""
    def few(rows, c_in, c_out, dtype, **kw):
        p = conv.make_linear_problem(rows, c_in, c_out, dtype=dtype, **kw)
        return conv.conv_linear_describe_plan(p, 0, 152).startswith("few_rows")
    for dtype in ("f32", "f16", "bf16"):
        assert few(8, 1001, 20000, dtype) and few(8, 1000, 20000, dtype)
        assert few(9, 1000, 1000, dtype) and not few(17, 1000, 1000, dtype)
    for dtype in ("f16", "bf16"):
        assert few(9, 1000, 9999, dtype) and not few(9, 1000, 10000, dtype)
        assert few(16, 1001, 20000, dtype) and few(16, 1000, 20000, dtype, x_stride=1001)  # operands would be copied
        assert few(16, 1000, 20000, dtype, flags=conv.FLAG_LINEAR_UNALIGNED)
    assert few(16, 1000, 20000, "f32") and not few(9, 1001, 100, "f32")
    assert not few(9, 1000, 100, "f32", w_stride=1002)


def test_rows_of_broadcast_dimensions_are_refused():
    """A dimension of stride 0 anywhere among the leading ones: its rows lie over each other, not one after another."""
    for bad in (torch.zeros(3, 1, 8).expand(3, 4, 8), torch.zeros(2, 1, 1, 8).expand(2, 3, 4, 8),
                torch.zeros(2, 3, 1, 8).expand(2, 3, 4, 8), torch.zeros(2, 1, 4, 8).expand(2, 3, 4, 8),
                torch.zeros(1, 4, 8).expand(3, 4, 8), torch.zeros(1, 1, 8).expand(3, 4, 8),
                torch.zeros(3, 1, 20)[:, :, :8].expand(3, 4, 8)):
        for rows in (dense._rows, dense._rows_dense):
            with pytest.raises(ValueError):
                rows(bad, 8, "x")
    with pytest.raises(ValueError):
        dense._rows(torch.zeros(3, 1, 1).expand(3, 4, 1), 1, "x")  # rows of one value
    # dimensions of one element have no stride
    assert dense._rows(torch.zeros(1, 8).expand(1, 8), 8, "x") == (1, 0)
    assert dense._rows(torch.zeros(3, 1, 8).expand(3, 1, 8), 8, "x") == (3, 8)


class _OnDevice(torch.Tensor):
    """A host tensor that says it is on device 0: what is refused before anything is enqueued can be tried without one."""

    def get_device(self):
        return 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="host addresses: for machines that could not use them")
def test_broadcast_operands_are_refused():
    def on(t):
        return t.as_subclass(_OnDevice)
    x, w = on(torch.zeros(3, 4, 8)), on(torch.zeros(6, 8))
    wide, row = on(torch.zeros(3, 1, 8).expand(3, 4, 8)), on(torch.zeros(3, 1, 6).expand(3, 4, 6))
    g, d = on(torch.zeros(12, 8)), on(torch.zeros(6, 12))
    for call in (lambda: conv.linear(wide, w), lambda: conv.linear(x, w, residual=row), lambda: conv.linear(x, w, out=row),
                 lambda: conv.linear_backward(row, x, w), lambda: conv.linear_backward(on(torch.zeros(3, 4, 6)), wide, w),
                 lambda: conv.gated_ffn(wide, g, g, d), lambda: conv.gated_ffn(x, g, g, d, row),
                 lambda: conv.gated_ffn(x, g, g, d, out=row), lambda: conv.gated_ffn_backward(row, x, g, g, d, None),
                 lambda: conv.gated_ffn_backward(on(torch.zeros(3, 4, 6)), wide, g, g, d, None)):
        with pytest.raises(ValueError, match="rows must not overlap|rows must be evenly spaced"):
            call()


def test_addresses_inside_an_element_are_refused(lib):
    """Every operand and output, each type, off its element's boundary: refused before a device is asked for."""
    at = [0x1000000 * i for i in range(1, 12)]
    for dtype, offs in (("f32", (1, 2, 3)), ("f16", (1,)), ("bf16", (1,))):
        linear = conv.make_linear_problem(20, 64, 64, dtype=dtype, act="relu", has_bias=True, has_residual=True)
        gated = conv.make_gated_problem(20, 64, 64, 64, dtype=dtype, has_residual=True)
        for fn, p, n, aligned in ((lib.conv_linear_forward, linear, 6, ()), (lib.conv_linear_backward, linear, 8, ()),
                                  (lib.conv_gated_forward, gated, 7, (6,)), (lib.conv_gated_backward, gated, 10, (5,))):
            def call(args):
                return fn(ctypes.byref(p), *args, None, 0, None)
            for i in range(n):
                for off in offs:
                    args = at[:n]
                    args[i] += off
                    assert call(args) == ARG, (fn.__name__, dtype, i, off)
            if not torch.cuda.is_available():
                assert call(at[:n]) == DEVICE
    # float32 beside 16-bit operands: the activation's argument, and the norm
    p = conv.make_linear_problem(20, 64, 64, dtype="f16", act="relu")
    assert lib.conv_linear_forward(ctypes.byref(p), *at[:2], None, None, at[4], at[5] + 2, None, 0, None) == ARG
    assert lib.conv_linear_backward(ctypes.byref(p), *at[:2], at[2] + 2, *at[3:8], None, 0, None) == ARG
    one = (ctypes.c_int64 * 1)(64)
    need = conv.conv_clip_scratch_bytes([64])
    for off in (1, 2, 3):
        assert lib.conv_clip_grads(1, (ctypes.c_void_p * 1)(at[0]), None, one, (ctypes.c_int32 * 1)(1), 1.0, 0.0, at[1] + off,
                                   at[2], need, None) == ARG


def test_plans_for_any_sm_count():
    """In a process of its own: a division by zero would end it.  Every SM count has a plan that keeps to its SMs."""
    code = """
import sys
sys.path.insert(0, %r)
import implicit_gemm_cnn_gb300 as conv
for dtype in ("f32", "f16", "bf16"):
    for size in ((64, 1024, 1024), (1, 64, 64), (300, 70, 900), (5000, 2000, 3)):
        for flags in (0, conv.FLAG_LINEAR_FORCE_FFMA, conv.FLAG_LINEAR_NO_FEW_ROWS):
            p = conv.make_linear_problem(*size, dtype=dtype, flags=flags)
            for which in (0, 1, 2):
                for sm in (1, 2, 3, 151, 2**31 - 1):
                    d = conv.conv_linear_describe_plan(p, which, sm)
                    assert f"sms={sm} " in d and not (sm == 1 and "sms_per_tile=2" in d), d
print("planned")
""" % ROOT
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "planned", (r.returncode, r.stderr[-500:])


def test_a_sum_of_no_terms_is_refused(monkeypatch):
    """c_in, hidden or c_out of 0: the library's own status, at whatever function meets it first."""
    def on(*shape):
        return torch.zeros(*shape).as_subclass(_OnDevice)
    # what runs on a device does not: the problem is refused before
    monkeypatch.setattr(dense, "_run", lambda call, index, stream, *args: call(0, *args))
    monkeypatch.setattr(dense, "_dense_out", lambda *a: None)
    dense._torch()
    assert dense._rows_dense(torch.zeros(4, 0), 0, "x")[0] == 4 and dense._rows_dense(torch.zeros(2, 3, 0), 0, "x")[0] == 6
    for call in (lambda: conv.linear(on(4, 0), on(6, 0)), lambda: conv.linear(on(2, 3, 0), on(6, 0)),
                 lambda: conv.linear(on(4, 8), on(0, 8)), lambda: conv.linear_backward(on(4, 6), on(4, 0), on(6, 0)),
                 lambda: conv.gated_ffn(on(4, 0), on(5, 0), on(5, 0), on(6, 5)),
                 lambda: conv.gated_ffn(on(4, 8), on(0, 8), on(0, 8), on(6, 0)),
                 lambda: conv.gated_ffn_backward(on(4, 6), on(4, 0), on(5, 0), on(5, 0), on(6, 5), on(0))):
        with pytest.raises(conv.ConvError, match="SHAPE"):
            call()


def test_empty_tensors_have_no_rows():
    for empty in (torch.zeros(2, 0, 8), torch.zeros(0, 3, 8), torch.zeros(2, 3, 0, 5, 8), torch.zeros(0, 8),
                  torch.zeros(4, 3, 20)[:, :0, 4:12], torch.zeros(0, 1, 8).expand(0, 3, 8),
                  torch.zeros(8, 0).t(), torch.zeros(2, 8, 0).transpose(1, 2)):
        assert dense._rows(empty, 8, "x") == (0, 0) and dense._rows_dense(empty, 8, "x") == (0, 0)
    with pytest.raises(ValueError):
        dense._rows(torch.zeros(2, 0, 7), 8, "x")


def test_scratch_sizes_are_kept_per_device(monkeypatch):
    """Plans go by the SM count: what one device's query said is not taken for another's."""
    now = []

    class On1(torch.Tensor):
        def get_device(self):
            return 1

    def run(call, index, stream, *args):
        now.append(index)
        return call(0, *args)

    class Library:
        def __getattr__(self, name):
            return lambda *a: 0

    asked = []
    monkeypatch.setattr(dense, "_run", run)
    monkeypatch.setattr(dense, "_load", lambda: Library())
    monkeypatch.setattr(dense, "_dense_out", lambda *a: None)
    monkeypatch.setattr(dense, "_scratch", lambda need, given, index, handle: (asked.append(need), None, 0))
    monkeypatch.setattr(dense, "conv_gated_saved_bytes", lambda p: 0)
    for name in ("linear", "linear_backward", "gated", "gated_backward"):
        monkeypatch.setattr(dense, f"conv_{name}_scratch_bytes", lambda p: 1000 + now[-1])
    monkeypatch.setattr(dense, "_linear_cache", {})
    monkeypatch.setattr(dense, "_gated_cache", {})
    dense._torch()
    for _ in range(2):
        for cls, want in ((_OnDevice, 1000), (On1, 1001)):
            x, w, dy, g, d = (torch.zeros(*s).as_subclass(cls) for s in ((4, 8), (6, 8), (4, 6), (12, 8), (6, 12)))
            saved = torch.zeros(0, dtype=torch.uint8).as_subclass(cls)
            del asked[:]
            conv.linear(x, w)
            conv.linear_backward(dy, x, w)
            conv.gated_ffn(x, g, g, d)
            conv.gated_ffn_backward(dy, x, g, g, d, saved)
            assert asked == [want] * 4


@pytest.mark.parametrize("op", ["linear", "linear_backward", "gated", "gated_backward"])
def test_only_calls_that_share_a_scratch_take_turns(monkeypatch, op):
    """One call stands in its launch (a full queue).  Calls on another stream or device, and calls on its own stream whose
    scratch is not the kept one, go on; a call on its stream that shares the scratch waits."""
    inside, go = threading.Event(), threading.Event()

    class On1(torch.Tensor):
        def get_device(self):
            return 1

    class Library:
        def __getattr__(self, name):
            def call(*args):
                if threading.current_thread().name == "first" and name in (f"conv_{op}", f"conv_{op}_forward"):
                    inside.set()
                    assert go.wait(30)
                return 0
            return call

    size = [4096]
    monkeypatch.setattr(dense, "_load", lambda: Library())
    monkeypatch.setattr(dense, "_run", lambda call, index, stream, *args: call(stream, *args))
    monkeypatch.setattr(dense, "_scratch", lambda need, given, index, handle: (given, 256, need))
    monkeypatch.setattr(dense, "_dense_out", lambda *a: None)
    for name in ("linear", "linear_backward", "gated", "gated_backward"):
        monkeypatch.setattr(dense, f"conv_{name}_scratch_bytes", lambda p: size[0])
    monkeypatch.setattr(dense, "conv_gated_saved_bytes", lambda p: 0)
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: empty(*a, **kw))
    dense._torch()

    def run(stream, cls=_OnDevice, need=4096, **kw):
        size[0] = need
        dense._linear_cache.clear()
        dense._gated_cache.clear()
        x, w, dy, g, d = (torch.zeros(*s).as_subclass(cls) for s in ((4, 8), (6, 8), (4, 6), (12, 8), (6, 12)))
        saved = torch.zeros(0, dtype=torch.uint8).as_subclass(cls)
        {"linear": lambda: conv.linear(x, w, stream=stream, **kw),
         "linear_backward": lambda: conv.linear_backward(dy, x, w, stream=stream, **kw),
         "gated": lambda: conv.gated_ffn(x, g, g, d, stream=stream, **kw),
         "gated_backward": lambda: conv.gated_ffn_backward(dy, x, g, g, d, saved, stream=stream, **kw)}[op]()

    def start(name, *args, **kw):
        t = threading.Thread(target=run, name=name, args=args, kwargs=kw, daemon=True)
        t.start()
        return t
    try:
        first = start("first", 7)
        assert inside.wait(30)
        for name, args, kw in (("other stream", (8,), {}), ("other device", (7, On1), {}), ("large", (7,), dict(need=dense._KEPT + 1)),
                               ("own", (7,), dict(scratch=empty(64, dtype=torch.uint8))), ("none", (7,), dict(need=0))):
            t = start(name, *args, **kw)
            t.join(10)
            assert not t.is_alive(), name
        second = start("second", 7)
        second.join(0.2)
        assert second.is_alive() and first.is_alive()
        go.set()
        for t in (first, second):
            t.join(10)
            assert not t.is_alive()
    finally:
        go.set()
        dense._linear_cache.clear()
        dense._gated_cache.clear()
