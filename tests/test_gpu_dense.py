"""The dense operators on the GPU against their float64 definitions, each value
within the bound that dense_ref derives for it."""
import pytest
import torch

import implicit_gemm_cnn_gb300 as conv
import dense_ref as ref

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

ACTS = [("identity", 0, 0), ("relu", 0, 0), ("silu", 0, 0), ("sigmoid", 0, 0), ("tanh", 0, 0), ("hard_swish", 0, 0),
        ("hard_sigmoid", 0.2, 0.5), ("clip", -0.7, 0.9), ("leaky_relu", 0.1, 0), ("gelu", 0, 0), ("gelu_tanh", 0, 0)]


def rand(*shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * scale).to(ref.TORCH[dtype])


def cuda(*ts):
    return [t.cuda() if t is not None else None for t in ts]


def wide(*ts):
    return [t.double() if t is not None else None for t in ts]


def linear_case(rows, c_in, c_out, dtype, act="identity", alpha=0.0, beta=0.0, bias=True, residual=True, last=False,
                flags=0, seed=0, scale=1.0):
    x = rand(rows, c_in, dtype=dtype, seed=seed)
    w = rand(c_out, c_in, dtype=dtype, seed=seed + 1, scale=scale * c_in ** -0.5)
    b = rand(c_out, dtype=dtype, seed=seed + 2) if bias else None
    r = rand(rows, c_out, dtype=dtype, seed=seed + 3) if residual else None
    dy = rand(rows, c_out, dtype=dtype, seed=seed + 4, scale=0.1)
    X, W, B, R, DY = cuda(x, w, b, r, dy)
    y, pre = conv.linear(X, W, B, R, act=act, alpha=alpha, beta=beta, residual_last=last, save=True, flags=flags)
    y2 = conv.linear(X, W, B, R, act=act, alpha=alpha, beta=beta, residual_last=last, flags=flags)
    grads = conv.linear_backward(DY, X, W, pre, act=act, alpha=alpha, beta=beta, residual_last=last, need_dbias=True,
                                 need_dresidual=True, flags=flags)
    torch.cuda.synchronize()
    assert conv.conv_linear_device_error() == 0
    assert torch.equal(y, y2)
    x, w, b, r, dy = wide(x, w, b, r, dy)
    want = ref.linear64(x, w, b, r, act, alpha, beta, last, dtype)
    ref.check(y, want["y"], "y")
    if act != "identity":
        ref.check(pre, want["z"], "pre")
    back = ref.linear_backward64(dy, x, w, *want["z"], act, alpha, beta, last, dtype)
    for name, got in zip(("dx", "dw", "dbias", "dresidual"), grads):
        ref.check(got, back[name], name)


# rows, c_in, c_out: one of everything, odd ones, sizes around tiles and ranges
SIZES = [(1, 1, 1), (1, 8, 8), (1, 64, 129), (2, 7, 5), (3, 65, 64), (5, 200, 33), (8, 1024, 24), (12, 250, 301),
         (16, 264, 256), (17, 512, 40), (33, 96, 1000), (64, 72, 200), (100, 136, 120), (127, 320, 257),
         (129, 129, 127), (200, 1000, 72), (256, 64, 256), (300, 257, 515), (513, 40, 384), (640, 520, 264), (50, 1, 3), (40, 3, 1), (1000, 2, 2)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_linear_sizes(size, dtype):
    linear_case(*size, dtype, act="gelu_tanh", seed=sum(size))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ACTS, ids=lambda a: a[0])
@pytest.mark.parametrize("rows", [3, 150])
def test_linear_activations(act, dtype, rows):
    linear_case(rows, 48, 72, dtype, *act, seed=11, scale=2.0)
    linear_case(rows, 48, 72, dtype, *act, last=True, bias=False, seed=12, scale=2.0)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("flags", [conv.FLAG_LINEAR_FORCE_FFMA, conv.FLAG_LINEAR_NO_FEW_ROWS,
                                   conv.FLAG_LINEAR_UNALIGNED])
def test_linear_other_kernels(flags, dtype):
    linear_case(9, 200, 130, dtype, act="silu", flags=flags)
    linear_case(150, 200, 130, dtype, act="silu", flags=flags)


def test_linear_long_sums_and_many_tiles():
    linear_case(40, 9000, 48, "bf16", seed=21)
    linear_case(2100, 300, 1400, "f16", act="silu", seed=22)
    linear_case(1, 20000, 17, "f16", seed=23)
    linear_case(70, 3000, 50, "f32", seed=24)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows", [0, 1, 5, 150])
def test_linear_strides_and_alignments(rows, dtype):
    """Rows of a wider array, at an odd offset and at an aligned one; outputs too. What lies between the rows stays."""
    for off, pad in ((0, 8), (1, 5), (8, 24), (3, 0)):
        c_in, c_out = 80, 56
        xs, ws = rand(rows, c_in + off + pad, dtype=dtype, seed=1), rand(c_out, c_in + off + pad, dtype=dtype, seed=2,
                                                                         scale=0.1)
        rs = rand(rows, c_out + off + pad, dtype=dtype, seed=3)
        X, W, R = cuda(xs, ws, rs)
        full = torch.full((rows, c_out + off + pad), 77.0, dtype=ref.TORCH[dtype], device="cuda")
        x, w, r, out = X[:, off:off + c_in], W[:, off:off + c_in], R[:, off:off + c_out], full[:, off:off + c_out]
        y = conv.linear(x, w, None, r, act="silu", out=out)
        torch.cuda.synchronize()
        want = ref.linear64(*wide(x.cpu(), w.cpu(), None, r.cpu()), "silu", 0, 0, False, dtype)
        ref.check(y, want["y"], (off, pad))
        assert (full[:, :off] == 77).all() and (full[:, off + c_out:] == 77).all()
        dyf = rand(rows, c_out + off + pad, dtype=dtype, seed=4).cuda()
        dy = dyf[:, off:off + c_out]
        dx, dw, db, _ = conv.linear_backward(dy, x, w, need_dbias=True)
        torch.cuda.synchronize()
        back = ref.linear_backward64(*wide(dy.cpu(), x.cpu(), w.cpu()), *want["z"], "identity", 0, 0, False, dtype)
        for name, got in (("dx", dx), ("dw", dw), ("dbias", db)):
            ref.check(got, back[name], (name, off, pad))


def test_linear_unaligned_without_scratch_runs_the_cuda_core_kernel():
    x, w = rand(40, 81, dtype="f16", seed=1).cuda()[:, 1:], rand(24, 88, dtype="f16", seed=2).cuda()[:, :80]
    p = conv.make_linear_problem(40, 80, 24, dtype="f16", x_stride=88, w_stride=88)
    x = torch.cat([x, x[:, :8]], 1).contiguous().flatten()[4:4 + 40 * 88 - 8]  # 8 bytes off a 16-byte boundary
    need = conv.conv_linear_scratch_bytes(p)
    scratch = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    y = torch.empty(40, 24, dtype=torch.float16, device="cuda")
    conv.conv_linear_forward(p, x, w, None, None, y, None, scratch, need)
    torch.cuda.synchronize()
    xs = torch.as_strided(x, (40, 80), (88, 1))
    ref.check(y, ref.linear64(*wide(xs.cpu(), w.cpu(), None, None), "identity", 0, 0, False, "f16")["y"])


def test_linear_leading_dimensions_and_another_stream():
    x, w = rand(2, 3, 5, 64, dtype="bf16", seed=1).cuda(), rand(40, 64, dtype="bf16", seed=2, scale=0.1).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = conv.linear(x, w, act="gelu", stream=side)
    y_raw = conv.linear(x, w, act="gelu", stream=side.cuda_stream)
    side.synchronize()
    assert y.shape == (2, 3, 5, 40) and torch.equal(y, y_raw)
    want = ref.linear64(*wide(x.cpu().reshape(30, 64), w.cpu(), None, None), "gelu", 0, 0, False, "bf16")["y"]
    ref.check(y.reshape(30, 40), want)


@pytest.mark.parametrize("rows", [4, 140])
def test_linear_infinities_and_nan_stay_in_their_rows(rows):
    for dtype in ("f32", "f16", "bf16"):
        x, w = rand(rows, 64, dtype=dtype, seed=1).cuda(), rand(40, 64, dtype=dtype, seed=2).cuda()
        x[1, 5], x[2, 7] = float("nan"), float("inf")
        y = conv.linear(x, w)
        assert y[1].isnan().all() and not y[2].isfinite().any()
        assert y[0].isfinite().all() and y[3:].isfinite().all()


@pytest.mark.parametrize("act", ACTS, ids=lambda a: a[0])
def test_a_nan_shows_in_values_and_gradients(act):
    name, alpha, beta = act
    for rows, dtype in ((4, "bf16"), (4, "f32"), (70, "f16"), (70, "f32")):
        x, w = rand(rows, 32, dtype=dtype, seed=1).cuda(), rand(24, 32, dtype=dtype, seed=2).cuda()
        x[2, 3] = float("nan")
        y, pre = conv.linear(x, w, act=name, alpha=alpha, beta=beta, save=True)
        dx = conv.linear_backward(torch.ones_like(y), x, w, pre, act=name, alpha=alpha, beta=beta, need_dw=False)[0]
        g = conv.gated_ffn(x, w, w.clone(), w.t().contiguous(), act=name, alpha=alpha, beta=beta)
        assert y[2].isnan().all() and g[2].isnan().all() and (name == "identity" or dx[2].isnan().all())
        for t in (y, dx, g):
            assert t[:2].isfinite().all() and t[3:].isfinite().all()


def test_linear_is_the_same_every_time():
    x, w = rand(260, 2000, dtype="bf16", seed=1).cuda(), rand(136, 2000, dtype="bf16", seed=2).cuda()
    first = conv.linear(x, w, act="silu", save=True)
    grads = conv.linear_backward(first[0], x, w, first[1], act="silu", need_dbias=True)
    for _ in range(3):
        y, pre = conv.linear(x, w, act="silu", save=True)
        again = conv.linear_backward(y, x, w, pre, act="silu", need_dbias=True)
        for a, b in zip((y, pre) + again[:3], first + grads[:3]):
            assert torch.equal(a, b)


def gated_case(rows, c_in, hidden, c_out, dtype, act="silu", alpha=0.0, beta=0.0, residual=True, flags=0, seed=0):
    x = rand(rows, c_in, dtype=dtype, seed=seed)
    wg, wu = (rand(hidden, c_in, dtype=dtype, seed=seed + i, scale=c_in ** -0.5) for i in (1, 2))
    wd = rand(c_out, hidden, dtype=dtype, seed=seed + 3, scale=hidden ** -0.5)
    r = rand(rows, c_out, dtype=dtype, seed=seed + 4) if residual else None
    dy = rand(rows, c_out, dtype=dtype, seed=seed + 5, scale=0.1)
    X, WG, WU, WD, R, DY = cuda(x, wg, wu, wd, r, dy)
    kw = dict(act=act, alpha=alpha, beta=beta, flags=flags)
    y, saved = conv.gated_ffn(X, WG, WU, WD, R, save=True, **kw)
    y2 = conv.gated_ffn(X, WG, WU, WD, R, **kw)
    grads = conv.gated_ffn_backward(DY, X, WG, WU, WD, saved, **kw)
    torch.cuda.synchronize()
    assert conv.conv_linear_device_error() == 0
    assert torch.equal(y, y2)
    want = ref.gated64(*wide(x, wg, wu, wd, r), act, alpha, beta, dtype, dy.double())
    for name, got in zip(("y", "dx", "dw_gate", "dw_up", "dw_down"), (y,) + grads):
        ref.check(got, want[name], name)


GATED = [(1, 1, 1, 1), (1, 64, 128, 64), (2, 9, 7, 5), (3, 200, 65, 33), (8, 256, 520, 256), (12, 72, 301, 40),
         (16, 128, 136, 96), (17, 64, 200, 72), (40, 1000, 48, 56), (64, 128, 384, 128), (130, 96, 257, 80),
         (200, 264, 129, 136), (257, 64, 500, 300), (520, 136, 264, 136)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("size", GATED, ids=str)
def test_gated_sizes(size, dtype):
    gated_case(*size, dtype, seed=sum(size))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("act", ACTS, ids=lambda a: a[0])
@pytest.mark.parametrize("rows", [2, 140])
def test_gated_activations(act, dtype, rows):
    gated_case(rows, 40, 88, 56, dtype, *act, residual=False, seed=5)


@pytest.mark.parametrize("flags", [conv.FLAG_LINEAR_FORCE_FFMA, conv.FLAG_LINEAR_NO_FEW_ROWS,
                                   conv.FLAG_LINEAR_UNALIGNED])
def test_gated_other_kernels(flags):
    gated_case(7, 72, 136, 64, "bf16", flags=flags)
    gated_case(150, 72, 136, 64, "f16", flags=flags)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows", [8, 9, 16])
def test_few_rows_on_both_sides_of_the_rule(rows, dtype):
    """From 9 rows on, many outputs (16 bits) and rows of no whole 16-byte pieces (float32) go to the tensor cores."""
    linear_case(rows, 72, 10008, dtype, act="silu", seed=31)
    linear_case(rows, 72, 5000, dtype, seed=32)
    linear_case(rows, 73, 200, dtype, seed=33)
    gated_case(rows, 64, 5008, 40, dtype, seed=34)
    gated_case(rows, 64, 5003, 40, dtype, seed=35)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_few_rows_at_any_address(dtype):
    """16 rows whose size alone would choose the tensor cores, at odd addresses, with scratch and without."""
    x, w = rand(16, 81, dtype=dtype, seed=36).cuda()[:, 1:], rand(6001 * 80 + 1, dtype=dtype, seed=37, scale=0.1).cuda()
    w = w[1:].view(6001, 80)
    want = ref.linear64(*wide(x.cpu(), w.cpu(), None, None), "identity", 0, 0, False, dtype)["y"]
    ref.check(conv.linear(x, w), want)
    y = torch.empty(16, 6001, dtype=ref.TORCH[dtype], device="cuda")
    dense = x.contiguous()
    p = conv.make_linear_problem(16, 80, 6001, dtype=dtype)
    n = conv.conv_linear_scratch_bytes(p)
    conv.conv_linear_forward(p, dense, w, None, None, y, None, torch.empty(n, dtype=torch.uint8, device="cuda") if n else None, n)
    ref.check(y, want)


def test_gated_some_gradients_and_no_rows():
    x, wg, wu, wd = (t.cuda() for t in (rand(70, 48, dtype="bf16", seed=1), rand(96, 48, dtype="bf16", seed=2),
                                        rand(96, 48, dtype="bf16", seed=3), rand(48, 96, dtype="bf16", seed=4)))
    y, saved = conv.gated_ffn(x, wg, wu, wd, save=True)
    full = conv.gated_ffn_backward(y, x, wg, wu, wd, saved)
    dx = conv.gated_ffn_backward(y, x, wg, wu, wd, saved, need_dw=False)
    dw = conv.gated_ffn_backward(y, x, wg, wu, wd, saved, need_dx=False)
    assert torch.equal(dx[0], full[0]) and dx[1:] == (None, None, None)
    assert dw[0] is None and all(torch.equal(a, b) for a, b in zip(dw[1:], full[1:]))
    # one of the two projections' gradients alone
    p = conv.make_gated_problem(70, 48, 96, 48, dtype="bf16")
    n = conv.conv_gated_backward_scratch_bytes(p)
    scratch = torch.empty(n, dtype=torch.uint8, device="cuda")
    for i in (1, 2):
        one = torch.empty_like(wg)
        conv.conv_gated_backward(p, x, wg, wu, wd, saved, y, None, one if i == 1 else None, one if i == 2 else None, None,
                                 scratch, n)
        assert torch.equal(one, full[i])
    e = x[:0]
    y, saved = conv.gated_ffn(e, wg, wu, wd, save=True)
    none = conv.gated_ffn_backward(y, e, wg, wu, wd, saved)
    assert y.shape == (0, 48) and none[0].shape == (0, 48) and not any(t.any() for t in none[1:])


def test_gradients_against_differences():
    """The gradients along a direction, against central differences of the float64 definition (step 1e-4: its own error
    is some 1e-8 of the terms), within the sum of the values' bounds."""
    step = 1e-4
    x, w, b = rand(6, 20, dtype="f32", seed=1), rand(9, 20, dtype="f32", seed=2, scale=0.3), rand(9, dtype="f32", seed=3)
    dy = rand(6, 9, dtype="f32", seed=4)
    X, W, B, DY = cuda(x, w, b, dy)
    for act, al, be in ACTS:
        _, pre = conv.linear(X, W, B, act=act, alpha=al, beta=be, save=True)
        got = conv.linear_backward(DY, X, W, pre, act=act, alpha=al, beta=be, need_dbias=True)
        x64, w64, b64, dy64 = wide(x, w, b, dy)
        z = ref.linear64(x64, w64, b64, None, act, al, be, False, "f32")["z"]
        bounds = ref.linear_backward64(dy64, x64, w64, *z, act, al, be, False, "f32")
        if any((z[0] - c).abs().min() < 1e-2 for c in ref.corners(act, al, be)):
            continue  # a difference across a corner is no slope

        def loss(x_, w_, b_):
            return (ref.act64(x_ @ w_.T + b_, act, al, be) * dy64).sum()
        for i, name in enumerate(("dx", "dw", "dbias")):
            d = torch.randn((x64, w64, b64)[i].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64)
            args = [x64, w64, b64]
            up, down = list(args), list(args)
            up[i], down[i] = args[i] + step * d, args[i] - step * d
            slope = (loss(*up) - loss(*down)) / (2 * step)
            mine = (got[i].cpu().double() * d).sum()
            assert abs(mine - slope) <= (bounds[name][1] * d.abs()).sum() + 1e-5, (act, name)
    wg, wu, wd = (rand(*s, dtype="f32", seed=9 + i, scale=0.3) for i, s in enumerate([(14, 20), (14, 20), (9, 14)]))
    G, U, D = cuda(wg, wu, wd)
    for act in ("silu", "gelu", "gelu_tanh", "tanh"):
        _, saved = conv.gated_ffn(X, G, U, D, act=act, save=True)
        got = conv.gated_ffn_backward(DY, X, G, U, D, saved, act=act)
        args = wide(x, wg, wu, wd)
        bounds = ref.gated64(*args, None, act, 0, 0, "f32", dy.double())

        def block(x_, g_, u_, d_):
            return (((ref.act64(x_ @ g_.T, act) * (x_ @ u_.T)) @ d_.T) * dy.double()).sum()
        for i, name in enumerate(("dx", "dw_gate", "dw_up", "dw_down")):
            d = torch.randn(args[i].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64)
            up, down = list(args), list(args)
            up[i], down[i] = args[i] + step * d, args[i] - step * d
            slope = (block(*up) - block(*down)) / (2 * step)
            mine = (got[i].cpu().double() * d).sum()
            assert abs(mine - slope) <= (bounds[name][1] * d.abs()).sum() + 1e-5, (act, name)


# ---- clipping ---------------------------------------------------------------
def clip64(tensors, max_norm, eps):
    norm = torch.stack([t.double().square().sum() for t in tensors]).sum().sqrt() if tensors else torch.tensor(0.0)
    scale = min(1.0, float(max_norm / (norm + eps)) if float(norm) + eps else 1.0)
    return norm, scale


def check_clip(tensors, max_norm, eps=1e-6, out=None, **kw):
    host = [t.cpu() for t in tensors]
    norm, scale = clip64(host, max_norm, eps)
    got = conv.clip_grad_norm(tensors, max_norm, eps=eps, out=out, **kw)
    torch.cuda.synchronize()
    # at most 32 float32 roundings per group of squares, then float64: 2^-19 of the sum, half of that of its root
    assert abs(got.item() - norm.item()) <= 2.0 ** -19 * norm.item() + 1e-45, (got.item(), norm.item())
    names = {torch.float32: "f32", torch.float16: "f16", torch.bfloat16: "bf16"}
    for t, o in zip(host, tensors if out is None else out):
        want = t.double() * scale
        d = names[t.dtype]
        ref.check(o, (want, (2.0 ** -18 + ref.HALF_UNIT[d]) * want.abs() + ref.TINY[d]), tuple(t.shape))
    if out is not None:
        assert all(torch.equal(a.cpu(), b) for a, b in zip(tensors, host))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("bound", [0.5, 1e6])
def test_clip_sizes(dtype, in_place, bound):
    sizes = [1, 3, 7, 8, 9, 16, 100, 1000, 16383, 16384, 16385, 16400, 40000, 70001, 0, 5]
    ts = [rand(n, dtype=dtype, seed=i).cuda() for i, n in enumerate(sizes)]
    check_clip(ts, bound, out=None if in_place else [torch.full_like(t, 3.0) for t in ts])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_clip_views_at_every_offset(dtype):
    flat = rand(40000, dtype=dtype, seed=1).cuda()
    out = torch.full_like(flat, 9.0)
    for shift in (0, 1, 3):  # inputs and outputs that lie differently within 16 bytes
        ins, outs, at = [], [], 0
        for n in (5, 17, 1, 64, 16391, 9, 3, 20000):
            ins.append(flat[at:at + n])
            outs.append(out[at + shift:at + n + shift])
            at += n + 1
        check_clip(ins, 1.0, out=outs)


def test_clip_many_tensors_of_mixed_types():
    g = torch.Generator().manual_seed(3)
    for count in (63, 64, 65, 1024, 2300):
        sizes = torch.randint(1, 300, (count,), generator=g).tolist()
        ts = [rand(n, dtype=("f32", "f16", "bf16")[i % 3], seed=i).cuda() for i, n in enumerate(sizes)]
        check_clip(ts, 2.0)
        check_clip(ts, 1.0, out=[torch.empty_like(t) for t in ts])


@pytest.mark.parametrize("dtype,low,high", [("f32", 1e-30, 1e30), ("bf16", 1e-30, 1e30), ("f16", 1e-7, 6e4)])
def test_clip_neither_overflows_nor_vanishes(dtype, low, high):
    for scale in (low, high):
        check_clip([(rand(5000, dtype="f32", seed=1).clamp(-1, 1) * scale).to(ref.TORCH[dtype]).cuda()], scale, eps=0.0)
    mixed = torch.ones(5000, dtype=ref.TORCH[dtype])
    mixed[::2] = high
    check_clip([mixed.cuda(), (torch.ones(77) * low).to(ref.TORCH[dtype]).cuda()], high, eps=0.0)
    tiny = torch.full((1000,), 2.0 ** -149 if dtype == "f32" else 2.0 ** -133 if dtype == "bf16" else 2.0 ** -24,
                      dtype=ref.TORCH[dtype]).cuda()
    norm = conv.clip_grad_norm([tiny.clone()], 1e30)
    want = tiny.cpu().double().norm().item()
    assert abs(norm.item() - want) <= 2.0 ** -19 * want + 2.0 ** -149


def test_clip_zero_nan_and_infinity():
    z = torch.zeros(100, device="cuda")
    assert conv.clip_grad_norm([z], 1.0).item() == 0 and not z.any()
    assert conv.clip_grad_norm([z], 0.0, eps=0.0).item() == 0 and not z.any()
    a, b = torch.ones(100, device="cuda"), torch.ones(20000, device="cuda", dtype=torch.bfloat16)
    b[777] = float("inf")
    assert conv.clip_grad_norm([a, b], 1.0).item() == float("inf")
    assert not a.any() and b[777].isnan() and not b[:777].any() and not b[778:].any()
    a, b = torch.ones(100, device="cuda"), torch.ones(20000, device="cuda", dtype=torch.float16)
    b[5] = float("nan")
    assert conv.clip_grad_norm([a, b], 1.0).isnan() and a.isnan().all() and b.isnan().all()


def test_clip_the_norm_alone():
    t = rand(30000, dtype="bf16", seed=1).cuda()
    before = t.clone()
    norm = torch.empty((), device="cuda")
    n = conv.conv_clip_scratch_bytes([30000])
    scratch = torch.empty(n, dtype=torch.uint8, device="cuda")
    conv.conv_clip_grads([t], None, [30000], ["bf16"], 1.0, 1e-6, norm, scratch, n)
    want = before.double().norm().item()
    assert torch.equal(t, before) and abs(norm.item() - want) <= 2.0 ** -19 * want
    conv.conv_clip_grads([], None, [], [], 1.0, 1e-6, norm, scratch, n)
    assert norm.item() == 0


# ---- as programs use them ---------------------------------------------------
def test_the_last_round_of_tiles_in_ranges():
    """Plans whose last tiles are cut into k ranges, for each operand order and for the gated products."""
    found = set()
    for rows, c_in, c_out, dtype in ((40, 3000, 300, "bf16"), (3328, 2048, 1536, "bf16"), (60, 2000, 200, "f32"),
                                     (1300, 1000, 1600, "f32"), (700, 2300, 2500, "f16")):
        p = conv.make_linear_problem(rows, c_in, c_out, dtype=dtype)
        for i in range(3):
            d = conv.conv_linear_describe_plan(p, i, 152)
            if "split=1 " not in d:
                found.add((dtype == "f32", " whole=0 " in d))
        linear_case(rows, c_in, c_out, dtype, act="silu", seed=rows)
    assert found == {(False, False), (False, True), (True, False), (True, True)}
    gated_case(90, 1500, 700, 300, "f16", seed=3)
    gated_case(3328, 1024, 768, 64, "bf16", seed=4)


def test_other_tile_widths():
    for c_out in (70, 130, 200, 260, 330, 450):
        linear_case(600, 192, c_out, "bf16", act="gelu", seed=c_out)


def test_in_a_graph():
    x, w, b = (t.cuda() for t in (rand(300, 200, dtype="bf16", seed=1), rand(250, 200, dtype="bf16", seed=2, scale=0.1),
                                  rand(250, dtype="bf16", seed=3)))
    wg, wu, wd = (t.cuda() for t in (rand(264, 200, dtype="bf16", seed=4, scale=0.1),
                                     rand(264, 200, dtype="bf16", seed=5, scale=0.1),
                                     rand(200, 264, dtype="bf16", seed=6, scale=0.1)))

    def step():
        y, pre = conv.linear(x, w, b, act="silu", save=True)
        grads = conv.linear_backward(y, x, w, pre, act="silu", need_dbias=True)[:3]
        z, saved = conv.gated_ffn(x, wg, wu, wd, x, save=True)
        more = conv.gated_ffn_backward(z, x, wg, wu, wd, saved)
        one = conv.gated_ffn(x[:1], wg, wu, wd, x[:1])
        outs = [torch.empty_like(t) for t in grads + more]
        norm = conv.clip_grad_norm(grads + more, 1.0, out=outs)
        return [y, z, one, norm, *outs]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in (7, 8):
        x.copy_(rand(300, 200, dtype="bf16", seed=seed))
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(step(), captured):
            assert torch.equal(a, c)


def test_two_streams_at_once():
    """Calls on two streams, each with its own scratch, overlap and give what they give alone."""
    cases = []
    for i in range(2):
        x, w = rand(50, 6000, dtype="bf16", seed=i).cuda(), rand(64, 6000, dtype="bf16", seed=9 + i, scale=0.02).cuda()
        cases.append((x, w, conv.linear(x, w)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[] for _ in cases]
    for _ in range(20):
        for (x, w, _), s, o in zip(cases, streams, outs):
            o.append(conv.linear(x, w, stream=s))
    torch.cuda.synchronize()
    for (_, _, want), o in zip(cases, outs):
        assert all(torch.equal(want, y) for y in o)


def test_two_host_threads_on_one_stream():
    """Their calls share the stream's scratch; each call's launches stay together."""
    import threading
    cases = [(rand(50, 6000, dtype="bf16", seed=i).cuda(), rand(64, 6000, dtype="bf16", seed=9 + i, scale=0.02).cuda())
             for i in range(2)]
    want = [conv.linear(x, w) for x, w in cases]
    outs = [[], []]

    def work(i):
        for _ in range(100):
            outs[i].append(conv.linear(*cases[i]))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert len(o) == 100 and all(torch.equal(w, y) for y in o)


def test_offsets_past_32_bits():
    big = torch.empty(600 << 22, dtype=torch.bfloat16, device="cuda")  # 2.5e9 elements
    x = big.view(600, 1 << 22)[:, 5000:5080]
    x.copy_(rand(600, 80, dtype="bf16", seed=1))
    w = rand(40, 80, dtype="bf16", seed=2, scale=0.1).cuda()
    y = conv.linear(x, w, out=big.view(600, 1 << 22)[:, 9000:9040])
    dx, dw, _, _ = conv.linear_backward(y, x, w)
    few = conv.linear(x[592:], w)
    want = ref.linear64(*wide(x.cpu(), w.cpu(), None, None), "identity", 0, 0, False, "bf16")
    ref.check(y, want["y"])
    ref.check(few, tuple(t[592:] for t in want["y"]))
    back = ref.linear_backward64(*wide(y.cpu(), x.cpu(), w.cpu()), *want["z"], "identity", 0, 0, False, "bf16")
    ref.check(dx, back["dx"])
    ref.check(dw, back["dw"])
    flat = big[:(1 << 31) + 77]
    flat.zero_()
    flat[[3, 1 << 30, (1 << 31) - 1, 1 << 31, (1 << 31) + 76]] = 2.0
    norm = conv.clip_grad_norm([flat], 1.0, eps=0.0)
    assert abs(norm.item() - 20 ** 0.5) < 1e-5
    assert (flat[[3, 1 << 30, (1 << 31) - 1, 1 << 31, (1 << 31) + 76]].float() - 2 / 20 ** 0.5).abs().max() < 2e-3
    del big, x, flat


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_the_example(dtype):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_block.py")
    spec = importlib.util.spec_from_file_location("train_block", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, norms, apart = example.train(12, dtype)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses  # a plain gradient step of a clipped size
    assert norms[0] > 0.5 and all(n == n for n in norms)
    # two float32 sums of 320 terms of h (their absolute values sum to below 64 here), and one rounding each
    assert apart <= 2 * 320 * 2.0 ** -23 * 64 + 2 * ref.HALF_UNIT[dtype] * 16


def test_refusals_of_tensors():
    x, w = torch.zeros(4, 8, device="cuda"), torch.zeros(6, 8, device="cuda")
    for bad in (dict(bias=torch.zeros(5, device="cuda")), dict(residual=torch.zeros(4, 5, device="cuda")),
                dict(out=torch.zeros(5, 6, device="cuda")), dict(bias=torch.zeros(6, device="cuda").half()),
                dict(residual=torch.zeros(4, 6))):
        with pytest.raises(ValueError):
            conv.linear(x, w, **bad)
    with pytest.raises(ValueError):
        conv.linear(x, torch.zeros(6, 9, device="cuda"))
    with pytest.raises(ValueError):
        conv.linear_backward(torch.zeros(4, 6, device="cuda"), x, w, act="silu")      # no pre
    with pytest.raises(KeyError):
        conv.linear(x, w, act="softmax")
    with pytest.raises(conv.ConvError, match="ALIAS"):
        conv.linear(x, w, out=torch.as_strided(w, (4, 6), (8, 1)))
    with pytest.raises(conv.ConvError, match="SCRATCH"):
        conv.linear(torch.zeros(64, 4096, device="cuda"), torch.zeros(64, 4096, device="cuda"),
                    scratch=torch.empty(16, dtype=torch.uint8, device="cuda"))
    g = torch.zeros(12, 8, device="cuda")
    with pytest.raises(ValueError):
        conv.gated_ffn(x, g, torch.zeros(11, 8, device="cuda"), torch.zeros(8, 12, device="cuda"))
    with pytest.raises(ValueError):
        conv.gated_ffn(x, g, g.clone(), torch.zeros(12, 8, device="cuda").t())
    y, saved = conv.gated_ffn(x, g, g.clone(), torch.zeros(8, 12, device="cuda"), save=True)
    with pytest.raises(ValueError):
        conv.gated_ffn_backward(y, x, g, g.clone(), torch.zeros(8, 12, device="cuda"), saved[:-256])
    with pytest.raises(ValueError):
        conv.clip_grad_norm([], 1.0)
    with pytest.raises(ValueError):
        conv.clip_grad_norm([x, w.t()], 1.0)
    with pytest.raises(TypeError):
        conv.clip_grad_norm([x.double()], 1.0)
    with pytest.raises(ValueError):
        conv.clip_grad_norm([x], 1.0, out=[w])
    with pytest.raises(conv.ConvError, match="ALIAS"):
        conv.clip_grad_norm([x, x], 1.0)
    with pytest.raises(conv.ConvError, match="ARG"):
        conv.clip_grad_norm([x], -1.0)


def queried(n):
    return (torch.empty(n, dtype=torch.uint8, device="cuda") if n else None), n


@pytest.mark.parametrize("rows", [16, 64])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_unaligned_operands_with_the_scratch_of_aligned_ones(dtype, rows):
    """Sums long enough for the CUDA-core kernel to cut, which it must not without scratch: each pass, with exactly what
    its query asks for an aligned call."""
    k, n, hidden = 1024, 1024, 640

    def off(*shape, seed, scale=1.0):  # one value off a 16-byte boundary
        t = rand(shape[0] * shape[1] + 1, dtype=dtype, seed=seed, scale=scale).cuda()
        return t[1:].view(shape)
    x, w, dy = off(rows, k, seed=1), off(n, k, seed=2, scale=k ** -0.5), off(rows, n, seed=3, scale=0.1)
    new = lambda *shape: torch.full(shape, 7.0, dtype=ref.TORCH[dtype], device="cuda")  # noqa: E731
    for act in ("identity", "silu"):
        p = conv.make_linear_problem(rows, k, n, dtype=dtype, act=act)
        y, pre = new(rows, n), torch.empty(rows, n, device="cuda")
        conv.conv_linear_forward(p, x, w, None, None, y, pre, *queried(conv.conv_linear_scratch_bytes(p)))
        want = ref.linear64(*wide(x.cpu(), w.cpu(), None, None), act, 0, 0, False, dtype)
        ref.check(y, want["y"], "y")
        ref.check(pre, want["z"], "pre")
        outs = new(rows, k), new(n, k), new(n), new(rows, n)
        conv.conv_linear_backward(p, x, w, pre, dy, *outs, *queried(conv.conv_linear_backward_scratch_bytes(p)))
        back = ref.linear_backward64(*wide(dy.cpu(), x.cpu(), w.cpu()), *want["z"], act, 0, 0, False, dtype)
        for name, got in zip(("dx", "dw", "dbias", "dresidual"), outs):
            ref.check(got, back[name], (act, name))
    p = conv.make_gated_problem(rows, k, hidden, n, dtype=dtype)
    wg, wu, wd = (off(hidden, k, seed=4, scale=k ** -0.5), off(hidden, k, seed=5, scale=k ** -0.5),
                  off(n, hidden, seed=6, scale=hidden ** -0.5))
    want = ref.gated64(*wide(x.cpu(), wg.cpu(), wu.cpu(), wd.cpu()), None, "silu", 0, 0, dtype, dy.cpu().double())
    saved = torch.empty(conv.conv_gated_saved_bytes(p), dtype=torch.uint8, device="cuda")
    for keep in (None, saved):
        y = new(rows, n)
        conv.conv_gated_forward(p, x, wg, wu, wd, None, y, keep, *queried(conv.conv_gated_scratch_bytes(p)))
        ref.check(y, want["y"], "y")
    outs = new(rows, k), new(hidden, k), new(hidden, k), new(n, hidden)
    conv.conv_gated_backward(p, x, wg, wu, wd, saved, dy, *outs, *queried(conv.conv_gated_backward_scratch_bytes(p)))
    for name, got in zip(("dx", "dw_gate", "dw_up", "dw_down"), outs):
        ref.check(got, want[name], name)
    torch.cuda.synchronize()
    assert conv.conv_linear_device_error() == 0


def tiny_operands(low, rows, more):
    """linear and its gradients with operands of 2^-low beside large ones, whose products are of ordinary size; `more`: of
    two factors, what is added to the bound of their product."""
    e, high = 2.0 ** -low, 2.0 ** min(low, 122)
    x, w = rand(rows, 200, dtype="f32", seed=low, scale=e), rand(90, 200, dtype="f32", seed=low + 1, scale=high)
    dy = rand(rows, 90, dtype="f32", seed=low + 2, scale=e)
    X, W, DY = cuda(x, w, dy)
    x, w, dy = wide(x, w, dy)
    y, pre = conv.linear(X, W, act="relu", save=True)
    want = ref.linear64(x, w, None, None, "relu", 0, 0, False, "f32")
    z = want["z"][0], want["z"][1] + more(x, w)
    ref.check(pre, z, (rows, "pre"))
    ref.check(y, (want["y"][0], want["y"][1] + 2 * more(x, w)), (rows, "y"))
    grads = conv.linear_backward(DY, X, W, pre, act="relu", need_dw=False, need_dbias=True)
    back = ref.linear_backward64(dy, x, w, *z, "relu", 0, 0, False, "f32")
    ref.check(grads[0], (back["dx"][0], back["dx"][1] + 2 * more(dy, w.T)), (rows, "dx"))
    ref.check(grads[2], back["dbias"], (rows, "dbias"))
    big = rand(rows, 90, dtype="f32", seed=low + 3, scale=high)
    back = ref.linear_backward64(big.double(), x, w, *z, "identity", 0, 0, False, "f32")
    ref.check(conv.linear_backward(big.cuda(), X, W, need_dx=False)[1],
              (back["dw"][0], back["dw"][1] + 2 * more(big.double().T, x.T)), (rows, "dw"))


@pytest.mark.parametrize("low", [100, 112, 118, 122])
def test_float32_operands_of_every_magnitude(low):
    """The bound of float32 sums holds for small operands as for others, in each pass and on both sides of the kernel for
    few rows."""
    for rows in (5, 70):
        tiny_operands(low, rows, lambda a, b: 0.0)
    scale, e = 2.0 ** min(low, 118), 2.0 ** -low
    x, dy = rand(70, 64, dtype="f32", seed=1, scale=e), rand(70, 40, dtype="f32", seed=2, scale=e)
    wg, wu = (rand(136, 64, dtype="f32", seed=i, scale=scale / 8) for i in (3, 4))
    wd = rand(40, 136, dtype="f32", seed=5, scale=2.0 ** 110)
    args = cuda(x, wg, wu, wd)
    y, saved = conv.gated_ffn(*args, save=True)
    grads = conv.gated_ffn_backward(dy.cuda(), *args, saved)
    want = ref.gated64(*wide(x, wg, wu, wd), None, "silu", 0, 0, "f32", dy.double())
    for name, got in zip(("y", "dx", "dw_gate", "dw_up", "dw_down"), (y,) + grads):
        ref.check(got, want[name], name)


@pytest.mark.parametrize("low", [126, 132, 140, 149])
def test_float32_subnormal_operands(low):
    """Subnormal operands count to two units of their last place: 2^-148 of the other factors' absolute values."""
    for rows in (5, 70):
        tiny_operands(low, rows, lambda a, b: 2.0 ** -148 * (a.abs().sum(1)[:, None] + b.abs().sum(1)))


@pytest.mark.parametrize("terms", [1, 2])
def test_float32_products_near_the_top_of_the_range(terms):
    """Products up to a half of the range's end (one term) and sums that stay below it (two): nothing of the parts'
    products overflows where the sum does not.  Values at the very end, which round up to infinity as bfloat16."""
    g = torch.Generator().manual_seed(terms)

    def signed(rows, scale):
        v = 1 + torch.rand(rows, terms, generator=g, dtype=torch.float64)
        v[: rows // 2] = 1 + 2.0 ** -8 * torch.randint(1, 4, (rows // 2, terms), generator=g)  # the largest remainders
        return (v * scale * (2 * torch.randint(0, 2, (rows, terms), generator=g) - 1)).float()
    x, w = signed(60, 2.0 ** 63), signed(50, 2.0 ** (63 - terms))
    want = ref.linear64(*wide(x, w, None, None), "identity", 0, 0, False, "f32")["y"]
    ref.check(conv.linear(*cuda(x, w)), want)
    top = torch.finfo(torch.float32).max
    x = (top * (1 - 2.0 ** -torch.arange(1, 25, dtype=torch.float64))).float().repeat(3)[:, None].repeat(1, terms)
    x[1::2] *= -1
    w = rand(30, terms, dtype="f32", seed=7).clamp(-1, 1) / terms
    ref.check(conv.linear(*cuda(x, w)), ref.linear64(*wide(x, w, None, None), "identity", 0, 0, False, "f32")["y"])


def same_specials(got, want, size, terms, what):
    """NaN and infinities where float64, rounded to float32, has them; elsewhere within the bound of a float32 sum of
    `terms` terms, whose absolute values' sum is `size` (within 1% of the range's end, it may be infinite)."""
    want = want.float().double()
    got, finite = got.cpu().double(), want.isfinite() & (size < 0.99 * torch.finfo(torch.float32).max)
    assert torch.equal(got.isnan(), want.isnan()), what
    assert torch.equal(got[want.isinf()], want[want.isinf()]), what
    bound = (terms + 3) * 2.0 ** -23 * size + 2.0 ** -149
    assert finite.any() and ((got - want).abs() <= bound)[finite].all(), what


@pytest.mark.parametrize("rows", [5, 12, 70, 200])
@pytest.mark.parametrize("k", [64, 200, 77])
def test_float32_infinities_are_those_of_the_formula(rows, k):
    """An infinity among the operands times anything but zero is one, whatever the kernel: 12 rows of 77 and 70 rows go to
    the tensor cores.  Factors of every size down to the smallest subnormal, and zeros, which make NaN."""
    inf = float("inf")
    x, w = rand(rows, k, dtype="f32", seed=1), rand(90, k, dtype="f32", seed=2)
    w[3, 5], w[4, 5], w[5, 5], w[6, 5], w[7, 5] = 2.0 ** -149, -(2.0 ** -140), 0.0, 1e-30, -3e38
    w[8, 5] = w[8, 60] = 1.0
    x[1, 5], x[2, 5], x[3, 60] = inf, -inf, inf
    x[4, 5], x[4, 60] = inf, -inf
    w[9, 7], w[10, 7], w[11, 7] = inf, -inf, float("nan")
    x[:, 7] = x[:, 7].abs() + 0.5
    dy = rand(rows, 90, dtype="f32", seed=3)
    dy[0, 9], dy[1, 30], dy[2, 40] = 0.0, -inf, inf
    X, W, DY = cuda(x, w, dy)
    x, w, dy = wide(x, w, dy)
    finite = lambda t: torch.nan_to_num(t, 0.0, 0.0, 0.0).abs()  # noqa: E731
    z, size = x @ w.T, finite(x) @ finite(w).T
    same_specials(conv.linear(X, W), z, size, k, "y")
    same_specials(conv.linear(X, W, act="relu"), torch.where(z < 0, torch.zeros_like(z), z), size, k, "relu")
    dx, dw, _, _ = conv.linear_backward(DY, X, W)
    same_specials(dw, dy.T @ x, finite(dy).T @ finite(x), rows, "dw")
    w[9:12, 7], x[1:5, 5], x[3:5, 60] = 1.0, 1.0, 1.0
    dx = conv.linear_backward(DY, x.float().cuda(), w.float().cuda(), need_dw=False)[0]
    same_specials(dx, dy @ w, finite(dy) @ finite(w), 90, "dx")
    # the gated block: an infinite g or u, then an infinite row of h
    wg, wu, wd = rand(80, k, dtype="f32", seed=4), rand(80, k, dtype="f32", seed=5), rand(50, 80, dtype="f32", seed=6)
    x[1, 5], x[2, 5] = inf, -inf
    got = conv.gated_ffn(x.float().cuda(), *cuda(wg, wu, wd), act="leaky_relu", alpha=0.5)
    wg, wu, wd = wide(wg, wu, wd)
    g, u = x @ wg.T, x @ wu.T
    a = torch.where(g >= 0, g, 0.5 * g)
    size = ((finite(x) @ wg.abs().T) * (finite(x) @ wu.abs().T)) @ wd.abs().T
    same_specials(got, (a * u) @ wd.T, size, 2 * k + 80, "gated")


def test_no_rows_among_leading_dimensions():
    x, w, dy = (torch.zeros(*s, device="cuda") for s in ((2, 0, 8), (6, 8), (2, 0, 6)))
    assert conv.linear(x, w).shape == (2, 0, 6)
    dx, dw, db, _ = conv.linear_backward(dy, x, w, need_dbias=True)
    assert dx.shape == x.shape and dw.shape == w.shape and not dw.any() and not db.any()
    g, d = torch.ones(12, 8, device="cuda"), torch.ones(6, 12, device="cuda")
    y, saved = conv.gated_ffn(x, g, g.clone(), d, save=True)
    grads = conv.gated_ffn_backward(dy, x, g, g.clone(), d, saved)
    assert y.shape == dy.shape and grads[0].shape == x.shape and not any(t.any() for t in grads[1:])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_dresidual_of_rows_far_apart(dtype):
    """dy's rows more than 2^31 bytes apart, every output: what is dy itself comes out bit for bit."""
    size = 4 if dtype == "f32" else 2
    stride = (1 << 31) // size + 8
    flat = torch.zeros(stride + 24, dtype=ref.TORCH[dtype], device="cuda")
    dy = torch.as_strided(flat, (2, 24), (stride, 1))
    dy.copy_(rand(2, 24, dtype=dtype, seed=1))
    x, w = rand(2, 40, dtype=dtype, seed=2).cuda(), rand(24, 40, dtype=dtype, seed=3, scale=0.2).cuda()
    for last, act in ((False, "identity"), (True, "relu"), (False, "relu")):
        r = rand(2, 24, dtype=dtype, seed=4).cuda()
        _, pre = conv.linear(x, w, None, r, act=act, residual_last=last, save=True)
        grads = conv.linear_backward(dy, x, w, pre, act=act, residual_last=last, need_dbias=True, need_dresidual=True)
        host = wide(*(t.cpu() for t in (dy, x, w, r)))
        want = ref.linear64(host[1], host[2], None, host[3], act, 0, 0, last, dtype)
        back = ref.linear_backward64(host[0], host[1], host[2], *want["z"], act, 0, 0, last, dtype)
        for name, got in zip(("dx", "dw", "dbias", "dresidual"), grads):
            ref.check(got, back[name], (act, last, name))
        if last or act == "identity":
            assert torch.equal(grads[3], dy)
    del flat, dy


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_dresidual_of_the_identity_is_dy(dtype):
    """Every value of 16 bits but NaN, and strided rows of odd widths."""
    if dtype != "f32":
        values = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(ref.TORCH[dtype])
        values = values[~values.isnan()]
    else:
        values = rand(70000, dtype="f32", seed=5) * 2.0 ** torch.randint(-149, 127, (70000,), generator=torch.Generator().manual_seed(1))
    for rows, cols, pad in ((100, 300, 0), (77, 301, 5), (5, 1000, 24), (1, 33, 0)):
        dy = values[:rows * (cols + pad)].view(rows, cols + pad)[:, :cols].cuda()
        x, w = torch.zeros(rows, 8, dtype=dy.dtype, device="cuda"), torch.zeros(cols, 8, dtype=dy.dtype, device="cuda")
        got = conv.linear_backward(dy, x, w, need_dx=False, need_dw=False, need_dresidual=True)[3]
        assert torch.equal(got, dy) and torch.equal(got.signbit(), dy.signbit())


def test_the_default_stream_by_its_number():
    """stream=0 is the legacy default stream, as a handle and as a stream object: work before and after it keeps its order."""
    from implicit_gemm_cnn_gb300 import dense
    big = torch.randn(8192, 8192, device="cuda")
    values, w = rand(64, 256, dtype="bf16", seed=1).cuda(), rand(40, 256, dtype="bf16", seed=2, scale=0.1).cuda()
    want = conv.linear(values, w)
    for stream in (0, torch.cuda.default_stream(), torch.cuda.default_stream().cuda_stream):
        assert dense._On(0, stream).handle == 0
    x = torch.zeros_like(values)
    torch.cuda.synchronize()
    for _ in range(10):
        big = big @ big * 1e-3  # some milliseconds before x is written
    x.copy_(values)
    y = conv.linear(x, w, stream=0)
    norm = conv.clip_grad_norm([x], 0.0, stream=0)  # x is read, then made zero
    torch.cuda.synchronize()
    assert torch.equal(y, want) and norm.item() > 0 and not x.any()
