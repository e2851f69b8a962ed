"""The row operators where float32 runs out of bits or range: means far from the
values' spread, rows at the ends of float32."""
import pytest
import torch

import implicit_gemm_cnn_gb300 as conv
import rows_ref as ref
from dense_ref import TORCH, check, rounded

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

TYPES = ["f32", "f16", "bf16"]
U = ref.U


def normal(*shape, dtype, seed, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * scale + shift).to(TORCH[dtype])


def nearly_constant(rows, width, dtype):
    """Rows of one value but for a few that are its last place larger: the mean lies between two float32 values, and what
    is left of the other values is far below the mean's rounding."""
    value, place = {"f32": (4096.0, 2.0 ** -11), "f16": (1024.0, 1.0), "bf16": (256.0, 2.0)}[dtype]
    x = torch.full((rows, width), value, dtype=torch.float64)
    for r in range(rows):
        x[r, (37 * r) % width] += place
        x[r, (11 * r + 5) % width] += place
    return x.to(TORCH[dtype])


# a warp to a row, a block, accesses of one value, rows too wide for registers (no powers of two: their means are exact)
NEARLY = [(700, 520, 0), (3, 4104, 0), (3, 1003, 0), (2, 16376, 0), (2, 40000, 0), (3, 2056, conv.FLAG_NORM_STREAM)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width,flags", NEARLY)
def test_norm_of_nearly_constant_rows(rows, width, flags, dtype):
    """Both means are taken off one after the other in every type, so the bound is float32's (that of 16-bit results in
    rows_ref has U |mean| for one rounded mean), and a rounding to the type."""
    x = nearly_constant(rows, width, dtype)
    w, b = (normal(width, dtype=dtype, seed=s, scale=0.3, shift=1.0) for s in (1, 2))
    for weight, bias in ((None, None), (w, b)):
        y = conv.layer_norm(x.cuda(), *(None if t is None else t.cuda() for t in (weight, bias)), flags=flags)
        want, err = ref.norm64(x.double(), *(None if t is None else t.double() for t in (weight, bias)), 1e-5, "f32")["y"]
        check(y, rounded(want, err, dtype), "y")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size,grad", [(1e-18, 1e4), (1e18, 1e-7)])
@pytest.mark.parametrize("rows,width,flags", [(5, 64, 0), (700, 96, 0), (3, 1500, 0), (4, 77, 0), (3, 300, conv.FLAG_NORM_STREAM)])
def test_norm_gradients_of_tiny_and_huge_rows(rows, width, flags, size, grad, dtype):
    """rstd of 1e18 and 1e-18: its square, times c2, is no factor that float32 has, while every gradient is.  (A row's sum of
    squared differences has to fit float32: that of 1500 values of 1e18, 1.5e39, is past 2^128.)"""
    if size > 1:
        size = size * min(1.0, 100 / width) ** 0.5
    x, dy = (normal(rows, width, dtype=dtype, seed=s, scale=k) for s, k in ((1, size), (2, grad)))
    w = normal(width, dtype=dtype, seed=3, scale=0.3, shift=1.0)
    _, stats = conv.layer_norm(x.cuda(), w.cuda(), eps=0.0, save=True, flags=flags)
    got = conv.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), stats, flags=flags)
    f = ref.norm64(x.double(), w.double(), None, 0.0, dtype)
    want = ref.norm_backward64(dy.double(), f, w.double(), dtype)
    for name, g in zip(("dx", "dweight", "dbias"), got):
        check(g, want[name], name)


def gradients64(x, dy, w, eps, dtype):
    """The gradients, with bounds for a backward pass that takes the saved mean's rounding out of xhat again: the mean of the
    differences to that mean is summed as the two other sums are, and taken off."""
    n = x.shape[1]
    k = ref.depth(n)
    f = ref.norm64(x, w, None, eps, "f32")
    (h, _), (r, er) = f["h"], f["r"]
    mean = x.mean(1, keepdim=True)
    spread = (x - mean).abs() + U * mean.abs() + k * U * x.abs().mean(1, keepdim=True)
    # of a difference: its own rounding and its product's, then what was taken off: the sum's, and the differences' in it
    ec = 3 * U * spread + (k + 5) * U * spread.mean(1, keepdim=True)
    eh = r * ec + spread * er + 2 * U * h.abs()
    return ref.norm_backward64(dy, {"h": (h, eh), "r": (r, er)}, w, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width,flags", NEARLY)
def test_norm_gradients_of_nearly_constant_rows(rows, width, flags, dtype):
    x, dy = nearly_constant(rows, width, dtype), normal(rows, width, dtype=dtype, seed=3, scale=0.5, shift=0.2)
    w = normal(width, dtype=dtype, seed=1, scale=0.3, shift=1.0)
    _, stats = conv.layer_norm(x.cuda(), w.cuda(), save=True, flags=flags)
    want = gradients64(x.double(), dy.double(), w.double(), 1e-5, dtype)
    for name, g in zip(("dx", "dweight", "dbias"), conv.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), stats, flags=flags)):
        check(g, want[name], name)
    alone = conv.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), stats, need_dx=False, need_dbias=False, flags=flags)[1]
    check(alone, want["dweight"], "dweight alone")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width,flags", [(9, 101, 0), (300, 1003, 0), (5, 4099, 0), (5, 8191, 0), (5, 17001, 0),
                                              (300, 260, 0), (200, 700, conv.FLAG_NORM_STREAM)])
def test_norm_gradients_alone_and_together_are_the_same_bits(rows, width, flags, dtype):
    x, dy = (normal(rows, width, dtype=dtype, seed=s, shift=1.0).cuda() for s in (1, 2))
    w = normal(width, dtype=dtype, seed=3).cuda()
    _, stats = conv.layer_norm(x, w, save=True, flags=flags)
    every = conv.layer_norm_backward(dy, x, w, stats, flags=flags)
    for i in range(3):
        need = [j == i for j in range(3)]
        some = conv.layer_norm_backward(dy, x, w, stats, need_dx=need[0], need_dweight=need[1], need_dbias=need[2], flags=flags)
        assert torch.equal(some[i], every[i])


@pytest.mark.parametrize("rows,width,shift,flags", [
    (1, 768, 3e4, 0), (20, 768, 1000.0, 0), (20, 5000, -3e4, 0), (3, 20000, 500.0, 0), (700, 200, 3e4, 0), (5, 1003, 3e4, 0),
    (150, 700, 3e4, conv.FLAG_NORM_STREAM)])
def test_norm_gradients_of_a_mean_far_from_zero(rows, width, shift, flags):
    x, dy = normal(rows, width, dtype="f32", seed=4, shift=shift), normal(rows, width, dtype="f32", seed=5, scale=0.5, shift=0.2)
    w = normal(width, dtype="f32", seed=6, scale=0.3, shift=1.0)
    _, stats = conv.layer_norm(x.cuda(), w.cuda(), save=True, flags=flags)
    want = gradients64(x.double(), dy.double(), w.double(), 1e-5, "f32")
    for name, g in zip(("dx", "dweight", "dbias"), conv.layer_norm_backward(dy.cuda(), x.cuda(), w.cuda(), stats, flags=flags)):
        check(g, want[name], name)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,width", [(700, 264), (300, 4096), (40, 5001), (3, 40000)])
def test_quantised_rows_beside_those_of_a_divided_scale(rows, width, dtype):
    """The scale is the product of a row's largest value with 1 / 127 rounded; the quotient by 127, rounded once, is another
    definition.  What tells them apart: a scale's bits by the rounding of 1 / 127 (U / 16 here) and the two results' (U each),
    so a quotient of at most 127 by less than 127 (2 + 1 / 16) U, and an 8-bit value by one, where the quotient lies so near a
    half.  (In 16 bits such quotients are common: both numbers are short.)"""
    x = normal(rows, width, dtype=dtype, seed=rows + width)
    q, scale = (t.cpu().double() for t in conv.quantize_rows(x.cuda()))
    wide = x.double()
    divided = (wide.abs().amax(1) / 127).float().double()
    apart = (2 + 1 / 16) * U * 1.001
    assert ((scale - divided).abs() <= apart * divided).all()
    exact = wide / divided[:, None]
    moved = q != exact.round().clamp(-127, 127)
    assert ((q - exact.round()).abs()[moved] == 1).all()
    assert (((exact - exact.floor())[moved] - 0.5).abs() <= 127 * apart).all()


def test_dropout_takes_seeds_and_offsets_of_any_whole_number_type():
    import numpy
    x = torch.ones(6, 40, device="cuda")
    want, back = conv.dropout(x, 0.5, 7, 3), conv.dropout_backward(x, 0.5, 7, 3)
    for seed, offset in ((numpy.int64(7), 3), (7, numpy.int64(3)), (numpy.uint64(7), numpy.int32(3))):
        assert torch.equal(conv.dropout(x, 0.5, seed, offset), want)
        assert torch.equal(conv.dropout_backward(x, 0.5, seed, offset), back)
    assert torch.equal(conv.dropout(x, 0.5, numpy.int64(-1), numpy.int64(-2)), conv.dropout(x, 0.5, -1, -2))
    assert torch.equal(conv.dropout(x, 0.5, numpy.uint64(2 ** 64 - 1)), conv.dropout(x, 0.5, -1))
    for bad in ((7.0, 0), (7, 1.5), ("7", 0)):
        with pytest.raises(TypeError):
            conv.dropout(x, 0.5, *bad)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("xs,qs,at", [(264, 264, 0), (272, 300, 4), (301, 265, 1), (266, 266, 2), (280, 264, 8)])
def test_quantised_rows_of_any_stride_and_address(xs, qs, at, dtype):
    """conv_quantize_rows into rows of their own stride, from any address; what lies between the rows stays."""
    for rows, width in ((1, 257), (40, 264), (700, 256), (9, 3)):
        flat = normal(at + rows * xs + width, dtype=dtype, seed=rows).cuda()
        x = flat[at:].as_strided((rows, width), (xs, 1))
        q = torch.full((at + rows * qs + width,), 99, dtype=torch.int8, device="cuda")
        scale = torch.empty(rows, device="cuda")
        conv.conv_quantize_rows(conv.make_quantize_problem(rows, width, dtype=dtype, x_stride=xs, q_stride=qs), x, q[at:], scale)
        want, s = ref.quantize64(x.cpu().double())
        assert torch.equal(scale.cpu(), s)
        full = torch.full_like(q, 99).cpu()
        full[at:].as_strided((rows, width), (qs, 1)).copy_(want)
        assert torch.equal(q.cpu(), full)


@pytest.mark.parametrize("dtype", TYPES)
def test_dropout_backward_into_strided_rows(dtype):
    for rows, width, off, pad in ((40, 301, 3, 5), (40, 304, 8, 8), (5, 17, 0, 1)):
        dy = normal(rows, width + 6, dtype=dtype, seed=1).cuda()[:, 2:2 + width]
        full = torch.full((rows, off + width + pad), 77.0, dtype=TORCH[dtype], device="cuda")
        out = full[:, off:off + width]
        assert conv.dropout_backward(dy, 0.3, 5, 6, out=out) is out
        assert torch.equal(out, conv.dropout_backward(dy.contiguous(), 0.3, 5, 6))
        assert (full[:, :off] == 77).all() and (full[:, off + width:] == 77).all()


def test_norm_of_wide_rows_in_two_graphs_at_once():
    """Rows too wide for registers: three kernels backward, whose scratch is each graph's own."""
    x, dy = (normal(9, 17000, dtype="f32", seed=s).cuda() for s in (1, 2))
    w = normal(17000, dtype="f32", seed=3).cuda()

    def step(x):
        y, stats = conv.layer_norm(x, w, save=True)
        return (y, *conv.layer_norm_backward(dy, x, w, stats), conv.layer_norm_backward(dy, x, w, stats, need_dx=False)[1])
    step(x)
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for k, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            outs.append(step(x if k else x * 2))
    x.copy_(normal(9, 17000, dtype="f32", seed=4))
    want = [step(x * 2), step(x)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for k in range(2) for a, b in zip(outs[k], want[k]))
    assert torch.equal(want[0][2], want[0][4])
