"""The 8-bit product's kernel for some tens of rows (weights in rows on 16-byte
boundaries), on operands with which it is the one that runs: each test asks the
plan first."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import implicit_gemm_cnn_gb300 as conv
import rows_ref as ref
from dense_ref import TORCH, check

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TYPES = ["f32", "f16", "bf16"]
MID = conv.FLAG_INT8_MID


def plan(rows, c_in, c_out, stride=0, flags=MID, quantized=False):
    p = conv.make_int8_problem(rows, c_in, c_out, w_stride=stride, flags=flags, x_quantized=quantized)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return conv.conv_int8_describe_plan(p, sms)


def runs(rows, c_in, c_out, stride=0, flags=MID):
    text = plan(rows, c_in, c_out, stride, flags)
    assert text.startswith("tcgen05_f16_stream"), text
    return text


def bytes_in(rows, width, stride, seed):
    """Random bytes, all 256 values, in rows of `stride`; what lies between the rows is not zero."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-128, 128, (rows, stride), generator=g, dtype=torch.int8).cuda()[:, :width]


def normal(*shape, dtype, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64).to(TORCH[dtype]).cuda()


# rows, c_in, the weights' row stride, c_out: k's last stage of 128 terms whole and cut at every phase, one output, outputs past
# a tile, one to four blocks a cluster, tiles of rows of 32 to 128 and several
SIZES = [(1, 1, 16, 1), (17, 77, 96, 130), (33, 129, 144, 257), (64, 1023, 1024, 515), (65, 127, 128, 129), (100, 1025, 1040, 300),
         (128, 4003, 4016, 200), (31, 255, 256, 1000), (96, 511, 512, 20000), (129, 333, 336, 140), (300, 641, 656, 70),
         (1000, 95, 96, 260), (40, 10007, 10016, 128), (64, 4096, 4096, 4752), (128, 2048, 2064, 9984)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,c_in,stride,c_out", SIZES, ids=str)
def test_any_number_of_terms(rows, c_in, stride, c_out, dtype):
    runs(rows, c_in, c_out, stride)
    w, q = bytes_in(c_out, c_in, stride, 1), bytes_in(rows, c_in, c_in + 3, 2)
    g = torch.Generator().manual_seed(3)
    ws, xs = ((torch.rand(n, generator=g) + 0.5).cuda() * s for n, s in ((c_out, c_in ** -0.5 / 75), (rows, 1 / 75)))
    b, r = normal(c_out, dtype=dtype, seed=4), normal(rows, c_out, dtype=dtype, seed=5)
    got = conv.linear_int8(q, w, ws, b, r, x_scale=xs, dtype=TORCH[dtype], act="silu", flags=MID)
    want = ref.int8_64(q.cpu(), xs.cpu(), w.cpu(), ws.cpu(), b.cpu().double(), r.cpu().double(), "silu", 0, 0, False, dtype)
    check(got, want)
    # rows that the call quantises give what those quantised before give
    x = normal(rows, c_in, dtype=dtype, seed=6)
    q, xs = conv.quantize_rows(x)
    assert torch.equal(conv.linear_int8(x, w, ws, flags=MID), conv.linear_int8(q, w, ws, x_scale=xs, dtype=TORCH[dtype], flags=MID))
    assert conv.conv_linear_device_error() == 0


@pytest.mark.parametrize("rows", [20, 64, 128])
@pytest.mark.parametrize("c_in,stride", [(1009, 1024), (1024, 1024), (4111, 4112), (131071, 131072)])
def test_sums_are_exact(rows, c_in, stride):
    """Sums past 2^24 and down to a few units, over odd numbers of terms; scales of 1 show every bit of float32."""
    runs(rows, c_in, 40, stride)
    q, w = bytes_in(rows, c_in, c_in, 1), bytes_in(40, c_in, stride, 2)
    q[0], w[0], w[1] = -128, -128, 127
    w[2] = torch.where(q[0] < 0, 127, -127).to(torch.int8)
    half = c_in // 2
    w[3, :half], w[3, half:2 * half], w[3, 2 * half:] = 127, -127, 1
    one, ones = torch.ones(rows, device="cuda"), torch.ones(40, device="cuda")
    got = conv.linear_int8(q, w, ones, x_scale=one, dtype=torch.float32, flags=MID)
    assert torch.equal(got.cpu(), (q.cpu().double() @ w.cpu().double().T).float())


# clusters of one, two and four blocks; the last as the choice by size takes it
LAYERS = [(50, 272, 304, MID), (50, 1040, 304, MID), (120, 1040, 9000, MID), (64, 4096, 4752, 0), (100, 2064, 6208, 0)]


@pytest.mark.parametrize("rows,c_in,c_out,flags", LAYERS, ids=str)
def test_streams_and_two_graphs_at_once(rows, c_in, c_out, flags):
    runs(rows, c_in, c_out, flags=flags)
    x, (w, ws) = normal(rows, c_in, dtype="f16", seed=1), conv.quantize_rows(normal(c_out, c_in, dtype="f16", seed=2))
    kw = dict(act="silu", flags=flags)
    y = conv.linear_int8(x, w, ws, **kw)
    # the same bits as from the kernel for few rows: exact sums, the same arithmetic behind them
    assert torch.equal(y, conv.linear_int8(x, w, ws, act="silu", flags=conv.FLAG_INT8_FEW))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        y2 = conv.linear_int8(x, w, ws, stream=stream, **kw)
        side.synchronize()
        assert torch.equal(y, y2)
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for k, graph in enumerate(graphs):
        with torch.cuda.graph(graph):  # a layer after another: the second's weights are read under the first
            h = conv.linear_int8(x if k else x * 2, w, ws, **kw)
            outs.append((h, conv.linear_int8(h[:, :c_in].contiguous() if c_out >= c_in else x, w, ws, **kw)))
    x.copy_(normal(rows, c_in, dtype="f16", seed=5))
    want = []
    for k in range(2):
        h = conv.linear_int8(x if k else x * 2, w, ws, **kw)
        want.append((h, conv.linear_int8(h[:, :c_in].contiguous() if c_out >= c_in else x, w, ws, **kw)))
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for k in range(2) for a, b in zip(outs[k], want[k]))
    assert conv.conv_linear_device_error() == 0


def test_weights_written_right_before_the_call():
    """Weights and scales are read early, under the kernel that makes the halves of x: they are there all the same when the
    kernel just before the call writes them."""
    runs(64, 1040, 2064)
    x = normal(64, 1040, dtype="bf16", seed=1)
    mats = [normal(2064, 1040, dtype="bf16", seed=s) for s in range(2, 8)]
    want = [conv.linear_int8(x, *conv.quantize_rows(m), flags=conv.FLAG_INT8_FEW) for m in mats]
    w, ws = (torch.empty_like(t) for t in conv.quantize_rows(mats[0]))
    p = conv.make_quantize_problem(2064, 1040, dtype="bf16")
    torch.cuda.synchronize()
    got = []
    for m in mats:
        conv.conv_quantize_rows(p, m, w, ws)
        got.append(conv.linear_int8(x, w, ws, flags=MID))
    assert all(map(torch.equal, got, want))


def test_threads_on_one_stream_and_on_their_own():
    shapes = [(40, 528), (64, 1040), (100, 272), (128, 2064)]
    layers = []
    for i, (rows, c_in) in enumerate(shapes):
        runs(rows, c_in, 320)
        x = normal(rows, c_in, dtype="f32", seed=i)
        w, ws = conv.quantize_rows(normal(320, c_in, dtype="f32", seed=10 + i))
        layers.append((x, w, ws, conv.linear_int8(x, w, ws, flags=MID)))
    torch.cuda.synchronize()
    side, wrong = torch.cuda.Stream(), []

    def work(i, stream):
        x, w, ws, want = layers[i]
        for _ in range(20):
            got = conv.linear_int8(x, w, ws, flags=MID, stream=stream)
            (stream or torch.cuda.current_stream()).synchronize()
            if not torch.equal(got, want):
                wrong.append(i)
    threads = [threading.Thread(target=work, args=(i, side if i % 2 else None)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and conv.conv_linear_device_error() == 0


FIRST_CALL = """
import torch
import implicit_gemm_cnn_gb300 as conv
torch.manual_seed(0)
x = torch.randn(100, 1040, device="cuda").half()
w = torch.randint(-128, 128, (320, 1040), dtype=torch.int8, device="cuda")
ws = torch.rand(320, device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y = conv.linear_int8(x, w, ws, flags=conv.FLAG_INT8_MID)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(y, conv.linear_int8(x, w, ws, flags=conv.FLAG_INT8_FEW))
print("captured")
"""


def test_a_process_may_capture_it_first():
    runs(100, 1040, 320)
    out = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and "captured" in out.stdout, out.stdout + out.stderr


def test_a_flag_is_passed_over_where_its_kernel_cannot_run():
    for rows, c_in, c_out, stride in ((50, 264, 300, 0), (50, 77, 300, 85), (50, 1001, 64, 1001)):
        assert not plan(rows, c_in, c_out, stride).startswith("tcgen05_f16_stream")
        w, q = bytes_in(c_out, c_in, stride or c_in, 1), bytes_in(rows, c_in, c_in, 2)
        ws, xs = torch.ones(c_out, device="cuda"), torch.ones(rows, device="cuda")
        got = conv.linear_int8(q, w, ws, x_scale=xs, dtype=torch.float32, flags=MID)
        assert torch.equal(got.cpu(), (q.cpu().double() @ w.cpu().double().T).float())
