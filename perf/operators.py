"""The dense operators as a user's program calls them: what is measured, on what sizes, and the same operators in plain torch.

linear          y = act(x W^T + bias + residual); a step adds dx, dW, dbias for a given dy
gated_ffn       y = (act(x Wg^T) * (x Wu^T)) Wd^T + residual; a step adds dx, dWg, dWu, dWd for a given dy
clip_grad_norm  the global 2-norm of many tensors, and the tensors scaled by min(1, max_norm / (norm + 1e-6))

x is [rows][in], weights are [out][in].  Sums are float32 or wider whatever the tensors' type."""
import math

import torch

own = False  # set by the measuring tools: False, the plain forms; True, the framework's kernels

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


# ---- cases ----------------------------------------------------------------------------------------------------------
def linear_case(name, rows, n_in, n_out, dtype, act="identity", bias=True, residual=False, step=False):
    return {"name": name, "op": "linear", "rows": rows, "in": n_in, "out": n_out, "dtype": dtype, "act": act,
            "bias": bias, "residual": residual, "step": step}


def ffn_case(name, rows, width, hidden, dtype, act="silu", residual=True, step=False):
    return {"name": name, "op": "ffn", "rows": rows, "width": width, "hidden": hidden, "dtype": dtype, "act": act,
            "residual": residual, "step": step}


def clip_case(name, tensors, values, dtype, clipped=True):
    return {"name": name, "op": "clip", "tensors": tensors, "values": values, "dtype": dtype, "clipped": clipped}


def listed():
    return [
        # one token through an output projection while text is generated: latency alone counts
        linear_case("linear one token", 1, 1024, 1024, "bf16", residual=True),
        # a few sequences decoded together; an output width that is no multiple of anything
        linear_case("linear 12 tokens odd width", 12, 2000, 5001, "f16", act="gelu_tanh"),
        # a prompt through an output projection with its residual stream
        linear_case("linear prompt", 2048, 4096, 4096, "bf16", residual=True),
        # a training step of a feed-forward layer's first projection
        linear_case("linear step 8192 rows", 8192, 2048, 8192, "bf16", act="gelu_tanh", step=True),
        # a small model trained in float32, every size odd or nearly so
        linear_case("linear step float32 odd", 1001, 515, 1030, "f32", act="gelu", step=True),
        # one token through a whole gated block: the weights' bytes are all there is
        ffn_case("gated ffn one token", 1, 4096, 12288, "bf16"),
        # a served batch, one token from each of 64 sequences
        ffn_case("gated ffn 64 tokens", 64, 2048, 8192, "f16"),
        # a long prompt
        ffn_case("gated ffn prompt", 4096, 4096, 12288, "bf16"),
        # a training step of a large block: the largest case
        ffn_case("gated ffn step 8192 rows", 8192, 4096, 12288, "bf16", step=True),
        # ragged packed sequences through a small block with an odd hidden width
        ffn_case("gated ffn step ragged", 1537, 1000, 2731, "f16", act="gelu_tanh", step=True),
        # the gradients of a small model: many short tensors
        clip_case("clip 40 short tensors", 40, 150_000, "f32"),
        # the gradients of a large model in its own type
        clip_case("clip 300 tensors", 300, 800_000_000, "bf16"),
    ]


def spread(rng, low, high):
    """A whole number from low to high, spread over its logarithm: mostly odd ones, now and then a multiple of 64."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() < 0.4:
        v = (v + 63) // 64 * 64
    v = v + 1 if v == 3072 else v
    return max(low, min(high, v))


def draw(rng):
    kind = rng.choice(["linear", "linear", "linear step", "ffn", "ffn", "ffn step", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f16", "f32"])
    top = 8192 if dtype != "f32" else 2048  # float32 has no tensor-core rate: smaller models use it
    if kind == "clip":
        c = clip_case("", spread(rng, 1, 400), spread(rng, 10_000, 800_000_000), dtype, rng.random() < 0.7)
    elif kind.startswith("linear"):
        step = kind == "linear step"
        c = linear_case("", spread(rng, 32 if step else 1, top), spread(rng, 256, top), spread(rng, 256, top), dtype,
                        act=rng.choice(["identity", "gelu", "gelu_tanh", "silu", "relu"]), bias=rng.random() < 0.7,
                        residual=not step and rng.random() < 0.5, step=step)
    else:
        step = kind == "ffn step"
        c = ffn_case("", spread(rng, 32 if step else 1, top), spread(rng, 256, top // 2), spread(rng, 512, top // 2 * 3), dtype,
                     act=rng.choice(["silu", "silu", "gelu_tanh", "gelu"]), residual=rng.random() < 0.7, step=step)
    del c["name"]
    return c


# ---- inputs ---------------------------------------------------------------------------------------------------------
def tensor_sizes(tensors, values):
    """The element counts of a model's tensors: vectors of a few hundred values, and matrices whose sizes grow evenly."""
    small = [min(301 + 64 * (i % 5), max(1, values // (4 * tensors))) for i in range(tensors // 2)]
    count = tensors - len(small)
    left = values - sum(small)
    weights = [1 + i % 7 for i in range(count)]
    big = [max(1, left * w // sum(weights)) for w in weights]
    sizes = []
    for i in range(tensors):  # a matrix, then its vector
        sizes.append(big.pop() if (i % 2 == 0 or not small) and big else small.pop())
    return sizes


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale).to(dt)

    s = {"case": case}
    if case["op"] == "linear":
        rows, k, n = case["rows"], case["in"], case["out"]
        s["x"] = normal(rows, k)
        s["w"] = normal(n, k, scale=k ** -0.5)
        s["bias"] = normal(n, scale=0.1) if case["bias"] else None
        s["residual"] = normal(rows, n) if case["residual"] else None
        s["dy"] = normal(rows, n, scale=0.02) if case["step"] else None
    elif case["op"] == "ffn":
        rows, d, f = case["rows"], case["width"], case["hidden"]
        s["x"] = normal(rows, d)
        s["w_gate"], s["w_up"] = normal(f, d, scale=d ** -0.5), normal(f, d, scale=d ** -0.5)
        s["w_down"] = normal(d, f, scale=f ** -0.5)
        s["residual"] = normal(rows, d) if case["residual"] else None
        s["dy"] = normal(rows, d, scale=0.02) if case["step"] else None
    else:
        # gradients lie in one buffer, one tensor after another, as a trainer's buckets have them
        sizes = tensor_sizes(case["tensors"], case["values"])
        total = sum(sizes)
        flat = torch.empty(total, device="cuda", dtype=dt)
        for at in range(0, total, 1 << 26):
            part = flat[at:at + (1 << 26)]
            part.copy_(torch.randn(part.numel(), generator=g, device="cuda", dtype=torch.float32).mul_(0.01))
        s["flat"], s["out"] = flat, torch.empty_like(flat)
        s["grads"], s["outs"] = list(flat.split(sizes)), list(s["out"].split(sizes))
        norm = 0.01 * math.sqrt(total)  # what the values' spread makes the norm, nearly
        s["max_norm"] = norm * (0.25 if case["clipped"] else 4.0)
    return s


# ---- one pass -------------------------------------------------------------------------------------------------------
def plain_act(t, act):
    """The activation and its derivative, in 32 bits."""
    if act == "identity":
        return t, torch.ones_like(t)
    if act == "relu":
        on = (t > 0).to(t.dtype)
        return t * on, on
    if act == "silu":
        s = 1 / (1 + torch.exp(-t))
        return t * s, s * (1 + t * (1 - s))
    if act == "gelu":
        c = 0.5 * (1 + torch.erf(t * math.sqrt(0.5)))
        return t * c, c + t * torch.exp(-0.5 * t * t) * (1 / math.sqrt(2 * math.pi))
    k = math.sqrt(2 / math.pi)
    h = torch.tanh(k * (t + 0.044715 * t * t * t))
    return 0.5 * t * (1 + h), 0.5 * (1 + h) + 0.5 * t * (1 - h * h) * k * (1 + 3 * 0.044715 * t * t)


def plain(s):
    c = s["case"]
    dt = DTYPES[c["dtype"]]
    if c["op"] == "linear":
        x, w = s["x"].float(), s["w"].float()
        z = x @ w.t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        if s["residual"] is not None:
            z = z + s["residual"].float()
        y, slope = plain_act(z, c["act"])
        out = {"y": y.to(dt)}
        if c["step"]:
            dz = s["dy"].float() * slope
            out["dx"], out["dw"] = (dz @ w).to(dt), (dz.t() @ x).to(dt)
            if s["bias"] is not None:
                out["dbias"] = dz.sum(0).to(dt)
        return out
    if c["op"] == "ffn":
        x, wg, wu, wd = s["x"].float(), s["w_gate"].float(), s["w_up"].float(), s["w_down"].float()
        gate, up = x @ wg.t(), x @ wu.t()
        a, slope = plain_act(gate, c["act"])
        h = a * up
        y = h @ wd.t()
        if s["residual"] is not None:
            y = y + s["residual"].float()
        out = {"y": y.to(dt)}
        if c["step"]:
            dy = s["dy"].float()
            dh = dy @ wd
            dg, du = dh * up * slope, dh * a
            out["dx"] = (dg @ wg + du @ wu).to(dt)
            out["dw_gate"], out["dw_up"], out["dw_down"] = (dg.t() @ x).to(dt), (du.t() @ x).to(dt), (dy.t() @ h).to(dt)
        return out
    norm = torch.stack([(t.float() * t.float()).sum() for t in s["grads"]]).sum().sqrt()
    scale = torch.clamp(s["max_norm"] / (norm + EPS), max=1.0)
    for t, o in zip(s["grads"], s["outs"]):
        o.copy_(t.float() * scale)
    return {"norm": norm, "out": s["out"]}


def run(s):
    if not own:
        return plain(s)
    import implicit_gemm_cnn_gb300 as conv

    c = s["case"]
    if c["op"] == "linear":
        if not c["step"]:
            return {"y": conv.linear(s["x"], s["w"], s["bias"], s["residual"], act=c["act"])}
        y, pre = conv.linear(s["x"], s["w"], s["bias"], s["residual"], act=c["act"], save=True)
        dx, dw, dbias, _ = conv.linear_backward(s["dy"], s["x"], s["w"], pre, act=c["act"], need_dbias=c["bias"])
        out = {"y": y, "dx": dx, "dw": dw}
        if c["bias"]:
            out["dbias"] = dbias
        return out
    if c["op"] == "ffn":
        weights = s["w_gate"], s["w_up"], s["w_down"]
        if not c["step"]:
            return {"y": conv.gated_ffn(s["x"], *weights, s["residual"], act=c["act"])}
        y, saved = conv.gated_ffn(s["x"], *weights, s["residual"], act=c["act"], save=True)
        dx, dwg, dwu, dwd = conv.gated_ffn_backward(s["dy"], s["x"], *weights, saved, act=c["act"])
        return {"y": y, "dx": dx, "dw_gate": dwg, "dw_up": dwu, "dw_down": dwd}
    norm = conv.clip_grad_norm(s["grads"], s["max_norm"], eps=EPS, out=s["outs"])
    return {"norm": norm, "out": s["out"]}


# ---- what a pass cannot do without ----------------------------------------------------------------------------------
def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "linear":
        r, k, n = case["rows"], case["in"], case["out"]
        moved = r * k + n * k + r * n * (2 if case["residual"] else 1) + (n if case["bias"] else 0)
        products = 1
        if case["step"]:
            moved += r * n + r * k + n * k + (n if case["bias"] else 0)  # dy in; dx, dw, dbias out
            products = 3
        return {"bytes": moved * size, "flops": 2.0 * r * k * n * products}
    if case["op"] == "ffn":
        r, d, f = case["rows"], case["width"], case["hidden"]
        moved = r * d * (3 if case["residual"] else 2) + 3 * d * f
        products = 3
        if case["step"]:
            moved += 2 * r * d + 3 * d * f  # dy in; dx and the weights' gradients out
            products = 9
        return {"bytes": moved * size, "flops": 2.0 * r * d * f * products}
    n = sum(tensor_sizes(case["tensors"], case["values"]))
    return {"bytes": 2 * n * size, "flops": 3.0 * n}


# ---- the definition in 64 bits --------------------------------------------------------------------------------------
def exact_act(t, act):
    if act == "identity":
        return t
    if act == "relu":
        return t.clamp(min=0)
    if act == "silu":
        return t * torch.special.expit(t)
    if act == "gelu":
        return t * torch.special.ndtr(t)
    return t * torch.special.expit(2 * math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3))  # (1 + tanh v) / 2 = expit(2v)


def exact(case, seed):
    """The forward formula in float64; the gradients by differentiating it, not by the formulas above."""
    s = prepare(case, seed)
    if case["op"] == "clip":
        total, flat = 0.0, s["flat"]
        blocks = range(0, flat.numel(), 1 << 26)
        for at in blocks:
            v = flat[at:at + (1 << 26)].double()
            total = total + v.dot(v)
        norm = total.sqrt()
        ratio = s["max_norm"] / (norm.item() + EPS)
        out = torch.empty(flat.numel(), dtype=torch.float64, device="cuda")
        for at in blocks:
            out[at:at + (1 << 26)] = flat[at:at + (1 << 26)].double() * min(1.0, ratio)
        return {"norm": norm, "out": out}
    wide = {k: v.double().requires_grad_(case["step"]) for k, v in s.items() if isinstance(v, torch.Tensor) and k != "dy"}
    with torch.set_grad_enabled(case["step"]):
        if case["op"] == "linear":
            y = torch.nn.functional.linear(wide["x"], wide["w"], wide.get("bias"))
            y = exact_act(y + wide["residual"] if "residual" in wide else y, case["act"])
            of = {"dx": "x", "dw": "w", "dbias": "bias"}
        else:
            linear = torch.nn.functional.linear
            h = exact_act(linear(wide["x"], wide["w_gate"]), case["act"]) * linear(wide["x"], wide["w_up"])
            y = linear(h, wide["w_down"])
            y = y + wide["residual"] if "residual" in wide else y
            of = {"dx": "x", "dw_gate": "w_gate", "dw_up": "w_up", "dw_down": "w_down"}
    out = {"y": y.detach()}
    if case["step"]:
        of = {k: v for k, v in of.items() if v in wide}
        grads = torch.autograd.grad(y, [wide[v] for v in of.values()], s["dy"].double())
        out.update(zip(of, grads))
    return out
