"""The dense operators in float64, with a bound on what float32 sums and one
rounding to the element type may add to each value.

The bounds follow from the arithmetic that include/linear.h promises:
  * a sum of K products is float32: at most K + 3 roundings (bias, residual and
    a join of k ranges among them), each of 2^-23 (a tensor core may cut instead
    of rounding to nearest) of the sum of absolute values;
  * an activation moves by at most its largest slope times that, and is itself
    evaluated to 2^-18 (1 + |z|) for 16-bit results (hardware exponential: 2^-21
    relative in its result and in its argument's product, times |z| below 8),
    2^-20 (1 + |z|) in float32;
  * a result is rounded once to its type: half a unit, and half the smallest
    subnormal of binary16;
  * 16-bit dz, h, dg and du are operands rounded once; their error goes through
    the next product's absolute values."""
import math

import torch

HALF_UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}
EVAL = {"f32": 2.0 ** -20, "f16": 2.0 ** -18, "bf16": 2.0 ** -18}
TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def act64(t, act, alpha=0.0, beta=0.0):
    if act == "identity":
        return t.clone()
    if act == "relu":
        return t.clamp(min=0)
    if act == "silu":
        return t * torch.special.expit(t)
    if act == "sigmoid":
        return torch.special.expit(t)
    if act == "tanh":
        return torch.tanh(t)
    if act == "hard_swish":
        return t * (t / 6 + 0.5).clamp(0, 1)
    if act == "hard_sigmoid":
        return (alpha * t + beta).clamp(0, 1)
    if act == "clip":
        return t.clamp(alpha, beta)
    if act == "leaky_relu":
        return torch.where(t >= 0, t, alpha * t)
    if act == "gelu":
        return t * torch.special.ndtr(t)
    assert act == "gelu_tanh"
    return 0.5 * t * (1 + torch.tanh(math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3)))


def slope64(t, act, alpha=0.0, beta=0.0):
    """act'(t), by formula."""
    one, zero = torch.ones_like(t), torch.zeros_like(t)
    if act == "identity":
        return one
    if act == "relu":
        return torch.where(t > 0, one, zero)
    if act in ("silu", "sigmoid"):
        s = torch.special.expit(t)
        return s * (1 + t * (1 - s)) if act == "silu" else s * (1 - s)
    if act == "tanh":
        return 1 - torch.tanh(t) ** 2
    if act == "hard_swish":
        return torch.where(t <= -3, zero, torch.where(t >= 3, one, t / 3 + 0.5))
    if act == "hard_sigmoid":
        s = alpha * t + beta
        return torch.where((s > 0) & (s < 1), alpha * one, zero)
    if act == "clip":
        return torch.where((t > alpha) & (t < beta), one, zero)
    if act == "leaky_relu":
        return torch.where(t >= 0, one, alpha * one)
    if act == "gelu":
        return torch.special.ndtr(t) + t * torch.exp(-0.5 * t * t) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    h = torch.tanh(k * (t + 0.044715 * t ** 3))
    return 0.5 * (1 + h) + 0.5 * t * (1 - h * h) * k * (1 + 3 * 0.044715 * t * t)


# largest |act'| and |act''| (piecewise linear ones: 0, and corners where act' jumps by at most MAX_SLOPE)
MAX_SLOPE = {"identity": 1, "relu": 1, "silu": 1.1, "sigmoid": 0.25, "tanh": 1, "hard_swish": 1.5, "hard_sigmoid": 1,
             "clip": 1, "leaky_relu": 1, "gelu": 1.13, "gelu_tanh": 1.13}
MAX_BEND = {"silu": 0.5, "sigmoid": 0.1, "tanh": 0.77, "hard_swish": 0.34, "gelu": 0.8, "gelu_tanh": 0.9}


def corners(act, alpha, beta):
    if act in ("relu", "leaky_relu"):
        return [0.0]
    if act == "hard_swish":
        return [-3.0, 3.0]
    if act == "hard_sigmoid":
        return [-beta / alpha, (1 - beta) / alpha]
    if act == "clip":
        return [alpha, beta]
    return []


def product(a, b, a_err=None, b_err=None):
    """a b^T in float64 and the bound of its float32 sum, given bounds of the operands' own errors."""
    v = a @ b.T
    size = a.abs() @ b.abs().T
    err = (a.shape[1] + 3) * 2.0 ** -23 * size
    if a_err is not None:
        err = err + a_err @ (b.abs() + (b_err if b_err is not None else 0)).T
    if b_err is not None:
        err = err + a.abs() @ b_err.T
    return v, err


def rounded(v, err, dtype):
    return v, err + HALF_UNIT[dtype] * (v.abs() + err) + TINY[dtype]


def act_bound(z, ez, act, dtype):
    return MAX_SLOPE[act] * ez + (0 if act == "identity" else EVAL[dtype] * (1 + z.abs()))


def slope_bound(z, ez, act, alpha, beta, dtype):
    if act == "identity":
        return torch.zeros_like(z)
    e = MAX_BEND.get(act, 0) * ez + EVAL[dtype] * (1 + z.abs())
    for c in corners(act, alpha, beta):
        e = e + 1.5 * ((z - c).abs() <= ez + 1e-6)
    return e


def linear64(x, w, bias, residual, act, alpha, beta, last, dtype):
    """{"y": (value, bound), "z": (value, bound)}"""
    z, ez = product(x, w)
    if bias is not None:
        z, ez = z + bias, ez + 2.0 ** -23 * 4 * bias.abs()
    if residual is not None and not last:
        z, ez = z + residual, ez + 2.0 ** -23 * 4 * residual.abs()
    y, ey = act64(z, act, alpha, beta), act_bound(z, ez, act, dtype)
    if residual is not None and last:
        y, ey = y + residual, ey + 2.0 ** -23 * (y.abs() + residual.abs())
    return {"y": rounded(y, ey, dtype), "z": (z, ez + 2.0 ** -23 * z.abs())}


def linear_backward64(dy, x, w, z, ez, act, alpha, beta, last, dtype):
    s, es = slope64(z, act, alpha, beta), slope_bound(z, ez, act, alpha, beta, dtype)
    dz = dy * s
    raw = dy.abs() * es + 2.0 ** -23 * dz.abs()
    _, edz = rounded(dz, raw, dtype) if act != "identity" else (dz, torch.zeros_like(dz))
    ones = torch.ones(1, dy.shape[0], dtype=torch.float64)
    db, edb = product(ones, dz.T.contiguous(), torch.zeros_like(ones), raw.T.contiguous())
    dr, edr = (dy, 0 * dy) if last else rounded(dz, raw, dtype)
    return {"dx": rounded(*product(dz, w.T, edz), dtype), "dw": rounded(*product(dz.T, x.T, edz.T), dtype),
            "dbias": rounded(db[0], edb[0], dtype), "dresidual": (dr, edr)}


def gated64(x, wg, wu, wd, residual, act, alpha, beta, dtype, dy=None):
    g, eg = product(x, wg)
    u, eu = product(x, wu)
    a, ea = act64(g, act, alpha, beta), act_bound(g, eg, act, dtype)
    h = a * u
    h, eh = rounded(h, ea * (u.abs() + eu) + a.abs() * eu + 2.0 ** -23 * h.abs(), dtype)
    y, ey = product(h, wd, eh)
    if residual is not None:
        y, ey = y + residual, ey + 2.0 ** -23 * 4 * residual.abs()
    out = {"y": rounded(y, ey, dtype)}
    if dy is None:
        return out
    dh, edh = product(dy, wd.T)
    s, es = slope64(g, act, alpha, beta), slope_bound(g, eg, act, alpha, beta, dtype)
    du, dg = dh * a, dh * u * s
    du, edu = rounded(du, edh * (a.abs() + ea) + dh.abs() * ea + 2.0 ** -22 * du.abs(), dtype)
    us = (u.abs() + eu) * (s.abs() + es) - u.abs() * s.abs()  # the product u s's bound
    dg, edg = rounded(dg, edh * (u * s).abs() + (dh.abs() + edh) * us + 2.0 ** -22 * dg.abs(), dtype)
    p, ep = product(dg, wg.T, edg)
    q, eq = product(du, wu.T, edu)
    size = dg.abs() @ wg.abs() + du.abs() @ wu.abs()
    out["dx"] = rounded(p + q, ep + eq + 2.0 ** -23 * (2 * wg.shape[0] + 3) * size, dtype)
    out["dw_gate"] = rounded(*product(dg.T, x.T, edg.T), dtype)
    out["dw_up"] = rounded(*product(du.T, x.T, edu.T), dtype)
    out["dw_down"] = rounded(*product(dy.T, h.T, None, eh.T), dtype)
    return out


def check(got, want, what=""):
    """Every value within its bound; NaN and infinity where the reference has them."""
    v, err = want
    got = got.detach().cpu().double()
    assert got.shape == v.shape, (what, got.shape, v.shape)
    off = (got - v).abs()
    bad = ~(off <= err)
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], v[bad][:4], err[bad][:4] if torch.is_tensor(err) else err)
