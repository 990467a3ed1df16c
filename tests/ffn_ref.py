"""The feed-forward operators in 64 bits (numpy), with a bound on how far a
kernel's output may be from each value.

Where the bounds come from, per element:
  * a value rounded to a type t is off by at most half a step, eps_t / 2
    relative (bf16 2^-8, fp16 2^-11, fp32 2^-24), plus half its smallest
    subnormal;
  * a sum of K products in the tensor cores: the products are exact, and
    each 16-deep step adds to a running fp32 sum, aligning and truncating:
    at most 4 units of 2^-23 of the sum of magnitudes S = sum |a b| per step,
    so (K / 16 + 2) 2^-21 S (the few-rows kernels' fragments are 16 deep too);
  * the activations: ex2.approx and a fast division are within 2^-20
    relative of the sigmoid, and so is the normal distribution function
    for |z| < 2; so act(z) is within
    2^-19 (|z| + 1) 2^-1 and act'(z) within 2^-18, on top of what an error
    in z makes of it: |act'| <= 1.13 and |act''| <= 1.2 for all of them but
    relu, whose derivative steps at 0 (values of z closer to 0 than their
    own error may take either side).
"""
import math

import numpy as np
import torch

EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
SLOPE, CURVE = 1.13, 1.2
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid")

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


def act(z, kind):
    """(act(z), act'(z)) of float64 arrays."""
    if kind == "none":
        return z, np.ones_like(z)
    if kind == "relu":
        return np.maximum(z, 0), (z > 0).astype(np.float64)
    if kind == "gelu":
        cdf = 0.5 * _erfc(-z * math.sqrt(0.5))
        return z * cdf, cdf + z * np.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if kind == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        t = np.tanh(a * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-z))
    return (s, s * (1 - s)) if kind == "sigmoid" else (z * s, s * (1 + z * (1 - s)))


def product(a, b, a_err=None):
    """(a b, bound) for a product in the tensor cores, a off by a_err."""
    S = np.abs(a) @ np.abs(b)
    bound = (a.shape[1] / 16 + 2) * 2.0 ** -21 * S
    if a_err is not None:
        bound = bound + a_err @ np.abs(b)
    return a @ b, bound


def rounded(v, err, dtype):
    """Bound of a value v, off by err before it is rounded to dtype."""
    return err + EPS[dtype] * (np.abs(v) + err) + TINY[dtype]


def _act_err(z, ez, kind):
    return ez if kind == "none" else SLOPE * ez + 2.0 ** -20 * (np.abs(z) + 1)


def _slope_err(z, ez, kind):
    if kind == "none":
        return np.zeros_like(z)
    if kind == "relu":
        return (np.abs(z) <= ez).astype(np.float64)
    return CURVE * ez + 2.0 ** -18


def linear(x, w, bias, kind, residual, out_dtype):
    """x, w, bias, residual: float64 arrays.  {"c": (value, bound), "z": ...}"""
    z, ez = product(x, w)
    if bias is not None:
        z = z + bias
        ez = ez + 2.0 ** -24 * (np.abs(z) + ez)
    y, ey = act(z, kind)[0], _act_err(z, ez, kind)
    if residual is not None:
        y = y + residual
        ey = ey + 2.0 ** -24 * (np.abs(y) + ey)
    return {"c": (y, rounded(y, ey, out_dtype)), "z": (z, ez)}


def _backward(x, w, d, ed, dtype, dw_dtype):
    """dX and dW of d (off by ed) rounded to dtype as an operand."""
    dx, ex = product(d, w.T, ed)
    dwt, ewt = product(d.T, x, ed.T)
    return {"dx": (dx, rounded(dx, ex, dtype)), "dw": (dwt.T, rounded(dwt.T, ewt.T, dw_dtype))}


def linear_backward(dc, x, w, bias, kind, dtype, dw_dtype, db_dtype):
    z, ez = linear(x, w, bias, kind, None, dtype)["z"]
    s = act(z, kind)[1]
    d = dc * s
    ed = np.abs(dc) * _slope_err(z, ez, kind) + (0 if kind == "none" else 2.0 ** -23 * np.abs(d))
    db = d.sum(0)
    edb = ed.sum(0) + d.shape[0] * 2.0 ** -24 * np.abs(d).sum(0)
    out = _backward(x, w, d, ed if kind == "none" else rounded(d, ed, dtype), dtype, dw_dtype)
    out["db"] = (db, rounded(db, edb, db_dtype))
    return out


def gated(x, w, kind, dtype):
    f = w.shape[1] // 2
    z, ez = product(x, w)
    g, u, eg, eu = z[:, :f], z[:, f:], ez[:, :f], ez[:, f:]
    a, ea = act(g, kind)[0], _act_err(g, eg, kind)
    h = a * u
    eh = ea * np.abs(u) + (np.abs(a) + ea) * eu + 2.0 ** -24 * np.abs(h)
    return {"h": (h, rounded(h, eh, dtype)), "z": (z, ez)}


def gated_backward(dh, x, w, kind, dtype, dw_dtype):
    f = w.shape[1] // 2
    z, ez = product(x, w)
    g, u, eg, eu = z[:, :f], z[:, f:], ez[:, :f], ez[:, f:]
    a, s = act(g, kind)
    ea, es = _act_err(g, eg, kind), _slope_err(g, eg, kind)
    dg, du = dh * u * s, dh * a
    edg = np.abs(dh) * (eu * (np.abs(s) + es) + np.abs(u) * es) + 2.0 ** -23 * np.abs(dg)
    edu = np.abs(dh) * ea + 2.0 ** -24 * np.abs(du)
    d = np.concatenate([dg, du], 1)
    ed = np.concatenate([edg, edu], 1)
    return _backward(x, w, d, rounded(d, ed, dtype), dtype, dw_dtype)


def clip(grads, max_norm):
    """(norm, coefficient) of a list of float64 arrays."""
    n = math.sqrt(math.fsum(float(np.dot(g.ravel(), g.ravel())) for g in grads))
    return n, min(1.0, max_norm / (n + 1e-6))


def check(got, want, what):
    """Every element of a tensor within its bound of (value, bound)."""
    value, bound = want
    g = f64(got)
    assert g.shape == value.shape, (what, g.shape, value.shape)
    off = np.abs(g - value)
    bad = ~(off <= bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, off / np.maximum(bound, 1e-300), 0)), g.shape)
        raise AssertionError("%s: %d of %d values off; at %s got %r, want %r within %r" %
                             (what, bad.sum(), bad.size, i, g[i], value[i], bound[i]))
