"""What is measured of the feed-forward operators: a linear layer with bias,
activation and residual, the gated feed-forward projection, their training
steps, and the clipping of gradients by their global norm.

`run` computes them in their plain form (elementary torch operations in 32
bits, rounded once at the end) or, where `own` is true, with the calls a
program makes of hierarchical_gemm_gb300.tsffn.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------- cases --

def listed():
    return [
        # one token of one sequence through an output projection, weights stored N x K: latency
        dict(name="linear decode 1", op="linear", M=1, N=4096, K=4096, dtype="bf16", layout="rcr", act="none",
             bias=True, residual=True, train=False, pad=0),
        # a batch of 128 tokens through the wide projection: weight streaming
        dict(name="linear skinny 128", op="linear", M=128, N=28672, K=8192, dtype="bf16", layout="rrr", act="gelu",
             bias=True, residual=False, train=False, pad=0),
        # a prompt through a square projection, everything in the epilogue: tensor cores
        dict(name="linear prefill 4096", op="linear", M=4096, N=4096, K=4096, dtype="bf16", layout="rrr",
             act="gelu_tanh", bias=True, residual=True, train=False, pad=0),
        # a training step on a ragged batch, rows of X, dC and C wider than the matrices
        dict(name="linear train ragged", op="linear", M=1003, N=2056, K=1541, dtype="f16", layout="rcr", act="gelu",
             bias=True, residual=True, train=True, pad=24),
        # a training step of the first layer of a plain feed-forward block
        dict(name="linear train 4096", op="linear", M=4096, N=16384, K=4096, dtype="bf16", layout="rrr", act="gelu",
             bias=True, residual=False, train=True, pad=0),
        # one token of one sequence through the gated projection
        dict(name="gated decode 1", op="gated", M=1, F=14336, K=4096, dtype="bf16", layout="rcr", act="silu",
             train=False, pad=0),
        # the running sequences of a server, an odd number of them
        dict(name="gated decode 57", op="gated", M=57, F=14336, K=8192, dtype="bf16", layout="rrr", act="silu",
             train=False, pad=0),
        # a prompt through the gated projection
        dict(name="gated prefill 4096", op="gated", M=4096, F=14336, K=4096, dtype="bf16", layout="rcr", act="silu",
             train=False, pad=0),
        # a training step on a ragged batch with a width that fills no tile
        dict(name="gated train ragged", op="gated", M=2047, F=5464, K=2048, dtype="f16", layout="rrr",
             act="gelu_tanh", train=True, pad=8),
        # a training step of a full-size layer
        dict(name="gated train 4096", op="gated", M=4096, F=14336, K=4096, dtype="bf16", layout="rcr", act="silu",
             train=True, pad=0),
        # the gradients of one small model: many tensors, few values each: latency
        dict(name="clip small", op="clip", tensors=48, largest=65536, dtype="mixed", max_norm=1.0, scale=0.02,
             shapes=7),
        # the weight gradients of four gated feed-forward layers
        dict(name="clip layers", op="clip", tensors=8, largest=28672 * 4096, dtype="bf16", max_norm=1.0, scale=0.001,
             shapes=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "gated", "gated", "clip"])
    if op == "clip":
        return dict(op="clip", tensors=rng.randint(1, 48), largest=_log(rng, 1000, 20_000_000),
                    dtype=rng.choice(["mixed", "bf16", "f16", "f32"]), max_norm=rng.choice([0.5, 1.0, 1e6]),
                    scale=rng.choice([0.001, 0.02, 1.0]), shapes=rng.randint(1, 1 << 30))
    M = _log(rng, 1, 4096)
    K = _log(rng, 64, 8192)
    if rng.random() < 0.7:
        K = max(64, K // 8 * 8)
    case = dict(op=op, M=M, K=K, dtype=rng.choice(["bf16", "bf16", "f16"]), layout=rng.choice(["rrr", "rcr"]),
                train=rng.random() < 0.4, pad=rng.choice([0, 0, 8, 40]))
    if op == "linear":
        N = _log(rng, 64, 8192)
        if rng.random() < 0.7:
            N = max(64, N // 8 * 8)
        case.update(N=N, act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid"]),
                    bias=rng.random() < 0.7, residual=rng.random() < 0.5)
    else:
        case.update(F=max(8, _log(rng, 64, 8192) // 8 * 8), act=rng.choice(["silu", "gelu", "gelu_tanh", "relu", "sigmoid"]))
    return case


# --------------------------------------------------------------- inputs --

def _rows(r, c, pad, dt, gen=None, std=1.0):
    """An r x c matrix whose rows start 16 bytes apart at least: normal values from `gen`, or unset."""
    ld = (c + 7) // 8 * 8 + pad
    if gen is None:
        return torch.empty((r, ld), dtype=dt, device="cuda")[:, :c]
    x = torch.randn((r, ld), dtype=torch.float32, device="cuda", generator=gen).mul_(std).to(dt)
    return x[:, :c]


def _clip_tensors(case):
    """(number of values, dtype) of each gradient."""
    n = case["tensors"]
    if case["shapes"] == 0:  # gate-and-up and down weights in turn
        return [(case["largest"] if i % 2 == 0 else case["largest"] // 2, case["dtype"]) for i in range(n)]
    import random
    r = random.Random(case["shapes"])
    kinds = ["bf16", "f32", "f16"]
    sizes = [_log(r, 1, case["largest"]) for _ in range(n)]
    sizes[n // 2] = case["largest"]
    return [(s, kinds[i % 3] if case["dtype"] == "mixed" else case["dtype"]) for i, s in enumerate(sizes)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "clip":
        s["grads"] = [torch.randn(n, dtype=torch.float32, device="cuda", generator=gen).mul_(case["scale"]).to(_DT[d])
                      for n, d in _clip_tensors(case)]
        s["out"] = [torch.empty_like(g) for g in s["grads"]]
        return s
    M, K, pad, dt = case["M"], case["K"], case["pad"], _DT[case["dtype"]]
    N = case["N"] if case["op"] == "linear" else 2 * case["F"]
    C = case["N"] if case["op"] == "linear" else case["F"]  # columns of the result
    s["x"] = _rows(M, K, pad, dt, gen)
    wstd = K ** -0.5
    # the stored weights: N x K, or K x N
    s["w"] = _rows(N, K, 0, dt, gen, wstd) if case["layout"] == "rcr" else _rows(K, N, 0, dt, gen, wstd)
    s["c"] = _rows(M, C, pad, dt)
    s["bias"] = torch.randn(N, dtype=torch.float32, device="cuda", generator=gen).mul_(0.1).to(dt) if case.get("bias") else None
    s["r"] = _rows(M, C, pad, dt, gen) if case.get("residual") else None
    if case["train"]:
        s["dc"] = _rows(M, C, pad, dt, gen)
        s["dx"] = _rows(M, K, pad, dt)
        s["dw"] = _rows(s["w"].shape[0], s["w"].shape[1], 0, dt)
        s["db"] = torch.empty_like(s["bias"]) if case.get("bias") else None
    return s


# ---------------------------------------------------------- plain forms --

def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    s = 1 / (1 + torch.exp(-z))
    return s if act == "sigmoid" else z * s


def _act_grad(z, act):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-2 * c * (z + 0.044715 * z * z * z)))
        return s + z * s * (1 - s) * (2 * c) * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 - s) if act == "sigmoid" else s * (1 + z * (1 - s))


def _plain_linear(s, case):
    x = s["x"].float()
    w = s["w"].float().t() if case["layout"] == "rcr" else s["w"].float()
    dt = s["x"].dtype
    z = x @ w
    if s["bias"] is not None:
        z += s["bias"].float()
    y = _act(z, case["act"])
    if s["r"] is not None:
        y = y + s["r"].float()
    out = {"c": y.to(dt)}
    if case["train"]:
        dz = s["dc"].float() * _act_grad(z, case["act"])
        out["dx"] = (dz @ w.t()).to(dt)
        out["dw"] = (dz.t() @ x if case["layout"] == "rcr" else x.t() @ dz).to(dt)
        if s["bias"] is not None:
            out["db"] = dz.sum(0).to(dt)
    return out


def _plain_gated(s, case):
    x = s["x"].float()
    w = s["w"].float().t() if case["layout"] == "rcr" else s["w"].float()
    dt, F = s["x"].dtype, case["F"]
    gu = x @ w
    g, u = gu[:, :F], gu[:, F:]
    a = _act(g, case["act"])
    out = {"c": (a * u).to(dt)}
    if case["train"]:
        dh = s["dc"].float()
        dgu = torch.cat([dh * u * _act_grad(g, case["act"]), dh * a], 1)
        out["dx"] = (dgu @ w.t()).to(dt)
        out["dw"] = (dgu.t() @ x if case["layout"] == "rcr" else x.t() @ dgu).to(dt)
    return out


def _plain_clip(s, case):
    norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum().sqrt().float()
    coef = torch.clamp(case["max_norm"] / (norm + 1e-6), max=1.0)
    return {"norm": norm, "out": [(g.float() * coef).to(g.dtype) for g in s["grads"]]}


def run(state):
    case = state["case"]
    if not own:
        return {"linear": _plain_linear, "gated": _plain_gated, "clip": _plain_clip}[case["op"]](state, case)
    from hierarchical_gemm_gb300 import tsffn
    s = state
    if case["op"] == "clip":
        return {"norm": tsffn.clip_grad_norm(s["grads"], case["max_norm"], out=s["out"]), "out": s["out"]}
    # the operators take W as (K x N): row-major, or a view of the stored N x K weights
    rcr, act, train = case["layout"] == "rcr", case["act"], case["train"]
    w = s["w"].t() if rcr else s["w"]
    out = {"c": s["c"]}
    if case["op"] == "linear":
        saved = tsffn.linear(s["x"], w, bias=s["bias"], act=act, residual=s["r"], C=s["c"], save=train)
    else:
        saved = tsffn.gated(s["x"], w, act=act, H=s["c"], save=train)
    if train:
        dw = s["dw"].t() if rcr else s["dw"]
        if case["op"] == "linear":
            tsffn.linear_backward(s["dc"], s["x"], w, saved[1], act=act, dX=s["dx"], dW=dw, dbias=s["db"])
        else:
            tsffn.gated_backward(s["dc"], s["x"], w, saved[1], act=act, dX=s["dx"], dW=dw)
        out.update(dx=s["dx"], dw=s["dw"])
        if case.get("bias"):
            out["db"] = s["db"]
    return out


# ----------------------------------------------------------------- work --

def work(case):
    if case["op"] == "clip":
        e = {"bf16": 2, "f16": 2, "f32": 4}
        sizes = _clip_tensors(case)
        return {"bytes": sum(2 * n * e[d] for n, d in sizes) + 4, "flops": sum(3 * n for n, _ in sizes)}
    M, K = case["M"], case["K"]
    N = case["N"] if case["op"] == "linear" else 2 * case["F"]
    C = case["N"] if case["op"] == "linear" else case["F"]
    values = M * K + K * N + M * C + (N if case.get("bias") else 0) + (M * C if case.get("residual") else 0)
    if case["train"]:  # dC in; dX, dW and dbias out
        values += M * C + M * K + K * N + (N if case.get("bias") else 0)
    return {"bytes": 2 * values, "flops": (6 if case["train"] else 2) * M * N * K}


# ---------------------------------------------------------------- exact --

def _phi(z):
    """The standard normal distribution function."""
    return torch.special.ndtr(z)


def _exact_act(z, act):
    """(act(z), act'(z)) in 64 bits."""
    one = torch.ones_like(z)
    if act == "none":
        return z, one
    if act == "relu":
        return z.clamp(min=0), torch.heaviside(z, torch.zeros_like(z))
    if act == "gelu":
        p = _phi(z)
        return z * p, p + z * torch.exp(-z.square() / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        t = torch.tanh(a * (z + 0.044715 * z ** 3))
        return z * (1 + t) / 2, (1 + t) / 2 + z * (1 - t * t) / 2 * a * (1 + 3 * 0.044715 * z ** 2)
    s = torch.sigmoid(z)
    if act == "sigmoid":
        return s, s * (1 - s)
    return z * s, s + z * s * (1 - s)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        g = [t.double() for t in s["grads"]]
        norm = math.sqrt(math.fsum(float(torch.dot(t, t)) for t in g))
        c = min(1.0, case["max_norm"] / (norm + 1e-6))
        return {"norm": torch.tensor(norm, dtype=torch.float64), "out": [t * c for t in g]}
    x, w = s["x"].double(), s["w"].double()
    if case["layout"] == "rcr":
        w = w.t()
    z = torch.matmul(x, w)
    if case["op"] == "linear":
        if case["bias"]:
            z = z + s["bias"].double()
        a, da = _exact_act(z, case["act"])
        out = {"c": a + s["r"].double() if case["residual"] else a}
        grad = s["dc"].double() * da if case["train"] else None
    else:
        gate, up = z.chunk(2, dim=1)
        a, da = _exact_act(gate, case["act"])
        out = {"c": a * up}
        if case["train"]:
            d = s["dc"].double()
            grad = torch.empty_like(z)
            grad[:, : case["F"]] = d * up * da
            grad[:, case["F"]:] = d * a
    if case["train"]:
        out["dx"] = torch.matmul(grad, w.t())
        dw = torch.matmul(x.t(), grad)
        out["dw"] = dw.t() if case["layout"] == "rcr" else dw
        if case.get("bias"):
            out["db"] = grad.sum(0)
    return out
