"""Feed-forward operators, on the host: the 64-bit reference the GPU tests
compare with (its derivatives against differences), the C ABI's exports and
structures, and every refusal that needs no device."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import ffn_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, ALIGNMENT = 0, 1, 2, 3


@pytest.fixture(scope="module")
def ff():
    from hierarchical_gemm_gb300 import build
    build.build()
    from hierarchical_gemm_gb300 import tsffn
    return tsffn


# --------------------------------------------------------- the reference --

@pytest.mark.parametrize("kind", ref.ACTS)
def test_derivatives_against_differences(kind):
    z = np.linspace(-9, 9, 400)  # (no point at 0, where relu has no derivative)
    h = 1e-5
    d = (ref.act(z + h, kind)[0] - ref.act(z - h, kind)[0]) / (2 * h)
    assert np.allclose(ref.act(z, kind)[1], d, rtol=1e-8, atol=1e-8)
    # the slopes and curvatures the bounds assume
    if kind != "relu":
        assert np.abs(ref.act(z, kind)[1]).max() <= ref.SLOPE
        dd = (ref.act(z + h, kind)[1] - ref.act(z - h, kind)[1]) / (2 * h)
        assert np.abs(dd).max() <= ref.CURVE


@pytest.mark.parametrize("kind", ref.ACTS)
def test_backward_against_differences(kind):
    rng = np.random.default_rng(5)
    M, K, F = 5, 6, 4
    x, w, dh = rng.normal(size=(M, K)), rng.normal(size=(K, 2 * F)), rng.normal(size=(M, F))
    b, dc = rng.normal(size=2 * F), rng.normal(size=(M, 2 * F))
    t = torch.bfloat16
    lin = ref.linear_backward(dc, x, w, b, kind, t, t, t)
    gat = ref.gated_backward(dh, x, w, kind, t, t)

    def loss_l(x, w, b):
        return (dc * ref.linear(x, w, b, kind, None, t)["c"][0]).sum()

    def loss_g(x, w):
        return (dh * ref.gated(x, w, kind, t)["h"][0]).sum()

    h = 1e-6
    for i in range(6):
        vx, vw, vb = rng.normal(size=x.shape), rng.normal(size=w.shape), rng.normal(size=b.shape)
        d = (loss_l(x + h * vx, w + h * vw, b + h * vb) - loss_l(x - h * vx, w - h * vw, b - h * vb)) / (2 * h)
        assert abs(d - (lin["dx"][0] * vx).sum() - (lin["dw"][0] * vw).sum() - (lin["db"][0] * vb).sum()) < 1e-6
        d = (loss_g(x + h * vx, w + h * vw) - loss_g(x - h * vx, w - h * vw)) / (2 * h)
        assert abs(d - (gat["dx"][0] * vx).sum() - (gat["dw"][0] * vw).sum()) < 1e-6


# ---------------------------------------------------------------- the ABI --

def test_exports(ff):
    text = open(os.path.join(ROOT, "include", "tsffn.h")).read()
    names = set(re.findall(r"TSGEMM_API\s+[\w\s\*]+?\b(tsffn_\w+)\s*\(", text))
    assert names == set(ff.EXPORTS)
    for n in names:
        assert hasattr(ff.lib, n), n


def test_structures_match_the_header(ff):
    text = open(os.path.join(ROOT, "include", "tsffn.h")).read()
    for cls, name in [(ff.LinearArgs, "tsffn_linear_args"), (ff.LinearBackwardArgs, "tsffn_linear_backward_args"),
                      (ff.GatedArgs, "tsffn_gated_args"), (ff.GatedBackwardArgs, "tsffn_gated_backward_args")]:
        body = re.search(r"typedef struct \{((?:(?!typedef)[\s\S])*?)\} %s;" % name, text).group(1)
        body = re.sub(r"/\*[\s\S]*?\*/", "", body)
        fields = []
        for decl in body.split(";"):
            m = re.match(r"\s*((?:const\s+)?\w+)\s*(\*?)\s*(.+)$", decl.strip())
            if m:
                size = 8 if m.group(2) else {"int64_t": 8, "int32_t": 4}[m.group(1)]
                fields += [(n.strip(" *"), size) for n in m.group(3).split(",")]
        assert [(n, ctypes.sizeof(t)) for n, t in cls._fields_] == fields


P = 1 << 20  # dummy addresses, a mebibyte apart; nothing is launched


def _linear(ff, **kw):
    a = dict(M=4, N=64, K=64, dtype=1, dtype_out=1, dtype_bias=1, layout=0, act=2, reserved=0, X=P, W=2 * P, bias=3 * P,
             residual=4 * P, C=5 * P, saved=6 * P, ldx=64, ldw=64, ldr=64, ldc=64)
    a.update(kw)
    return ff.lib.tsffn_linear(None, ctypes.byref(ff.LinearArgs(**a)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=0), INVALID), (dict(N=-1), INVALID), (dict(K=0), INVALID),
    (dict(M=2 ** 31), UNSUPPORTED), (dict(N=2 ** 62), UNSUPPORTED), (dict(K=2 ** 31), UNSUPPORTED),
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED), (dict(dtype=9), INVALID),
    (dict(dtype_out=0), UNSUPPORTED), (dict(dtype_out=3), UNSUPPORTED), (dict(dtype_out=-1), INVALID),
    (dict(dtype_bias=0), UNSUPPORTED), (dict(layout=2), UNSUPPORTED), (dict(layout=4), INVALID),
    (dict(act=6), INVALID), (dict(act=-1), INVALID), (dict(reserved=1), INVALID),
    (dict(X=None), INVALID), (dict(W=None), INVALID), (dict(C=None), INVALID),
    (dict(X=P + 8), ALIGNMENT), (dict(bias=3 * P + 2), ALIGNMENT), (dict(saved=6 * P + 4), ALIGNMENT),
    (dict(ldx=56), INVALID), (dict(ldx=68), ALIGNMENT), (dict(ldc=66), ALIGNMENT), (dict(ldw=2 ** 32), UNSUPPORTED),
    (dict(residual=4 * P + 4), ALIGNMENT), (dict(ldr=32), INVALID),
    (dict(C=P), INVALID), (dict(C=2 * P + 128), INVALID), (dict(C=3 * P), INVALID), (dict(C=6 * P), INVALID),
    (dict(residual=5 * P + 128), INVALID),            # C shifted by a row
    (dict(residual=5 * P, ldr=72), INVALID),          # C with another stride
    (dict(residual=6 * P), INVALID),                  # on the saved pre-activations
    # what is right but for the missing handle
    (dict(), INVALID),
])
def test_linear_refusals(ff, kw, code):
    assert _linear(ff, **kw) == code


def test_refusals_are_the_stated_ones(ff):
    """The last, valid call is refused for its handle alone: the others'
    errors come from their arguments (another code, or found before it)."""
    assert _linear(ff, dtype_out=2, ldc=64) == INVALID
    assert _linear(ff, dtype_out=2, ldc=66) == ALIGNMENT
    assert _linear(ff, residual=5 * P, X=P + 8) == ALIGNMENT


def _backward(ff, **kw):
    a = dict(M=4, N=64, K=64, dtype=1, dtype_dw=1, dtype_bias=1, layout=0, act=2, reserved=0, dC=P, X=2 * P, W=3 * P,
             saved=4 * P, dX=5 * P, dW=6 * P, dbias=7 * P, workspace=8 * P, lddc=64, ldx=64, ldw=64, lddx=64, lddw=64)
    a.update(kw)
    return ff.lib.tsffn_linear_backward(None, ctypes.byref(ff.LinearBackwardArgs(**a)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(M=0), INVALID), (dict(K=2 ** 31), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(dtype_dw=0), UNSUPPORTED),
    (dict(dtype_bias=0), UNSUPPORTED), (dict(layout=2), UNSUPPORTED), (dict(act=7), INVALID),
    (dict(dC=None), INVALID), (dict(X=None), INVALID), (dict(W=None), INVALID), (dict(saved=None), INVALID),
    (dict(workspace=None), INVALID), (dict(dX=None, dW=None, dbias=None), INVALID),
    (dict(lddc=63), INVALID), (dict(lddw=60), INVALID), (dict(lddx=68), ALIGNMENT), (dict(dW=6 * P + 8), ALIGNMENT),
    (dict(dtype_dw=2, lddw=66), ALIGNMENT),
    (dict(dX=P), INVALID), (dict(dW=3 * P), INVALID), (dict(dX=6 * P), INVALID), (dict(dbias=8 * P), INVALID),
    (dict(workspace=4 * P), INVALID), (dict(workspace=P), INVALID),
])
def test_linear_backward_refusals(ff, kw, code):
    assert _backward(ff, **kw) == code


def _gated(ff, **kw):
    a = dict(M=4, F=32, K=64, dtype=0, layout=0, act=4, reserved=0, X=P, W=2 * P, H=3 * P, saved=4 * P, ldx=64, ldw=64,
             ldh=32)
    a.update(kw)
    return ff.lib.tsffn_gated(None, ctypes.byref(ff.GatedArgs(**a)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(F=0), INVALID), (dict(F=-8), INVALID), (dict(F=36, ldw=72, ldh=40), ALIGNMENT), (dict(F=2 ** 30), UNSUPPORTED),
    (dict(F=2 ** 62), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(dtype=4), UNSUPPORTED), (dict(layout=3), UNSUPPORTED),
    (dict(ldw=56), INVALID), (dict(ldh=36), ALIGNMENT), (dict(H=2 * P + 64), INVALID), (dict(H=None), INVALID),
    (dict(saved=3 * P), INVALID), (dict(reserved=3), INVALID),
])
def test_gated_refusals(ff, kw, code):
    assert _gated(ff, **kw) == code


def _gated_backward(ff, **kw):
    a = dict(M=4, F=32, K=64, dtype=0, dtype_dw=0, layout=0, act=4, dH=P, X=2 * P, W=3 * P, saved=4 * P, dX=5 * P,
             dW=6 * P, workspace=7 * P, lddh=32, ldx=64, ldw=64, lddx=64, lddw=64)
    a.update(kw)
    return ff.lib.tsffn_gated_backward(None, ctypes.byref(ff.GatedBackwardArgs(**a)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(F=12, lddh=16), ALIGNMENT), (dict(dX=None, dW=None), INVALID), (dict(saved=None), INVALID),
    (dict(workspace=None), INVALID), (dict(dX=None, X=None), INVALID), (dict(dW=None, W=None), INVALID),
    (dict(dtype_dw=1), UNSUPPORTED), (dict(dX=P), INVALID), (dict(workspace=4 * P), INVALID), (dict(lddh=24), INVALID),
])
def test_gated_backward_refusals(ff, kw, code):
    assert _gated_backward(ff, **kw) == code


def test_column_slices_of_one_buffer_do_not_overlap(ff):
    # X in columns [0, 64) and C in columns [64, 128) of the same 128-wide
    # rows: apart (refused for the missing handle only, and with another
    # stride for the overlap: the same code, so the bad stride tells)
    one = dict(ldx=128, ldc=128, C=P + 128, residual=None)
    assert _linear(ff, act=-1, **one) == INVALID
    assert _linear(ff, dtype_out=0, **one) == UNSUPPORTED      # got past the overlap check
    assert _linear(ff, dtype_out=0, ldx=136, ldc=128, C=P + 128, residual=None) == INVALID  # did not


def _clip(ff, grads, out, numel, dtype, max_norm=1.0, norm=9 * P):
    n = len(grads)
    return ff.lib.tsffn_clip_grad_norm(None, n, (ctypes.c_void_p * n)(*grads), (ctypes.c_void_p * n)(*out),
                                       (ctypes.c_int64 * n)(*numel), (ctypes.c_int32 * n)(*dtype), max_norm, norm, None)


@pytest.mark.parametrize("args,code", [
    (([P], [P], [-1], [1]), INVALID), (([P], [P], [4], [7]), INVALID), (([P], [P], [4], [3]), UNSUPPORTED),
    (([None], [P], [4], [1]), INVALID), (([P], [None], [4], [1]), INVALID),
    (([P + 1], [P + 1], [4], [1]), ALIGNMENT), (([P + 2], [2 * P], [4], [2]), ALIGNMENT),
    (([P, P + 4], [P, P + 4], [4, 4], [1, 1]), INVALID),          # two in place that overlap
    (([P, 2 * P], [2 * P, 3 * P], [4, 4], [1, 1]), INVALID),      # an output on another's input
    (([P], [P + 2], [4], [1]), INVALID),                          # shifted onto itself
    (([P, 2 * P], [3 * P, 3 * P], [4, 4], [1, 1]), INVALID),
    (([P], [P], [4], [1], float("nan")), INVALID), (([P], [P], [4], [1], -1.0), INVALID),
    (([P], [P], [4], [1], 1.0, None), INVALID), (([P], [P], [4], [1], 1.0, P + 4), INVALID),
    (([P], [P], [4], [1], 1.0, 9 * P + 2), ALIGNMENT),
])
def test_clip_refusals(ff, args, code):
    assert _clip(ff, *args) == code


def test_entry_points_refuse_null(ff):
    for f in (ff.lib.tsffn_linear, ff.lib.tsffn_linear_backward, ff.lib.tsffn_gated, ff.lib.tsffn_gated_backward):
        assert f(None, None, None) == INVALID
    assert ff.lib.tsffn_create(None) == INVALID
    assert ff.lib.tsffn_destroy(None) == OK
    assert ff.lib.tsffn_status(None) == INVALID


# ------------------------------------------------------------ the binding --

def test_binding_reads_strides(ff):
    w = torch.empty(48, 96, dtype=torch.bfloat16)
    assert ff._weights(w, "W") == (0, 96)
    assert ff._weights(w.t(), "W") == (1, 96)
    assert ff._weights(w[:, :40], "W") == (0, 96)
    assert ff._weights(w[:, :40].t(), "W") == (1, 96)
    assert ff._weights(w[:, :1], "W") == (0, 96)         # one column of a row-major matrix
    assert ff._weights(w[:, :1].t(), "W") == (1, 96)     # K = 1, stored N x K
    assert ff._weights(w[:1], "W") == (0, 96)            # K = 1
    assert ff._weights(w[:1].t(), "W") == (1, 96)        # N = 1, stored 1 x K
    assert ff._weights(torch.empty(5, 1), "W") == (1, 8)  # N = 1, dense: the same memory
    with pytest.raises(ValueError):
        ff._weights(w[:, ::2], "W")
    with pytest.raises(ValueError):
        ff._rows(w.t(), "X")
    assert ff._rows(w[:1, :33], "X") == 40               # a single row: any stride
    assert ff._rows(w[3:, :33], "X") == 96


def test_binding_refusals(ff):
    x, w = torch.empty(4, 64, dtype=torch.bfloat16), torch.empty(64, 32, dtype=torch.bfloat16)
    bad = [lambda: ff.linear(x, w.t()), lambda: ff.linear(x[0], w), lambda: ff.linear(x, w.half()),
           lambda: ff.linear(x, w, act="tanh"), lambda: ff.linear(x, w, C=torch.empty(4, 31, dtype=torch.bfloat16)),
           lambda: ff.linear(x, w, residual=torch.empty(4, 32)), lambda: ff.linear(x, w, bias=torch.empty(31)),
           lambda: ff.linear(x, w, residual=torch.empty(3, 32, dtype=torch.bfloat16)),
           lambda: ff.gated(x, torch.empty(64, 33, dtype=torch.bfloat16)), lambda: ff.gated(x, w, act="swish"),
           lambda: ff.linear_backward(torch.empty(4, 32, dtype=torch.bfloat16), x, w, act="gelu"),
           lambda: ff.linear_backward(torch.empty(4, 31, dtype=torch.bfloat16), x, w),
           lambda: ff.linear_backward(torch.empty(4, 32, dtype=torch.bfloat16), x, w,
                                      dW=torch.empty(32, 64, dtype=torch.bfloat16).t()),
           lambda: ff.linear_backward(torch.empty(4, 32, dtype=torch.bfloat16), x, w, torch.empty(4, 32).half(), "gelu"),
           lambda: ff.gated_backward(torch.empty(4, 16, dtype=torch.bfloat16), x, w, None),
           lambda: ff.clip_grad_norm([w.t()], 1.0), lambda: ff.clip_grad_norm([w], 1.0, out=[]),
           lambda: ff.clip_grad_norm([w], 1.0, out=[w.float()]),
           lambda: ff.clip_grad_norm([w], 1.0, norm=torch.empty(2))]
    for f in bad:
        with pytest.raises(ValueError):
            f()
