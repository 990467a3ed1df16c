"""Python binding of the feed-forward operators (include/tsffn.h).

    linear(X, W, ...)            C = act(X W + b) + R
    linear_backward(dC, ...)     dX, dW, db of it
    gated(X, W, ...)             H = act(X Wg) * (X Wu),  W = [Wg | Wu]
    gated_backward(dH, ...)      dX, dW of it
    clip_grad_norm(grads, ...)   gradients scaled to a largest global norm

Argument marshalling only, as in tsgemm: every step runs in the CUDA kernels
of libtsgemm.so.  Tensors are on the current device; matrices have unit
stride along their rows and a row stride that is a multiple of 16 bytes (a
contiguous matrix whose rows are, or a column slice of one).  W is given as
(K x N): row-major, or the transposed view of weights stored N x K (for
example weight.t() of a layer whose weight is N x K).

Calls run on the current stream (or `stream`) with a workspace that belongs
to that stream: see handle().
"""
import ctypes
from array import array

from .tsgemm import (BF16, F16, F32, LAYOUT_RCR, LAYOUT_RRR, _check, _stream_handle, dtype_code, lib, status_string)

ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU, ACT_SIGMOID = range(6)
_ACTS = {"none": ACT_NONE, "relu": ACT_RELU, "gelu": ACT_GELU, "gelu_tanh": ACT_GELU_TANH, "silu": ACT_SILU,
         "sigmoid": ACT_SIGMOID}

# Every entry point include/tsffn.h declares.
EXPORTS = ("tsffn_create", "tsffn_destroy", "tsffn_status", "tsffn_linear", "tsffn_linear_backward", "tsffn_gated",
           "tsffn_gated_backward", "tsffn_clip_grad_norm")

_i64, _i32, _vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p


def _fields(sizes, ints, ptrs, strides):
    return ([(n, _i64) for n in sizes.split()] + [(n, _i32) for n in ints.split()] +
            [(n, _vp) for n in ptrs.split()] + [(n, _i64) for n in strides.split()])


class LinearArgs(ctypes.Structure):
    """Mirror of tsffn_linear_args."""
    _fields_ = _fields("M N K", "dtype dtype_out dtype_bias layout act reserved", "X W bias residual C saved",
                       "ldx ldw ldr ldc")


class LinearBackwardArgs(ctypes.Structure):
    """Mirror of tsffn_linear_backward_args."""
    _fields_ = _fields("M N K", "dtype dtype_dw dtype_bias layout act reserved",
                       "dC X W saved dX dW dbias workspace", "lddc ldx ldw lddx lddw")


class GatedArgs(ctypes.Structure):
    """Mirror of tsffn_gated_args."""
    _fields_ = _fields("M F K", "dtype layout act reserved", "X W H saved", "ldx ldw ldh")


class GatedBackwardArgs(ctypes.Structure):
    """Mirror of tsffn_gated_backward_args."""
    _fields_ = _fields("M F K", "dtype dtype_dw layout act", "dH X W saved dX dW workspace",
                       "lddh ldx ldw lddx lddw")


lib.tsffn_create.restype = _i32
lib.tsffn_create.argtypes = [ctypes.POINTER(_vp)]
for _name in ("tsffn_destroy", "tsffn_status"):
    getattr(lib, _name).restype = _i32
    getattr(lib, _name).argtypes = [_vp]
for _name in ("tsffn_linear", "tsffn_linear_backward", "tsffn_gated", "tsffn_gated_backward"):
    getattr(lib, _name).restype = _i32
    getattr(lib, _name).argtypes = [_vp, _vp, _vp]
lib.tsffn_clip_grad_norm.restype = _i32
lib.tsffn_clip_grad_norm.argtypes = [_vp, _i64, _vp, _vp, _vp, _vp, ctypes.c_float, _vp, _vp]


class Handle:
    """The workspace of the calls made with it, on the current device.  Its
    calls must be ordered on one stream (replays of a graph they were
    captured into included)."""

    def __init__(self):
        self._h = _vp()
        _check(lib.tsffn_create(ctypes.byref(self._h)), "tsffn_create")

    @property
    def raw(self):
        return self._h.value

    def status(self):
        """Device status word after the calls have completed (0 = OK)."""
        return lib.tsffn_status(self._h)

    def close(self):
        if self._h:
            lib.tsffn_destroy(self._h)
            self._h = _vp()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


_handles = {}


def handle(stream=None):
    """The handle of a stream (default: the current one) of the current
    device, made on first use and kept.  To replay a captured graph beside
    eager calls, capture it with a Handle() of its own (`handle=`)."""
    import torch
    s = _stream_handle(stream)
    key = (torch.cuda.current_device(), s)
    h = _handles.get(key)
    if h is None:
        h = _handles[key] = Handle()
    return h


def status(stream=None):
    """handle(stream).status()."""
    return handle(stream).status()


def _act(act):
    if isinstance(act, int):
        return act
    try:
        return _ACTS[act]
    except KeyError:
        raise ValueError("unknown activation %r" % (act,)) from None


def _rows(t, what):
    """Row stride of a 2-D tensor with unit stride along its rows."""
    r, c = t.shape
    s0, s1 = t.stride()
    if c > 1 and s1 != 1:
        raise ValueError("%s must have unit stride along its rows" % what)
    if r == 1:  # the stride of a single row says nothing
        return (c + 7) // 8 * 8
    return s0


def _weights(W, what):
    """(layout, row stride) of a K x N tensor stored K x N or N x K."""
    K, N = W.shape
    s0, s1 = W.stride()
    if (s0 == 1 and K > 1 and (N == 1 or s1 != 1)) or (K == 1 and N > 1 and s1 != 1):
        return LAYOUT_RCR, ((K + 7) // 8 * 8 if N == 1 else s1)
    if s1 != 1 and N > 1:
        raise ValueError("%s must be row-major or the transposed view of a row-major matrix" % what)
    return LAYOUT_RRR, ((N + 7) // 8 * 8 if K == 1 else s0)


def _empty(rows, cols, dtype, device):
    """rows x cols with rows that start on 16-byte boundaries."""
    import torch
    ld = (cols + 7) // 8 * 8
    return torch.empty((rows, ld), dtype=dtype, device=device)[:, :cols]


def _empty_weights(W, layout, dtype):
    """A K x N tensor stored as W is."""
    K, N = W.shape
    if layout == LAYOUT_RCR:
        return _empty(N, K, dtype, W.device).t()
    return _empty(K, N, dtype, W.device)


def _shape(t, shape, what):
    if t is not None and tuple(t.shape) != shape:
        raise ValueError("%s must be %s" % (what, " x ".join(map(str, shape))))


def _vec(t, n, what):
    if t is not None and (tuple(t.shape) != (n,) or (n > 1 and t.stride(0) != 1)):
        raise ValueError("%s must be a contiguous vector of %d" % (what, n))


def _same(dtype, **tensors):
    for name, t in tensors.items():
        if t is not None and t.dtype != dtype:
            raise ValueError("%s must be %s, as X is" % (name, dtype))


def _p(t):
    return None if t is None else t.data_ptr()


def _saved_ok(saved, rows, cols):
    import torch
    if saved is not None and (saved.dtype != torch.float32 or tuple(saved.shape) != (rows, cols) or
                              not saved.is_contiguous()):
        raise ValueError("saved must be the contiguous %d x %d float32 tensor of the forward pass" % (rows, cols))


def linear(X, W, bias=None, act="none", residual=None, C=None, out_dtype=None, save=False, stream=None, handle=None):
    """C = act(X W + bias) + residual for X (M x K) and W (K x N), both
    float16 or both bfloat16.  C and residual are of that type or float32
    (`out_dtype`, or C's), bias of that type or float32; residual may be C.
    act: "none", "relu", "gelu" (of the normal distribution), "gelu_tanh",
    "silu" or "sigmoid".

    With `save`, returns (C, saved) for linear_backward: the float32
    pre-activations X W + bias, in rows padded to a multiple of 8, or None
    without an activation, whose backward pass needs none."""
    import torch
    if X.dim() != 2 or W.dim() != 2 or X.shape[1] != W.shape[0]:
        raise ValueError("expected X (M x K) and W (K x N)")
    M, K = X.shape
    N = W.shape[1]
    _same(X.dtype, W=W)
    code = _act(act)
    if C is None:
        C = _empty(M, N, X.dtype if out_dtype is None else out_dtype, X.device)
    _shape(C, (M, N), "C")
    if out_dtype is not None and C.dtype != out_dtype:
        raise ValueError("C is not of out_dtype")
    _shape(residual, (M, N), "residual")
    if residual is not None and residual.dtype != C.dtype:
        raise ValueError("residual must have C's dtype")
    _vec(bias, N, "bias")
    layout, ldw = _weights(W, "W")
    saved = None
    if save and code != ACT_NONE:
        saved = torch.empty((M, (N + 7) // 8 * 8), dtype=torch.float32, device=X.device)
    din = dtype_code(X.dtype)
    args = LinearArgs(M, N, K, din, dtype_code(C.dtype), din if bias is None else dtype_code(bias.dtype), layout, code,
                      0, X.data_ptr(), W.data_ptr(), _p(bias), _p(residual), C.data_ptr(), _p(saved), _rows(X, "X"),
                      ldw, 0 if residual is None else _rows(residual, "residual"), _rows(C, "C"))
    s = _stream_handle(stream)
    h = handle if handle is not None else _handle_of(s)
    _check(lib.tsffn_linear(h.raw, ctypes.byref(args), s), "tsffn_linear")
    return (C, saved) if save else C


def linear_backward(dC, X, W, saved=None, act="none", dX=None, dW=None, dbias=None, need=("dX", "dW"), dw_dtype=None,
                    stream=None, handle=None):
    """Gradients of linear(X, W, bias, act): (dX, dW, dbias) for the gradient
    dC (M x N) of its result; the residual's gradient is dC itself.

    `saved` is what linear(..., save=True) returned.  Outputs that are given
    are written; of the others those named in `need` ("dX", "dW", "dbias")
    are made, dW stored as W is, and the rest are None.  dW and dbias may be
    float32."""
    import torch
    if dC.dim() != 2 or X.dim() != 2 or W.dim() != 2:
        raise ValueError("expected dC (M x N), X (M x K) and W (K x N)")
    M, N = dC.shape
    K = X.shape[1]
    _shape(X, (M, K), "X")
    _shape(W, (K, N), "W")
    _same(X.dtype, W=W, dC=dC, dX=dX)
    code = _act(act)
    layout, ldw = _weights(W, "W")
    if dX is None and "dX" in need:
        dX = _empty(M, K, X.dtype, X.device)
    if dW is None and "dW" in need:
        dW = _empty_weights(W, layout, dw_dtype or X.dtype)
    if dbias is None and "dbias" in need:
        dbias = torch.empty(N, dtype=X.dtype, device=X.device)
    _shape(dX, (M, K), "dX")
    _shape(dW, (K, N), "dW")
    _vec(dbias, N, "dbias")
    lddw = _like_weights(dW, layout)
    ldz = (N + 7) // 8 * 8
    if code == ACT_NONE:
        saved = None
    elif saved is None:
        raise ValueError("saved is needed with an activation")
    _saved_ok(saved, M, ldz)
    ws = None
    if code != ACT_NONE and (dX is not None or dW is not None):
        ws = torch.empty((M, ldz), dtype=X.dtype, device=X.device)
    din = dtype_code(X.dtype)
    args = LinearBackwardArgs(M, N, K, din, din if dW is None else dtype_code(dW.dtype),
                              din if dbias is None else dtype_code(dbias.dtype), layout, code, 0, dC.data_ptr(),
                              X.data_ptr(), W.data_ptr(), _p(saved), _p(dX), _p(dW), _p(dbias), _p(ws),
                              _rows(dC, "dC"), _rows(X, "X"), ldw, 0 if dX is None else _rows(dX, "dX"), lddw)
    s = _stream_handle(stream)
    h = handle if handle is not None else _handle_of(s)
    _check(lib.tsffn_linear_backward(h.raw, ctypes.byref(args), s), "tsffn_linear_backward")
    return dX, dW, dbias


def gated(X, W, act="silu", H=None, save=False, stream=None, handle=None):
    """H = act(X Wg) * (X Wu) for X (M x K) and W = [Wg | Wu] (K x 2F), both
    float16 or both bfloat16; F a multiple of 8.  Both products, the
    activation and the product of the two run in one kernel.

    With `save`, returns (H, saved) for gated_backward: the float32 products
    (M x 2F)."""
    import torch
    if X.dim() != 2 or W.dim() != 2 or X.shape[1] != W.shape[0] or W.shape[1] % 2:
        raise ValueError("expected X (M x K) and W (K x 2F)")
    M, K = X.shape
    F = W.shape[1] // 2
    _same(X.dtype, W=W, H=H)
    code = _act(act)
    if H is None:
        H = _empty(M, F, X.dtype, X.device)
    _shape(H, (M, F), "H")
    layout, ldw = _weights(W, "W")
    saved = torch.empty((M, 2 * F), dtype=torch.float32, device=X.device) if save else None
    args = GatedArgs(M, F, K, dtype_code(X.dtype), layout, code, 0, X.data_ptr(), W.data_ptr(), H.data_ptr(),
                     _p(saved), _rows(X, "X"), ldw, _rows(H, "H"))
    s = _stream_handle(stream)
    h = handle if handle is not None else _handle_of(s)
    _check(lib.tsffn_gated(h.raw, ctypes.byref(args), s), "tsffn_gated")
    return (H, saved) if save else H


def gated_backward(dH, X, W, saved, act="silu", dX=None, dW=None, need=("dX", "dW"), dw_dtype=None, stream=None,
                   handle=None):
    """Gradients of gated(X, W, act): (dX, dW) for the gradient dH (M x F) of
    its result; `saved`, `need` and `dw_dtype` as for linear_backward."""
    import torch
    if dH.dim() != 2 or X.dim() != 2 or W.dim() != 2:
        raise ValueError("expected dH (M x F), X (M x K) and W (K x 2F)")
    M, F = dH.shape
    K = X.shape[1]
    _shape(X, (M, K), "X")
    _shape(W, (K, 2 * F), "W")
    _same(X.dtype, W=W, dH=dH, dX=dX)
    code = _act(act)
    layout, ldw = _weights(W, "W")
    if dX is None and "dX" in need:
        dX = _empty(M, K, X.dtype, X.device)
    if dW is None and "dW" in need:
        dW = _empty_weights(W, layout, dw_dtype or X.dtype)
    _shape(dX, (M, K), "dX")
    _shape(dW, (K, 2 * F), "dW")
    lddw = _like_weights(dW, layout)
    if saved is None:
        raise ValueError("saved is needed")
    _saved_ok(saved, M, 2 * F)
    ws = torch.empty((M, 2 * F), dtype=X.dtype, device=X.device)
    din = dtype_code(X.dtype)
    args = GatedBackwardArgs(M, F, K, din, din if dW is None else dtype_code(dW.dtype), layout, code, dH.data_ptr(),
                             X.data_ptr(), W.data_ptr(), saved.data_ptr(), _p(dX), _p(dW), ws.data_ptr(),
                             _rows(dH, "dH"), _rows(X, "X"), ldw, 0 if dX is None else _rows(dX, "dX"), lddw)
    s = _stream_handle(stream)
    h = handle if handle is not None else _handle_of(s)
    _check(lib.tsffn_gated_backward(h.raw, ctypes.byref(args), s), "tsffn_gated_backward")
    return dX, dW


def clip_grad_norm(grads, max_norm, out=None, norm=None, stream=None, handle=None):
    """Scale the dense tensors `grads` (float16, bfloat16 or float32, mixed)
    by min(1, max_norm / (n + 1e-6)), n the 2-norm of all their values, in
    place or into the tensors `out` (same sizes and types).  Returns n as a
    float32 tensor on the device (`norm`, if given: one value); the host does
    not wait for it."""
    import torch
    grads = list(grads)
    outs = grads if out is None else list(out)
    if len(outs) != len(grads):
        raise ValueError("out must have a tensor for each of grads")
    for g in grads:
        if not g.is_contiguous():
            raise ValueError("gradients must be contiguous")
    if out is not None:
        for g, o in zip(grads, outs):
            if o.dtype != g.dtype or o.numel() != g.numel() or not o.is_contiguous():
                raise ValueError("each of out must be contiguous, of its gradient's size and type")
    if norm is None:
        norm = torch.empty((), dtype=torch.float32, device=grads[0].device if grads else "cuda")
    elif norm.dtype != torch.float32 or norm.numel() != 1:
        raise ValueError("norm must be one float32 value")
    codes = {}
    kinds = array("i")
    for g in grads:
        k = codes.get(g.dtype)
        if k is None:
            k = codes[g.dtype] = dtype_code(g.dtype)
        kinds.append(k)
    ins = array("Q", [g.data_ptr() for g in grads])
    to = ins if out is None else array("Q", [o.data_ptr() for o in outs])
    sizes = array("q", [g.numel() for g in grads])
    s = _stream_handle(stream)
    h = handle if handle is not None else _handle_of(s)
    _check(lib.tsffn_clip_grad_norm(h.raw, len(grads), ins.buffer_info()[0], to.buffer_info()[0],
                                    sizes.buffer_info()[0], kinds.buffer_info()[0], float(max_norm), norm.data_ptr(),
                                    s), "tsffn_clip_grad_norm")
    return norm


def _handle_of(s):
    import torch
    h = _handles.get((torch.cuda.current_device(), s))
    return h if h is not None else handle(s)


def _like_weights(dW, layout):
    """dW's row stride; it has to be stored as W is."""
    if dW is None:
        return 0
    K, N = dW.shape
    if K > 1 and N > 1:
        got, ld = _weights(dW, "dW")
        if got != layout:
            raise ValueError("dW must be stored as W is")
        return ld
    rows, cols = (N, K) if layout == LAYOUT_RCR else (K, N)
    t = dW.t() if layout == LAYOUT_RCR else dW
    return (cols + 7) // 8 * 8 if rows == 1 else t.stride(0)


__all__ = ["BF16", "F16", "F32", "Handle", "clip_grad_norm", "gated", "gated_backward", "handle", "linear",
           "linear_backward", "status", "status_string"]
