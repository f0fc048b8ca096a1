"""ctypes binding of the state-space block's operators in include/rnn.h: the
short causal convolution, the selective scan and the gated feed-forward.

As in block_ops.py, only argument marshalling happens here, and nothing
synchronises, so the calls can be captured into a graph. The C structs are
packed as bytes (a serving step's kernels take as long as filling the ctypes
classes would; those are there for callers of the C functions), and the sizes
of workspaces, which depend on the descriptor alone, are asked for once.
"""

import ctypes
import functools
import struct

import torch

from . import block_ops
from .binding import DTYPES
from .block_ops import (
    _I32, _I64, _P, _REF, _SZ, BlockContext, _buffer, _call, _dense_like, _lengths, _lib, _ok, _plain, _rows, _strided, _tensor,
)

ACTIVATIONS = {None: 0, "silu": 1, "gelu_tanh": 2, "sigmoid": 3}


class RnnCausalConvDesc(ctypes.Structure):
    _fields_ = [("dtype", _I32), ("T", _I32), ("B", _I32), ("C", _I32), ("W", _I32), ("activation", _I32), ("x_t", _I64),
                ("x_b", _I64)]


class RnnCausalConvIO(ctypes.Structure):
    _fields_ = [("x", _P), ("weight", _P), ("bias", _P), ("lengths", _P), ("state", _P), ("y", _P), ("state_n", _P)]


class RnnCausalConvGrads(ctypes.Structure):
    _fields_ = [("dy", _P), ("dstate_n", _P), ("dx", _P), ("dweight", _P), ("dbias", _P), ("dstate", _P)]


class RnnSelectiveScanDesc(ctypes.Structure):
    _fields_ = [("dtype", _I32), ("T", _I32), ("B", _I32), ("H", _I32), ("N", _I32), ("G", _I32), ("softplus", _I32),
                ("gate", _I32), ("x_t", _I64), ("x_b", _I64), ("dt_t", _I64), ("dt_b", _I64), ("z_t", _I64), ("z_b", _I64),
                ("B_t", _I64), ("B_b", _I64), ("B_g", _I64), ("C_t", _I64), ("C_b", _I64), ("C_g", _I64)]


class RnnSelectiveScanIO(ctypes.Structure):
    _fields_ = [("x", _P), ("dt", _P), ("z", _P), ("Bm", _P), ("Cm", _P), ("A", _P), ("D", _P), ("dt_bias", _P),
                ("lengths", _P), ("h0", _P), ("y", _P), ("h_n", _P)]


class RnnSelectiveScanGrads(ctypes.Structure):
    _fields_ = [("dy", _P), ("dh_n", _P), ("dx", _P), ("ddt", _P), ("dz", _P), ("dB", _P), ("dC", _P), ("dA", _P),
                ("dD", _P), ("ddt_bias", _P), ("dh0", _P)]


class RnnFeedForwardDesc(ctypes.Structure):
    _fields_ = [("dtype", _I32), ("activation", _I32), ("rows", _I64), ("N", _I32), ("F", _I32), ("N_out", _I32),
                ("aligned", _I32), ("x_ld", _I64), ("in_ld", _I64), ("out_ld", _I64), ("residual_ld", _I64)]


class RnnFeedForwardIO(ctypes.Structure):
    _fields_ = [("x", _P), ("w_in", _P), ("w_out", _P), ("residual", _P), ("y", _P)]


class RnnFeedForwardGrads(ctypes.Structure):
    _fields_ = [("dy", _P), ("dx", _P), ("dw_in", _P), ("dw_out", _P)]


# descriptor, pointers and gradients are taken as bytes or by reference
_SIZE = [_P, _REF(_SZ)]
block_ops._SIGNATURES.update({
    "rnn_causal_conv": [_P, _P, _P],
    "rnn_causal_conv_backward_workspace_bytes": _SIZE,
    "rnn_causal_conv_backward": [_P, _P, _P, _P, _SZ, _P],
    "rnn_selective_scan_workspace_bytes": _SIZE,
    "rnn_selective_scan_reserve_bytes": _SIZE,
    "rnn_selective_scan_backward_workspace_bytes": _SIZE,
    "rnn_selective_scan": [_P, _P, _P, _SZ, _P],
    "rnn_selective_scan_train": [_P, _P, _P, _SZ, _P, _SZ, _P],
    "rnn_selective_scan_backward": [_P, _P, _P, _P, _SZ, _P, _SZ, _P],
    "rnn_feed_forward_workspace_bytes": _SIZE,
    "rnn_feed_forward_train_workspace_bytes": _SIZE,
    "rnn_feed_forward_backward_workspace_bytes": _SIZE,
    "rnn_feed_forward_reserve_bytes": _SIZE,
    "rnn_feed_forward": [_P, _P, _P, _SZ, _P],
    "rnn_feed_forward_train": [_P, _P, _P, _SZ, _P, _SZ, _P],
    "rnn_feed_forward_backward": [_P, _P, _P, _P, _SZ, _P, _SZ, _P],
})

# the structs above, in the order of their fields
_CONV_DESC, _CONV_IO, _CONV_GRADS = struct.Struct("6i2q").pack, struct.Struct("7Q").pack, struct.Struct("6Q").pack
_SCAN_DESC, _SCAN_IO, _SCAN_GRADS = struct.Struct("8i12q").pack, struct.Struct("12Q").pack, struct.Struct("11Q").pack
_FEED_DESC, _FEED_IO, _FEED_GRADS = struct.Struct("2iq4i4q").pack, struct.Struct("5Q").pack, struct.Struct("4Q").pack


def _ptr(t):
    return 0 if t is None else t.data_ptr()


@functools.lru_cache(maxsize=4096)
def _bytes(fn, desc):
    n = _SZ(0)
    _ok(getattr(_lib(), fn)(desc, ctypes.byref(n)), fn)
    return n.value


def _activation(name, allowed):
    if name not in allowed:
        raise ValueError(f"activation: {name!r} is not one of {', '.join(map(repr, allowed))}")
    return ACTIVATIONS[name]


def _view(t, name, shape, like):
    """(t, its strides) where t's last dimension is contiguous, else of a dense copy."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.shape == shape and t.dtype is like.dtype and t.device == like.device:
        s = t.stride()
        if s[-1] == 1:
            return t, s
    t = _strided(t, name, shape, like)
    return t, t.stride()


# ---------------------------------------------------------------------------
# Short causal convolution
# ---------------------------------------------------------------------------

def _causal_conv(x, weight, bias, state, lengths, activation, train):
    act = _activation(activation, (None, "silu"))
    _tensor(x, "x", 3)
    _tensor(weight, "weight", 2)
    T, B, C = x.shape
    W = weight.shape[1]
    if W < 1:
        raise ValueError("weight: a filter has at least one tap")
    device, dtype = x.device, x.dtype
    x, (xt, xb, _) = _view(x, "x", x.shape, x)
    weight = _plain(weight, "weight", (C, W), dtype, device)
    bias = _plain(bias, "bias", (C,), dtype, device)
    state = _plain(state, "state", (W - 1, B, C), dtype, device)
    lengths = _lengths(lengths, B, T, device)
    y = _dense_like(x)
    state_n = x.new_empty((W - 1, B, C))
    desc = _CONV_DESC(DTYPES[dtype], T, B, C, W, act, xt, xb)
    io = _CONV_IO(x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(lengths), _ptr(state), y.data_ptr(), state_n.data_ptr())
    stream = _call("rnn_causal_conv", device, desc, io)
    if not train:
        return y, state_n
    return (y, state_n), BlockContext(device, stream, desc=desc, shape=(T, B, C, W), x=x, weight=weight, bias=bias,
                                      lengths=lengths, state=state)


def causal_conv(x, weight, bias=None, *, state=None, lengths=None, activation=None):
    """Causal convolution over time, one filter of W taps per channel:

        y_t = act(bias + sum_k weight[:, k] x_{t - W + 1 + k})

    x: [T, B, C] (float32 or bfloat16; may be a slice of a projection: only
    the last dimension has to be contiguous). weight: [C, W], W from 2 to 8;
    bias: [C]. state: [W - 1, B, C], the inputs before the first step, newest
    last (None = zeros). lengths: B row lengths in [0, T], a device int32
    tensor or host values (which are copied). activation: None or "silu".
    Returns (y [T, B, C] with zeros past a row's length, state_n [W - 1, B, C]
    to go on with). A serving step is T = 1 with the last call's state_n."""
    return _causal_conv(x, weight, bias, state, lengths, activation, False)


def causal_conv_train(x, weight, bias=None, *, state=None, lengths=None, activation=None):
    """causal_conv for training. Returns ((y, state_n), ctx); pass ctx to
    causal_conv_backward. ctx holds x, weight, bias, state and a device tensor
    of lengths: do not change them in place before the backward pass."""
    return _causal_conv(x, weight, bias, state, lengths, activation, True)


def causal_conv_backward(ctx, dy, dstate_n=None):
    """Gradients of causal_conv_train, given dy (shape and dtype of y) and
    optionally dstate_n. Returns (dx, dweight, dbias, dstate): dweight and
    dbias fp32, dbias None without a bias, dstate in x's dtype."""
    d, device, dtype = ctx.desc, ctx.device, ctx.x.dtype
    T, B, C, W = ctx.shape
    dy = _plain(dy, "dy", (T, B, C), dtype, device)
    dstate_n = _plain(dstate_n, "dstate_n", (W - 1, B, C), dtype, device)
    dx = _dense_like(dy)
    dw = torch.empty((C, W), dtype=torch.float32, device=device)
    db = None if ctx.bias is None else torch.empty((C,), dtype=torch.float32, device=device)
    dstate = dy.new_empty((W - 1, B, C))
    io = _CONV_IO(ctx.x.data_ptr(), ctx.weight.data_ptr(), _ptr(ctx.bias), _ptr(ctx.lengths), _ptr(ctx.state), 0, 0)
    grads = _CONV_GRADS(dy.data_ptr(), _ptr(dstate_n), dx.data_ptr(), dw.data_ptr(), _ptr(db), dstate.data_ptr())
    size = _bytes("rnn_causal_conv_backward_workspace_bytes", d)
    ws = _buffer(size, device)
    ctx._use(ctx.x, ctx.weight, ctx.bias, ctx.lengths, ctx.state)
    _call("rnn_causal_conv_backward", device, d, io, grads, _ptr(ws), size)
    return dx, dw, db, dstate


# ---------------------------------------------------------------------------
# Selective scan
# ---------------------------------------------------------------------------

def _selective_scan(x, dt, A, B, C, D, z, dt_bias, softplus, h0, lengths, train):
    _tensor(x, "x", 3)
    _tensor(B, "B", 4)
    _tensor(A, "A", 2)
    T, rows, H = shape = x.shape
    _, _, G, N = groups = B.shape
    if groups[:2] != shape[:2]:
        raise ValueError(f"B: shape {tuple(groups)} does not begin with {tuple(shape[:2])}")
    device = x.device
    x, (xt, xb, _) = _view(x, "x", shape, x)
    dt, (dtt, dtb, _) = _view(dt, "dt", shape, x)
    B, (Bt, Bb, Bg, _) = _view(B, "B", groups, x)
    C, (Ct, Cb, Cg, _) = _view(C, "C", groups, x)
    zt = zb = 0
    if z is not None:
        z, (zt, zb, _) = _view(z, "z", shape, x)
    A = _plain(A, "A", (H, N), torch.float32, device)
    D = _plain(D, "D", (H,), torch.float32, device)
    dt_bias = _plain(dt_bias, "dt_bias", (H,), torch.float32, device)
    h0 = _plain(h0, "h0", (rows, H, N), torch.float32, device)
    lengths = _lengths(lengths, rows, T, device)
    y = _dense_like(x)
    h_n = torch.empty((rows, H, N), dtype=torch.float32, device=device)
    desc = _SCAN_DESC(DTYPES[x.dtype], T, rows, H, N, G, 1 if softplus else 0, 0 if z is None else 1, xt, xb, dtt, dtb, zt, zb,
                      Bt, Bb, Bg, Ct, Cb, Cg)
    io = _SCAN_IO(x.data_ptr(), dt.data_ptr(), _ptr(z), B.data_ptr(), C.data_ptr(), A.data_ptr(), _ptr(D), _ptr(dt_bias),
                  _ptr(lengths), _ptr(h0), y.data_ptr(), h_n.data_ptr())
    size = _bytes("rnn_selective_scan_workspace_bytes", desc)
    ws = _buffer(size, device)
    if not train:
        _call("rnn_selective_scan", device, desc, io, _ptr(ws), size)
        return y, h_n
    rsize = _bytes("rnn_selective_scan_reserve_bytes", desc)
    reserve = _buffer(rsize, device)
    stream = _call("rnn_selective_scan_train", device, desc, io, _ptr(reserve), rsize, _ptr(ws), size)
    return (y, h_n), BlockContext(device, stream, desc=desc, shape=(T, rows, H, N), x=x, dt=dt, z=z, B=B, C=C, A=A, D=D, dt_bias=dt_bias,
                                  lengths=lengths, reserve=reserve)


def selective_scan(x, dt, A, B, C, D=None, *, z=None, dt_bias=None, softplus=True, h0=None, lengths=None):
    """Linear recurrence with a state of N numbers per channel and a step
    length of its own at every time:

        d_t = softplus(dt_t + dt_bias)                  (softplus=False: dt_t + dt_bias)
        h_t = exp(d_t A) h_{t-1} + d_t x_t B_t          (h: [H, N])
        y_t = (sum_n C_t h_t + D x_t) silu(z_t)         (z None: no factor)

    x, dt, z: [T, B, H], B, C: [T, B, G, N] (float32 or bfloat16; may be
    slices of projections: only the last dimension has to be contiguous).
    Channel h reads group h // (H // G); N is at most 64. A: fp32 [H, N],
    finite; D, dt_bias: fp32 [H]; h0: fp32 [B, H, N]. lengths: B row lengths
    in [0, T], a device int32 tensor or host values (which are copied).
    Returns (y [T, B, H] with zeros past a row's length, h_n fp32 [B, H, N]).
    A serving step is T = 1 with the last call's h_n as h0."""
    return _selective_scan(x, dt, A, B, C, D, z, dt_bias, softplus, h0, lengths, False)


def selective_scan_train(x, dt, A, B, C, D=None, *, z=None, dt_bias=None, softplus=True, h0=None, lengths=None):
    """selective_scan that also keeps the fp32 state at every 16th step.
    Returns ((y, h_n), ctx); pass ctx to selective_scan_backward. ctx holds the
    inputs (a device tensor of lengths among them): do not change them in place
    before the backward pass."""
    return _selective_scan(x, dt, A, B, C, D, z, dt_bias, softplus, h0, lengths, True)


def selective_scan_backward(ctx, dy, dh_n=None):
    """Gradients of selective_scan_train, given dy (shape and dtype of y) and
    optionally dh_n (fp32 [B, H, N]). Returns them by the inputs' names: "x",
    "dt", "z", "B", "C" in x's dtype, "A", "D", "dt_bias", "h0" in fp32; None
    for z, D and dt_bias where they were not given."""
    d, device, dtype = ctx.desc, ctx.device, ctx.x.dtype
    T, rows, H, N = ctx.shape
    dy = _plain(dy, "dy", (T, rows, H), dtype, device)
    dh_n = _plain(dh_n, "dh_n", (rows, H, N), torch.float32, device)

    def f32(*shape):
        return torch.empty(shape, dtype=torch.float32, device=device)

    g = {"x": _dense_like(dy), "dt": _dense_like(dy), "z": None if ctx.z is None else _dense_like(dy),
         "B": dy.new_empty(ctx.B.shape), "C": dy.new_empty(ctx.B.shape), "A": f32(H, N),
         "D": None if ctx.D is None else f32(H), "dt_bias": None if ctx.dt_bias is None else f32(H),
         "h0": f32(rows, H, N)}
    io = _SCAN_IO(ctx.x.data_ptr(), ctx.dt.data_ptr(), _ptr(ctx.z), ctx.B.data_ptr(), ctx.C.data_ptr(), ctx.A.data_ptr(),
                  _ptr(ctx.D), _ptr(ctx.dt_bias), _ptr(ctx.lengths), 0, 0, 0)
    grads = _SCAN_GRADS(dy.data_ptr(), _ptr(dh_n), *(_ptr(g[k]) for k in ("x", "dt", "z", "B", "C", "A", "D", "dt_bias", "h0")))
    size = _bytes("rnn_selective_scan_backward_workspace_bytes", d)
    ws = _buffer(size, device)
    ctx._use(ctx.x, ctx.dt, ctx.z, ctx.B, ctx.C, ctx.A, ctx.D, ctx.dt_bias, ctx.lengths, ctx.reserve)
    _call("rnn_selective_scan_backward", device, d, io, grads, _ptr(ctx.reserve),
          ctx.reserve.numel(), _ptr(ws), size)
    return g


# ---------------------------------------------------------------------------
# Gated feed-forward
# ---------------------------------------------------------------------------

def _weight(w, name, like):
    """(w, elements between its rows) of a matrix whose rows are contiguous."""
    _tensor(w, name, 2)
    rows, n = w.shape
    w, (ld, _) = _view(w, name, w.shape, like)
    if rows == 1:
        return w, n
    return (w, ld) if ld >= n else (w.contiguous(), n)


def _feed_forward(x, w_in, w_out, residual, activation, train):
    act = _activation(activation, ("silu", "gelu_tanh", "sigmoid"))
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x must be a tensor of at least one dimension")
    _tensor(x, "x", x.dim())
    device, dtype, n = x.device, x.dtype, x.shape[-1]
    rows = x.numel() // n if n else 0
    w_in, in_ld = _weight(w_in, "w_in", x)
    w_out, out_ld = _weight(w_out, "w_out", x)
    n_out, F = w_out.shape
    if tuple(w_in.shape) != (2 * F, n):
        raise ValueError(f"w_in: shape {tuple(w_in.shape)} != {(2 * F, n)}")
    shape = x.shape[:-1] + (n_out,)
    x, x_ld = _rows(x)
    r_ld = 0
    if residual is not None:
        residual, r_ld = _rows(_strided(residual, "residual", shape, x))
    y = x.new_empty(shape)
    aligned = (x.data_ptr() | w_in.data_ptr() | w_out.data_ptr()) % 16 == 0
    fields = (DTYPES[dtype], act, rows, n, F, n_out, 1 if aligned else 0, x_ld, in_ld, out_ld, r_ld)
    desc = _FEED_DESC(*fields)
    io = _FEED_IO(x.data_ptr(), w_in.data_ptr(), w_out.data_ptr(), _ptr(residual), y.data_ptr())
    if not train:
        size = _bytes("rnn_feed_forward_workspace_bytes", desc)
        ws = _buffer(size, device)
        _call("rnn_feed_forward", device, desc, io, _ptr(ws), size)
        return y
    size = _bytes("rnn_feed_forward_train_workspace_bytes", desc)
    ws = _buffer(size, device)
    rsize = _bytes("rnn_feed_forward_reserve_bytes", desc)
    reserve = _buffer(rsize, device)
    stream = _call("rnn_feed_forward_train", device, desc, io, _ptr(reserve), rsize, _ptr(ws), size)
    return y, BlockContext(device, stream, fields=fields, x=x, w_in=w_in, w_out=w_out, reserve=reserve, shape=shape)


def feed_forward(x, w_in, w_out, *, residual=None, activation="silu"):
    """Gated feed-forward over the last dimension of x [..., N] (float32 or
    bfloat16):

        y = (act(x w_in[:F]^T) * (x w_in[F:]^T)) w_out^T + residual

    w_in: [2 F, N], the gate's rows first; w_out: [N_out, F]; residual:
    [..., N_out] or None. activation: "silu", "gelu_tanh" or "sigmoid". x, the
    weights and the residual may be strided (contiguous last dimension).
    Returns y [..., N_out]. In bf16 the hidden values are rounded once on the
    way into the second product. A serving step is a few rows (64 at most take
    a path of their own, which reads operands at any address; with more, one
    that is off 16 bytes, or whose rows are no whole 16 bytes, is copied)."""
    return _feed_forward(x, w_in, w_out, residual, activation, False)


def feed_forward_train(x, w_in, w_out, *, residual=None, activation="silu"):
    """feed_forward that also keeps both projections in fp32 and the hidden
    values (in all 12 bytes a row and hidden unit in fp32, 10 in bf16).
    Returns (y, ctx); pass ctx to feed_forward_backward. ctx holds x and the
    weights: do not change them in place before the backward pass."""
    return _feed_forward(x, w_in, w_out, residual, activation, True)


def feed_forward_backward(ctx, dy):
    """Gradients of feed_forward_train, given dy (shape and dtype of y).
    Returns (dx, dw_in, dw_out) in x's dtype; the residual's gradient is dy."""
    x, device = ctx.x, ctx.device
    dy = _plain(dy, "dy", ctx.shape, x.dtype, device)
    _, _, _, n, F, n_out, aligned = ctx.fields[:7]
    if dy.data_ptr() % 16:
        aligned = 0
    d = _FEED_DESC(*ctx.fields[:6], aligned, *ctx.fields[7:])
    dx = dy.new_empty(ctx.shape[:-1] + (n,))
    dw_in, dw_out = dy.new_empty((2 * F, n)), dy.new_empty((n_out, F))
    io = _FEED_IO(x.data_ptr(), ctx.w_in.data_ptr(), ctx.w_out.data_ptr(), 0, 0)
    grads = _FEED_GRADS(dy.data_ptr(), dx.data_ptr(), dw_in.data_ptr(), dw_out.data_ptr())
    size = _bytes("rnn_feed_forward_backward_workspace_bytes", d)
    ws = _buffer(size, device)
    ctx._use(x, ctx.w_in, ctx.w_out, ctx.reserve)
    _call("rnn_feed_forward_backward", device, d, io, grads, _ptr(ctx.reserve),
          ctx.reserve.numel(), _ptr(ws), size)
    return dx, dw_in, dw_out
