"""ctypes binding of the state-space block's operators in include/rnn.h: the
short causal convolution, the selective scan and the gated feed-forward.

As in block_ops.py, only argument marshalling happens here, and nothing
synchronises, so the calls can be captured into a graph.
"""

import ctypes

import torch

from . import block_ops
from .binding import DTYPES
from .block_ops import (
    _F32, _I32, _I64, _P, _REF, _SZ, BlockContext, _buffer, _bytes, _call, _dense_like, _lengths, _plain, _ptr, _strided,
    _tensor,
)

ACTIVATIONS = {None: 0, "silu": 1, "gelu_tanh": 2, "sigmoid": 3}


class RnnCausalConvDesc(ctypes.Structure):
    _fields_ = [("dtype", _I32), ("T", _I32), ("B", _I32), ("C", _I32), ("W", _I32), ("activation", _I32), ("x_t", _I64),
                ("x_b", _I64)]


class RnnCausalConvIO(ctypes.Structure):
    _fields_ = [("x", _P), ("weight", _P), ("bias", _P), ("lengths", _P), ("state", _P), ("y", _P), ("state_n", _P)]


class RnnCausalConvGrads(ctypes.Structure):
    _fields_ = [("dy", _P), ("dstate_n", _P), ("dx", _P), ("dweight", _P), ("dbias", _P), ("dstate", _P)]


block_ops._SIGNATURES.update({
    "rnn_causal_conv": [_REF(RnnCausalConvDesc), _REF(RnnCausalConvIO), _P],
    "rnn_causal_conv_backward_workspace_bytes": [_REF(RnnCausalConvDesc), _REF(_SZ)],
    "rnn_causal_conv_backward": [_REF(RnnCausalConvDesc), _REF(RnnCausalConvIO), _REF(RnnCausalConvGrads), _P, _SZ, _P],
})


def _activation(name, allowed):
    if name not in allowed:
        raise ValueError(f"activation: {name!r} is not one of {', '.join(map(repr, allowed))}")
    return ACTIVATIONS[name]


# ---------------------------------------------------------------------------
# Short causal convolution
# ---------------------------------------------------------------------------

def _causal_conv(x, weight, bias, state, lengths, activation, train):
    act = _activation(activation, (None, "silu"))
    _tensor(x, "x", 3)
    _tensor(weight, "weight", 2)
    T, B, C = x.shape
    W = weight.shape[1]
    device, dtype = x.device, x.dtype
    x = _strided(x, "x", x.shape, x)
    weight = _plain(weight, "weight", (C, W), dtype, device)
    bias = _plain(bias, "bias", (C,), dtype, device)
    state = _plain(state, "state", (W - 1, B, C), dtype, device)
    lengths = _lengths(lengths, B, T, device)
    y = _dense_like(x)
    state_n = x.new_empty((W - 1, B, C))
    xt, xb, _ = x.stride()
    desc = RnnCausalConvDesc(DTYPES[dtype], T, B, C, W, act, xt, xb)
    io = RnnCausalConvIO(x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(lengths), _ptr(state), y.data_ptr(),
                         state_n.data_ptr())
    stream = _call("rnn_causal_conv", device, ctypes.byref(desc), ctypes.byref(io))
    if not train:
        return y, state_n
    return (y, state_n), BlockContext(device, stream, desc=desc, x=x, weight=weight, bias=bias, lengths=lengths, state=state)


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
    dy = _plain(dy, "dy", (d.T, d.B, d.C), dtype, device)
    dstate_n = _plain(dstate_n, "dstate_n", (d.W - 1, d.B, d.C), dtype, device)
    dx = _dense_like(dy)
    dw = torch.empty((d.C, d.W), dtype=torch.float32, device=device)
    db = None if ctx.bias is None else torch.empty((d.C,), dtype=torch.float32, device=device)
    dstate = dy.new_empty((d.W - 1, d.B, d.C))
    io = RnnCausalConvIO(ctx.x.data_ptr(), ctx.weight.data_ptr(), _ptr(ctx.bias), _ptr(ctx.lengths), _ptr(ctx.state), None, None)
    grads = RnnCausalConvGrads(dy.data_ptr(), _ptr(dstate_n), dx.data_ptr(), dw.data_ptr(), _ptr(db), dstate.data_ptr())
    size = _bytes("rnn_causal_conv_backward_workspace_bytes", d)
    ws = _buffer(size, device)
    ctx._use(ctx.x, ctx.weight, ctx.bias, ctx.lengths, ctx.state)
    _call("rnn_causal_conv_backward", device, ctypes.byref(d), ctypes.byref(io), ctypes.byref(grads), _ptr(ws), size)
    return dx, dw, db, dstate
