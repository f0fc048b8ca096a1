"""ctypes binding of the decoder block's operators in include/rnn.h: layer
norm, the gated linear scan and cross attention.

As in binding.py, only argument marshalling happens here: checks, strides,
outputs and workspace from torch, and the call on torch's current HIP stream
of the tensors' device. Nothing synchronises, so the calls can be captured
into a graph.
"""

import ctypes

import torch

from . import binding
from .binding import DTYPES, RnnError, _check, _dense

_P, _I32, _I64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class RnnNormDesc(ctypes.Structure):
    _fields_ = [("dtype", _I32), ("N", _I32), ("rows", _I64), ("x_ld", _I64), ("residual_ld", _I64),
                ("eps", ctypes.c_float), ("reserved", _I32)]


class RnnGatedScanDesc(ctypes.Structure):
    _fields_ = [("dtype", _I32), ("T", _I32), ("B", _I32), ("H", _I32), ("reverse", _I32), ("input_gate", _I32),
                ("x_t", _I64), ("x_b", _I64), ("f_t", _I64), ("f_b", _I64), ("i_t", _I64), ("i_b", _I64)]


class RnnGatedScanIO(ctypes.Structure):
    _fields_ = [("x", _P), ("f", _P), ("i", _P), ("lengths", _P), ("h0", _P), ("y", _P), ("h_n", _P)]


class RnnGatedScanGrads(ctypes.Structure):
    _fields_ = [("dy", _P), ("dh_n", _P), ("dx", _P), ("df", _P), ("di", _P), ("dh0", _P)]


class RnnAttentionDesc(ctypes.Structure):
    _fields_ = [("dtype", _I32), ("B", _I32), ("Tq", _I32), ("Tk", _I32), ("heads", _I32), ("kv_heads", _I32),
                ("D", _I32), ("scale", ctypes.c_float), ("q_t", _I64), ("q_b", _I64), ("q_h", _I64), ("k_t", _I64),
                ("k_b", _I64), ("k_h", _I64), ("v_t", _I64), ("v_b", _I64), ("v_h", _I64)]


class RnnAttentionIO(ctypes.Structure):
    _fields_ = [("q", _P), ("k", _P), ("v", _P), ("lengths", _P), ("o", _P)]


class RnnAttentionGrads(ctypes.Structure):
    _fields_ = [("d_o", _P), ("dq", _P), ("dk", _P), ("dv", _P)]


_REF = ctypes.POINTER
_SIGNATURES = {
    "rnn_layer_norm": [_REF(RnnNormDesc)] + [_P] * 8,
    "rnn_layer_norm_backward_workspace_bytes": [_REF(RnnNormDesc), _REF(_SZ)],
    "rnn_layer_norm_backward": [_REF(RnnNormDesc)] + [_P] * 9 + [_SZ, _P],
    "rnn_gated_scan_workspace_bytes": [_REF(RnnGatedScanDesc), _REF(_SZ)],
    "rnn_gated_scan_reserve_bytes": [_REF(RnnGatedScanDesc), _REF(_SZ)],
    "rnn_gated_scan": [_REF(RnnGatedScanDesc), _REF(RnnGatedScanIO), _P, _SZ, _P],
    "rnn_gated_scan_train": [_REF(RnnGatedScanDesc), _REF(RnnGatedScanIO), _P, _SZ, _P, _SZ, _P],
    "rnn_gated_scan_backward": [_REF(RnnGatedScanDesc), _REF(RnnGatedScanIO), _REF(RnnGatedScanGrads), _P, _SZ, _P, _SZ,
                                _P],
    "rnn_cross_attention_workspace_bytes": [_REF(RnnAttentionDesc), _REF(_SZ)],
    "rnn_cross_attention_reserve_bytes": [_REF(RnnAttentionDesc), _REF(_SZ)],
    "rnn_cross_attention_backward_workspace_bytes": [_REF(RnnAttentionDesc), _REF(_SZ)],
    "rnn_cross_attention": [_REF(RnnAttentionDesc), _REF(RnnAttentionIO), _P, _SZ, _P],
    "rnn_cross_attention_train": [_REF(RnnAttentionDesc), _REF(RnnAttentionIO), _P, _SZ, _P, _SZ, _P],
    "rnn_cross_attention_backward": [_REF(RnnAttentionDesc), _REF(RnnAttentionIO), _REF(RnnAttentionGrads), _P, _SZ, _P,
                                     _SZ, _P],
}

_ready = None


def _lib():
    global _ready
    if _ready is None:
        L = binding.lib()
        for name, args in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = ctypes.c_int
            fn.argtypes = args
        _ready = L
    return _ready


_device = torch.cuda.current_device
# the handle alone, without a Stream object around it (1 us less a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(name, device, *args):
    """Calls the C function on the device's current stream, with that device
    current, and returns the stream's handle."""
    index = device.index
    if _device() == index:
        stream = _raw_stream(index)
        status = getattr(_lib(), name)(*args, stream)
    else:
        with torch.cuda.device(index):
            stream = _raw_stream(index)
            status = getattr(_lib(), name)(*args, stream)
    if status != 0:
        raise RnnError(status, name)
    return stream


def _ok(status, where):
    if status != 0:
        raise RnnError(status, where)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _bytes(fn, desc):
    n = _SZ(0)
    _ok(getattr(_lib(), fn)(ctypes.byref(desc), ctypes.byref(n)), fn)
    return n.value


def _buffer(n, device):
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _tensor(t, name, dims):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if t.dim() != dims:
        raise ValueError(f"{name}: expected {dims} dimensions, got shape {tuple(t.shape)}")
    if t.dtype not in DTYPES:
        raise ValueError(f"{name}: dtype {t.dtype} not supported (float32, bfloat16)")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")


def _strided(t, name, shape, like):
    """t itself where its last dimension is contiguous, else a dense copy."""
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if t.dtype != like.dtype:
        raise ValueError(f"{name}: dtype {t.dtype} != {like.dtype}")
    if t.device != like.device:
        raise ValueError(f"{name}: device {t.device} != {like.device}")
    return t if t.shape[-1] == 1 or t.stride(-1) == 1 else _dense(t)


def _plain(t, name, shape, dtype, device):
    """_check with a short way for a tensor that is as it should be."""
    if t is None or (t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous()):
        return t
    return _check(t, name, shape, dtype, device)


def _dense_like(t):
    """A new dense tensor of t's shape."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _lengths(lengths, B, T, device):
    """A device int32 tensor of the B row lengths. Host values are checked
    against [0, T]; a device tensor's are clamped by the kernels."""
    if lengths is None:
        return None
    if isinstance(lengths, torch.Tensor) and lengths.device.type == "cuda":
        if tuple(lengths.shape) != (B,):
            raise ValueError(f"lengths: shape {tuple(lengths.shape)} != ({B},)")
        if lengths.device != device:
            raise ValueError(f"lengths: device {lengths.device} != {device}")
        if lengths.dtype != torch.int32:
            lengths = lengths.clamp(0, T).to(torch.int32)
        return lengths.contiguous()
    vals = [int(v) for v in lengths]
    if len(vals) != B:
        raise ValueError(f"lengths: {len(vals)} values for a batch of {B} rows")
    if any(v < 0 or v > T for v in vals):
        raise ValueError(f"lengths: values must lie in [0, {T}]")
    return torch.tensor(vals, dtype=torch.int32, device=device)


class BlockContext:
    """What a backward call needs from its forward: the tensors and the
    reserve, kept alive here."""

    def __init__(self, device, stream, **kw):
        self.device, self.stream = device, stream
        self.__dict__.update(kw)

    def _use(self, *tensors):
        # memory that the caller cannot see must outlive work on another
        # stream than the one it was allocated on
        if _raw_stream(self.device.index) != self.stream:
            for t in tensors:
                if t is not None:
                    t.record_stream(torch.cuda.current_stream(self.device))


# ---------------------------------------------------------------------------
# Layer norm
# ---------------------------------------------------------------------------

def _rows(t):
    """(t, elements between rows) of t seen as rows of its last dimension,
    with a copy only where its leading dimensions do not step evenly."""
    n = t.shape[-1]
    if t.dim() == 1:
        return (t if t.stride(0) == 1 or n == 1 else _dense(t)), n
    if n == 1 or t.stride(-1) == 1:
        ld, span = None, None
        for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
            if size == 1:
                continue
            if ld is None:
                ld, span = stride, stride * size
            elif stride == span:
                span *= size
            else:
                break
        else:
            ld = n if ld is None else ld
            if ld >= n:
                return t, ld
    return _dense(t), n


def _layer_norm(x, weight, bias, residual, eps, train):
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError("x must be a tensor of at least one dimension")
    _tensor(x, "x", x.dim())
    n, device = x.shape[-1], x.device
    rows = x.numel() // n if n else 0
    weight = _plain(weight, "weight", (n,), x.dtype, device)
    bias = _plain(bias, "bias", (n,), x.dtype, device)
    xr, ld = _rows(x)
    ldr, total = 0, None
    if residual is not None:
        residual, ldr = _rows(_strided(residual, "residual", x.shape, x))
        total = _dense_like(x)
    y = _dense_like(x)
    stats = torch.empty((rows, 2), dtype=torch.float32, device=device) if train else None
    desc = RnnNormDesc(DTYPES[x.dtype], n, rows, ld, ldr, eps, 0)
    stream = _call("rnn_layer_norm", device, ctypes.byref(desc), xr.data_ptr(), _ptr(residual), _ptr(weight), _ptr(bias),
                   y.data_ptr(), _ptr(total), _ptr(stats))
    if not train:
        return y if total is None else (y, total)
    if total is not None:
        xr, desc = total, RnnNormDesc(desc.dtype, n, rows, n, 0, eps, 0)
    return (y, total), BlockContext(device, stream, desc=desc, x=xr, weight=weight, stats=stats, shape=x.shape,
                                    has_params=weight is not None or bias is not None)


def layer_norm(x, weight=None, bias=None, *, residual=None, eps=1e-5):
    """Layer norm over the last dimension of x [..., N] (float32 or bfloat16).

    weight, bias: [N] in x's dtype, None = ones, zeros. residual: a tensor of
    x's shape that is added first; the sum, rounded to x's dtype, is what is
    normalised. Returns y, or (y, sum) with a residual. x and the residual
    may be strided; N is at most 16384."""
    return _layer_norm(x, weight, bias, residual, eps, False)


def layer_norm_train(x, weight=None, bias=None, *, residual=None, eps=1e-5):
    """layer_norm that also keeps each row's fp32 statistics. Returns
    ((y, sum), ctx), sum None without a residual; pass ctx to
    layer_norm_backward. ctx holds x (or the sum) and the weight: do not
    change them in place before the backward pass."""
    return _layer_norm(x, weight, bias, residual, eps, True)


def layer_norm_backward(ctx, dy, dsum=None):
    """Gradients of layer_norm_train. dy: gradient of y; dsum: gradient that
    reaches the sum (or x) by another way, added to dx. Returns (dx, dweight,
    dbias): dx in x's dtype is the gradient of x and of the residual alike;
    dweight and dbias are fp32 (None when the forward had neither)."""
    x, device = ctx.x, ctx.device
    dy = _plain(dy, "dy", ctx.shape, x.dtype, device)
    dsum = _plain(dsum, "dsum", ctx.shape, x.dtype, device)
    n = ctx.shape[-1]
    dx = _dense_like(dy)
    dw = db = ws = None
    size = 0
    if ctx.has_params:
        dw, db = torch.empty((2, n), dtype=torch.float32, device=device).unbind(0)
        size = _bytes("rnn_layer_norm_backward_workspace_bytes", ctx.desc)
        ws = _buffer(size, device)
    ctx._use(x, ctx.weight, ctx.stats)
    _call("rnn_layer_norm_backward", device, ctypes.byref(ctx.desc), x.data_ptr(), _ptr(ctx.weight), ctx.stats.data_ptr(),
          dy.data_ptr(), _ptr(dsum), dx.data_ptr(), _ptr(dw), _ptr(db), _ptr(ws), size)
    return dx, dw, db


# ---------------------------------------------------------------------------
# Gated linear scan
# ---------------------------------------------------------------------------

def _gated_scan(x, f, i, h0, lengths, reverse, train):
    _tensor(x, "x", 3)
    T, B, H = x.shape
    device, dtype = x.device, x.dtype
    shape = x.shape
    x = _strided(x, "x", shape, x)
    f = _strided(f, "f", shape, x)
    i = None if i is None else _strided(i, "i", shape, x)
    h0 = _plain(h0, "h0", (B, H), torch.float32, device)
    lengths = _lengths(lengths, B, T, device)
    y = _dense_like(x)
    h_n = torch.empty((B, H), dtype=torch.float32, device=device) if h0 is None else torch.empty_like(h0)
    (xt, xb, _), (ft, fb, _) = x.stride(), f.stride()
    it, ib, _ = (0, 0, 0) if i is None else i.stride()
    desc = RnnGatedScanDesc(DTYPES[dtype], T, B, H, 1 if reverse else 0, 0 if i is None else 1, xt, xb, ft, fb, it, ib)
    io = RnnGatedScanIO(x.data_ptr(), f.data_ptr(), _ptr(i), _ptr(lengths), _ptr(h0), y.data_ptr(), h_n.data_ptr())
    size = _bytes("rnn_gated_scan_workspace_bytes", desc)
    ws = _buffer(size, device)
    if not train:
        _call("rnn_gated_scan", device, ctypes.byref(desc), ctypes.byref(io), _ptr(ws), size)
        return y, h_n
    rsize = _bytes("rnn_gated_scan_reserve_bytes", desc)
    reserve = _buffer(rsize, device)
    stream = _call("rnn_gated_scan_train", device, ctypes.byref(desc), ctypes.byref(io), _ptr(reserve), rsize, _ptr(ws), size)
    return (y, h_n), BlockContext(device, stream, desc=desc, x=x, f=f, i=i, lengths=lengths, reserve=reserve)


def gated_scan(x, f, i=None, *, h0=None, lengths=None, reverse=False):
    """Gated linear recurrence over time, per channel:

        h_t = sigmoid(f_t) h_{t-1} + (1 - sigmoid(f_t)) x_t    (i None)
        h_t = sigmoid(f_t) h_{t-1} + sigmoid(i_t) x_t

    x, f, i: [T, B, H] (float32 or bfloat16; may be slices of one projection:
    only the last dimension has to be contiguous). h0: fp32 [B, H]. lengths:
    B row lengths in [0, T], a device int32 tensor or host values (which are
    copied). reverse runs each row from its last step to its first.
    Returns (y [T, B, H] with zeros past a row's length, h_n fp32 [B, H]). A
    serving step is T = 1 with the last call's h_n as h0."""
    return _gated_scan(x, f, i, h0, lengths, reverse, False)


def gated_scan_train(x, f, i=None, *, h0=None, lengths=None, reverse=False):
    """gated_scan that also keeps the fp32 state at every 128th step. Returns
    ((y, h_n), ctx); pass ctx to gated_scan_backward. ctx holds x, f, i and a
    device tensor of lengths: do not change them in place before the backward
    pass (a lengths buffer that is used again neither)."""
    return _gated_scan(x, f, i, h0, lengths, reverse, True)


def gated_scan_backward(ctx, dy, dh_n=None):
    """Gradients of gated_scan_train, given dy (shape and dtype of y) and
    optionally dh_n (fp32 [B, H]). Returns (dx, df, di, dh0): di None without
    an input gate, dh0 fp32."""
    d, device, dtype = ctx.desc, ctx.device, ctx.x.dtype
    shape = (d.T, d.B, d.H)
    dy = _plain(dy, "dy", shape, dtype, device)
    dh_n = _plain(dh_n, "dh_n", (d.B, d.H), torch.float32, device)
    dx, df = _dense_like(dy), _dense_like(dy)
    di = _dense_like(dy) if ctx.i is not None else None
    dh0 = torch.empty((d.B, d.H), dtype=torch.float32, device=device)
    io = RnnGatedScanIO(ctx.x.data_ptr(), ctx.f.data_ptr(), _ptr(ctx.i), _ptr(ctx.lengths), None, None, None)
    grads = RnnGatedScanGrads(dy.data_ptr(), _ptr(dh_n), dx.data_ptr(), df.data_ptr(), _ptr(di), dh0.data_ptr())
    size = _bytes("rnn_gated_scan_workspace_bytes", d)
    ws = _buffer(size, device)
    ctx._use(ctx.x, ctx.f, ctx.i, ctx.lengths, ctx.reserve)
    _call("rnn_gated_scan_backward", device, ctypes.byref(d), ctypes.byref(io), ctypes.byref(grads), _ptr(ctx.reserve),
          ctx.reserve.numel(), _ptr(ws), size)
    return dx, df, di, dh0


# ---------------------------------------------------------------------------
# Cross attention
# ---------------------------------------------------------------------------

def _cross_attention(q, k, v, lengths, scale, train):
    _tensor(q, "q", 4)
    _tensor(k, "k", 4)
    Tq, B, heads, D = q.shape
    Tk, _, kv_heads, _ = k.shape
    device, dtype = q.device, q.dtype
    q = _strided(q, "q", q.shape, q)
    shape = (Tk, B, kv_heads, D)
    k = _strided(k, "k", shape, q)
    v = _strided(v, "v", shape, q)
    lengths = _lengths(lengths, B, Tk, device)
    o = _dense_like(q)
    if scale is None:
        scale = D ** -0.5 if D else 1.0
    desc = RnnAttentionDesc(DTYPES[dtype], B, Tq, Tk, heads, kv_heads, D, scale, *q.stride()[:3], *k.stride()[:3],
                            *v.stride()[:3])
    io = RnnAttentionIO(q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(lengths), o.data_ptr())
    size = _bytes("rnn_cross_attention_workspace_bytes", desc)
    ws = _buffer(size, device)
    if not train:
        _call("rnn_cross_attention", device, ctypes.byref(desc), ctypes.byref(io), _ptr(ws), size)
        return o
    rsize = _bytes("rnn_cross_attention_reserve_bytes", desc)
    reserve = _buffer(rsize, device)
    stream = _call("rnn_cross_attention_train", device, ctypes.byref(desc), ctypes.byref(io), _ptr(reserve), rsize, _ptr(ws),
                   size)
    return o, BlockContext(device, stream, desc=desc, io=io, q=q, k=k, v=v, lengths=lengths, o=o, reserve=reserve)


def cross_attention(q, k, v, *, lengths=None, scale=None):
    """Attention of queries q [Tq, B, heads, D] over an encoder's states k, v
    [Tk, B, kv_heads, D] (float32 or bfloat16): softmax(scale q k^T) v over
    the first lengths[b] states of each batch row, zero where there are none.

    heads is a multiple of kv_heads, whose query heads share a key head; D is
    at most 128. Every tensor may be a strided view (time-major, batch-major,
    slices of one projection) whose last dimension is contiguous. lengths: B
    values in [0, Tk], a device int32 tensor or host values (which are
    copied); states past them are not read. scale: default D ** -0.5.
    Returns o [Tq, B, heads, D]. A serving step is Tq = 1."""
    return _cross_attention(q, k, v, lengths, scale, False)


def cross_attention_train(q, k, v, *, lengths=None, scale=None):
    """cross_attention that also keeps the fp32 log-sum-exp of every query's
    scores. Returns (o, ctx); pass ctx to cross_attention_backward. ctx holds
    q, k, v, o and a device tensor of lengths: do not change them in place
    before the backward pass (a lengths buffer that is used again neither)."""
    return _cross_attention(q, k, v, lengths, scale, True)


def cross_attention_backward(ctx, do):
    """Gradients of cross_attention_train, given do (shape and dtype of o).
    Returns dense (dq, dk, dv); dk and dv are summed over the query heads of
    a key head and zero past a row's length. In bf16, o and dq are as exact as
    their own rounding; dk and dv too for small calls, and sqrt(2) times as far
    off where ceil(Tk / (64 if D <= 64 else 128)) * B * kv_heads passes 256
    (probabilities and score gradients are rounded once there)."""
    o, device = ctx.o, ctx.device
    do = _plain(do, "do", o.shape, o.dtype, device)
    dq = torch.empty_like(o)
    dk, dv = o.new_empty(ctx.k.shape), o.new_empty(ctx.k.shape)
    grads = RnnAttentionGrads(do.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr())
    size = _bytes("rnn_cross_attention_backward_workspace_bytes", ctx.desc)
    ws = _buffer(size, device)
    ctx._use(ctx.q, ctx.k, ctx.v, ctx.lengths, o, ctx.reserve)
    _call("rnn_cross_attention_backward", device, ctypes.byref(ctx.desc), ctypes.byref(ctx.io), ctypes.byref(grads),
          ctx.reserve.data_ptr(), ctx.reserve.numel(), _ptr(ws), size)
    return dq, dk, dv
