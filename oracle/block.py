"""Float64 definitions of the decoder block's operators: layer norm with a
residual add, the gated linear recurrence, and cross attention to an
encoder's states, each with its gradient written out from its formula.

Plain and slow: one step, row or head at a time.
"""

import numpy as np

from .rnn import sigmoid


def layer_norm(s, weight=None, bias=None, eps=1e-5):
    """(y, mean, rstd) of the rows of s [rows, N]."""
    s = np.asarray(s, dtype=np.float64)
    mu = s.mean(-1, keepdims=True)
    rstd = 1.0 / np.sqrt(((s - mu) ** 2).mean(-1, keepdims=True) + eps)
    y = (s - mu) * rstd
    if weight is not None:
        y = y * weight
    if bias is not None:
        y = y + bias
    return y, mu[..., 0], rstd[..., 0]


def layer_norm_backward(s, weight, dy, dsum=None, eps=1e-5):
    """(dx, dweight, dbias) for dy [rows, N]."""
    s, dy = np.asarray(s, dtype=np.float64), np.asarray(dy, dtype=np.float64)
    n, _, rstd = layer_norm(s, eps=eps)
    g = dy if weight is None else dy * weight
    dx = rstd[..., None] * (g - g.mean(-1, keepdims=True) - n * (g * n).mean(-1, keepdims=True))
    if dsum is not None:
        dx = dx + dsum
    return dx, (dy * n).sum(0), dy.sum(0)


def _steps(T, B, lengths, reverse):
    """For each row, the times of its steps in the order they run."""
    lengths = [T] * B if lengths is None else [int(v) for v in lengths]
    return [list(range(L - 1, -1, -1)) if reverse else list(range(L)) for L in lengths]


def gated_scan(x, f, i=None, h0=None, lengths=None, reverse=False):
    """(y [T, B, H], h_n [B, H], states entering each step [T, B, H])."""
    x, f = np.asarray(x, dtype=np.float64), np.asarray(f, dtype=np.float64)
    T, B, H = x.shape
    y, before = np.zeros_like(x), np.zeros_like(x)
    hn = np.zeros((B, H))
    for b, times in enumerate(_steps(T, B, lengths, reverse)):
        h = np.zeros(H) if h0 is None else np.asarray(h0[b], dtype=np.float64)
        for t in times:
            before[t, b] = h
            u = sigmoid(-f[t, b]) if i is None else sigmoid(np.asarray(i[t, b], dtype=np.float64))
            h = sigmoid(f[t, b]) * h + u * x[t, b]
            y[t, b] = h
        hn[b] = h
    return y, hn, before


def gated_scan_backward(x, f, i, dy, dh_n=None, h0=None, lengths=None, reverse=False):
    """(dx, df, di or None, dh0)."""
    x, f, dy = (np.asarray(v, dtype=np.float64) for v in (x, f, dy))
    T, B, H = x.shape
    before = gated_scan(x, f, i, h0, lengths, reverse)[2]
    dx, df = np.zeros_like(x), np.zeros_like(x)
    di = None if i is None else np.zeros_like(x)
    dh0 = np.zeros((B, H))
    for b, times in enumerate(_steps(T, B, lengths, reverse)):
        c = np.zeros(H) if dh_n is None else np.asarray(dh_n[b], dtype=np.float64)
        for t in reversed(times):
            a, keep = sigmoid(f[t, b]), sigmoid(-f[t, b])
            g = dy[t, b] + c
            if i is None:
                dx[t, b] = g * keep
                df[t, b] = g * (before[t, b] - x[t, b]) * a * keep
            else:
                s, no = sigmoid(np.asarray(i[t, b], dtype=np.float64)), sigmoid(-np.asarray(i[t, b], dtype=np.float64))
                dx[t, b] = g * s
                df[t, b] = g * before[t, b] * a * keep
                di[t, b] = g * x[t, b] * s * no
            c = a * g
        dh0[b] = c
    return dx, df, di, dh0


def _pairs(q, k, lengths):
    """(batch row, query head, key head, keys) of every attention problem."""
    group = q.shape[2] // k.shape[2]
    for b in range(q.shape[1]):
        n = k.shape[0] if lengths is None else int(lengths[b])
        for h in range(q.shape[2]):
            yield b, h, h // group, n


def _softmax(s):
    e = np.exp(s - s.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


def cross_attention(q, k, v, lengths=None, scale=None):
    """o [Tq, B, heads, D] for q [Tq, B, heads, D] and k, v [Tk, B, kv, D]."""
    q, k, v = (np.asarray(t, dtype=np.float64) for t in (q, k, v))
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    o = np.zeros_like(q)
    for b, h, hk, n in _pairs(q, k, lengths):
        if n:
            o[:, b, h] = _softmax(scale * q[:, b, h] @ k[:n, b, hk].T) @ v[:n, b, hk]
    return o


def cross_attention_backward(q, k, v, do, lengths=None, scale=None):
    """(dq, dk, dv)."""
    q, k, v, do = (np.asarray(t, dtype=np.float64) for t in (q, k, v, do))
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for b, h, hk, n in _pairs(q, k, lengths):
        if not n:
            continue
        p = _softmax(scale * q[:, b, h] @ k[:n, b, hk].T)
        dp = do[:, b, h] @ v[:n, b, hk].T
        ds = p * (dp - (p * dp).sum(-1, keepdims=True)) * scale
        dq[:, b, h] = ds @ k[:n, b, hk]
        dk[:n, b, hk] += ds.T @ q[:, b, h]
        dv[:n, b, hk] += p.T @ do[:, b, h]
    return dq, dk, dv


def attention_bounds(q, k, v, do, lengths=None, scale=None, unit=0.0):
    """First-order bounds of (o, dq, dk, dv) against one rounding of relative
    size `unit` of each probability p and score gradient ds inside the sums,
    and of o inside delta = sum_d do o:
      |d o| <= u p |v|,  |d dv| <= u p^T |do|,
      |d ds| <= u |ds| + p |d delta|,  |d delta| <= 2 u sum_d |do| p |v|
    (o carries its own rounding and p's), carried through ds k and ds^T q."""
    q, k, v, do = (np.asarray(t, dtype=np.float64) for t in (q, k, v, do))
    scale = q.shape[-1] ** -0.5 if scale is None else scale
    bo, bq, bk, bv = np.zeros_like(q), np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for b, h, hk, n in _pairs(q, k, lengths):
        if not n:
            continue
        p = _softmax(scale * q[:, b, h] @ k[:n, b, hk].T)
        dp = do[:, b, h] @ v[:n, b, hk].T
        ds = np.abs(p * (dp - (p * dp).sum(-1, keepdims=True)))
        bo[:, b, h] = p @ np.abs(v[:n, b, hk])
        delta = 2.0 * (np.abs(do[:, b, h]) * bo[:, b, h]).sum(-1, keepdims=True)
        ds = (ds + p * delta) * abs(scale)
        bq[:, b, h] = ds @ np.abs(k[:n, b, hk])
        bk[:n, b, hk] += ds.T @ np.abs(q[:, b, h])
        bv[:n, b, hk] += p.T @ np.abs(do[:, b, h])
    return unit * bo, unit * bq, unit * bk, unit * bv
