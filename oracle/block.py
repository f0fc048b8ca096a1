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
