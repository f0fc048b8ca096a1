"""Float64 definitions of the state-space block's operators: the short causal
convolution, the selective scan and the gated feed-forward, each with its
gradient written out from its formula.

Plain and slow: one row and one step at a time.
"""

import numpy as np

from .rnn import sigmoid, softplus


def _f64(v):
    return None if v is None else np.asarray(v, dtype=np.float64)


def _row_lengths(T, B, lengths):
    return [T] * B if lengths is None else [int(v) for v in lengths]


def silu(v):
    return v * sigmoid(v)


def silu_slope(v):
    return sigmoid(v) + v * sigmoid(v) * sigmoid(-v)


# -- causal convolution --

def _history(x, state, b, L, W):
    """The inputs that row b's filter sees: W - 1 of the state, then its own."""
    front = np.zeros((W - 1, x.shape[2])) if state is None else state[:, b]
    return np.concatenate([front, x[:L, b]])


def causal_conv(x, weight, bias=None, state=None, lengths=None, activation=None):
    """(y [T, B, C], state_n [W - 1, B, C])."""
    x, weight, bias, state = _f64(x), _f64(weight), _f64(bias), _f64(state)
    T, B, C = x.shape
    W = weight.shape[1]
    y, last = np.zeros_like(x), np.zeros((W - 1, B, C))
    for b, L in enumerate(_row_lengths(T, B, lengths)):
        seq = _history(x, state, b, L, W)
        for t in range(L):
            p = (weight.T * seq[t:t + W]).sum(0) + (0.0 if bias is None else bias)
            y[t, b] = silu(p) if activation == "silu" else p
        last[:, b] = seq[L:]
    return y, last


def causal_conv_backward(x, weight, bias, dy, dstate_n=None, state=None, lengths=None, activation=None):
    """(dx, dweight, dbias, dstate)."""
    x, weight, bias, dy, dstate_n, state = (_f64(v) for v in (x, weight, bias, dy, dstate_n, state))
    T, B, C = x.shape
    W = weight.shape[1]
    dx, dw, db, dstate = np.zeros_like(x), np.zeros_like(weight), np.zeros(C), np.zeros((W - 1, B, C))
    for b, L in enumerate(_row_lengths(T, B, lengths)):
        seq = _history(x, state, b, L, W)
        dseq = np.zeros_like(seq)
        for t in range(L):
            g = dy[t, b]
            if activation == "silu":
                g = g * silu_slope((weight.T * seq[t:t + W]).sum(0) + (0.0 if bias is None else bias))
            dseq[t:t + W] += weight.T * g
            dw += (seq[t:t + W] * g).T
            db += g
        if dstate_n is not None:
            dseq[L:] += dstate_n[:, b]
        dstate[:, b], dx[:L, b] = dseq[:W - 1], dseq[W - 1:]
    return dx, dw, db, dstate


# -- selective scan --

def _steps_of(dt, dt_bias, soft):
    raw = dt if dt_bias is None else dt + dt_bias
    return raw, softplus(raw) if soft else raw


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, soft=True, h0=None, lengths=None):
    """(y [T, B, H], h_n [B, H, N], states entering each step [T, B, H, N])
    for x, dt, z [T, B, H], A [H, N], B and C [T, B, G, N], D and dt_bias [H]."""
    x, dt, A, Bm, Cm, D, z, dt_bias, h0 = (_f64(v) for v in (x, dt, A, B, C, D, z, dt_bias, h0))
    T, rows, H = x.shape
    N, heads = A.shape[1], np.arange(H) // (H // Bm.shape[2])
    y, before, hn = np.zeros_like(x), np.zeros((T, rows, H, N)), np.zeros((rows, H, N))
    for b, L in enumerate(_row_lengths(T, rows, lengths)):
        h = np.zeros((H, N)) if h0 is None else h0[b]
        for t in range(L):
            before[t, b] = h
            delta = _steps_of(dt[t, b], dt_bias, soft)[1]
            h = np.exp(delta[:, None] * A) * h + (delta * x[t, b])[:, None] * Bm[t, b, heads]
            v = (h * Cm[t, b, heads]).sum(-1) + (0.0 if D is None else D * x[t, b])
            y[t, b] = v if z is None else v * silu(z[t, b])
        hn[b] = h
    return y, hn, before


def selective_scan_backward(x, dt, A, B, C, D, dy, dh_n=None, z=None, dt_bias=None, soft=True, h0=None, lengths=None):
    """Gradients by name: x, dt, A, B, C, D, z, dt_bias, h0."""
    before = selective_scan(x, dt, A, B, C, D, z, dt_bias, soft, h0, lengths)[2]
    x, dt, A, Bm, Cm, D, z, dt_bias, dy, dh_n = (_f64(v) for v in (x, dt, A, B, C, D, z, dt_bias, dy, dh_n))
    T, rows, H = x.shape
    N, heads = A.shape[1], np.arange(H) // (H // Bm.shape[2])
    out = {"x": np.zeros_like(x), "dt": np.zeros_like(x), "A": np.zeros_like(A), "B": np.zeros_like(Bm), "C": np.zeros_like(Cm),
           "D": np.zeros(H), "z": np.zeros_like(x), "dt_bias": np.zeros(H), "h0": np.zeros((rows, H, N))}
    for b, L in enumerate(_row_lengths(T, rows, lengths)):
        carry = np.zeros((H, N)) if dh_n is None else dh_n[b]
        for t in range(L - 1, -1, -1):
            raw, delta = _steps_of(dt[t, b], dt_bias, soft)
            a, bt, ct, xt = np.exp(delta[:, None] * A), Bm[t, b, heads], Cm[t, b, heads], x[t, b]
            now = a * before[t, b] + (delta * xt)[:, None] * bt
            do = dy[t, b]
            if z is not None:
                v = (now * ct).sum(-1) + (0.0 if D is None else D * xt)
                out["z"][t, b] = do * v * silu_slope(z[t, b])
                do = do * silu(z[t, b])
            np.add.at(out["C"][t, b], heads, do[:, None] * now)
            g = carry + do[:, None] * ct
            np.add.at(out["B"][t, b], heads, g * (delta * xt)[:, None])
            w = g * a * before[t, b]
            through = (g * bt).sum(-1)
            out["A"] += w * delta[:, None]
            out["x"][t, b] = delta * through + (0.0 if D is None else D * do)
            slope = sigmoid(raw) if soft else 1.0
            out["dt"][t, b] = ((w * A).sum(-1) + xt * through) * slope
            out["dt_bias"] += out["dt"][t, b]
            out["D"] += do * xt
            carry = a * g
        out["h0"][b] = carry
    return out


# -- gated feed-forward --

_GELU = np.sqrt(2.0 / np.pi)


def activation(g, kind):
    """(act(g), act'(g))."""
    if kind == "silu":
        return silu(g), silu_slope(g)
    if kind == "sigmoid":
        return sigmoid(g), sigmoid(g) * sigmoid(-g)
    if kind != "gelu_tanh":
        raise ValueError(kind)
    t = np.tanh(_GELU * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * _GELU * (1 + 3 * 0.044715 * g * g)


def feed_forward(x, w_in, w_out, residual=None, kind="silu"):
    """y [rows, n_out] of x [rows, n], w_in [2 F, n] (the gate's rows first),
    w_out [n_out, F]."""
    x, w_in, w_out, residual = (_f64(v) for v in (x, w_in, w_out, residual))
    F = w_out.shape[1]
    y = (activation(x @ w_in[:F].T, kind)[0] * (x @ w_in[F:].T)) @ w_out.T
    return y if residual is None else y + residual


def feed_forward_backward(x, w_in, w_out, dy, kind="silu"):
    """(dx, dw_in, dw_out)."""
    x, w_in, w_out, dy = (_f64(v) for v in (x, w_in, w_out, dy))
    F = w_out.shape[1]
    u = x @ w_in[F:].T
    act, slope = activation(x @ w_in[:F].T, kind)
    dh = dy @ w_out
    dp = np.concatenate([dh * u * slope, dh * act], 1)
    return dp @ w_in, dp.T @ x, dy.T @ (act * u)
