"""What the operators of a state-space block are measured on: the short causal
convolution, the selective scan and the gated feed-forward, each beside its
plain form.

A block uses them in turn: projection, causal convolution over time, selective
scan with its output gate, projection, residual add, and the feed-forward.
Tensors are time-major, [T, B, ...], as the library's padded layout has them.
"""

import math
import random

import torch

own = False

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ESIZE = {"f32": 4, "bf16": 2}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _conv(T, B, C, W, dtype, silu, lo, train):
    # lo: the shortest row of a ragged batch; -1: every row has T steps
    return {"op": "conv", "T": T, "B": B, "C": C, "W": W, "dtype": dtype, "silu": silu, "lo": lo, "train": train}


def _scan(T, B, H, N, groups, dtype, gate, lo, train):
    return {"op": "scan", "T": T, "B": B, "H": H, "N": N, "groups": groups, "dtype": dtype, "gate": gate, "lo": lo,
            "train": train}


def _feed(rows, n, F, dtype, activation, residual, train):
    return {"op": "feed", "rows": rows, "n": n, "F": F, "dtype": dtype, "activation": activation, "residual": residual,
            "train": train}


def listed():
    named = [
        # one decoding step for 64 requests, each with the last inputs of its own
        ("conv_step_b64", _conv(1, 64, 2048, 4, "bf16", True, -1, False)),
        # training on 64 ragged sequences, a width that is not a whole number of cache lines
        ("conv_train_varlen_b64", _conv(500, 64, 1000, 3, "f32", False, 50, True)),
        # training on 32 sequences of 1000 steps
        ("conv_train_t1000_b32", _conv(1000, 32, 2048, 4, "bf16", True, -1, True)),
        # one decoding step of the state for 64 requests: the state is what moves
        ("scan_step_b64", _scan(1, 64, 2048, 16, 1, "bf16", True, -1, False)),
        # reading 32 prompts of 1000 steps
        ("scan_prompt_t1000_b32", _scan(1000, 32, 1024, 16, 1, "bf16", True, -1, False)),
        # training on 64 ragged sequences, two groups of channels, without an output gate
        ("scan_train_varlen_b64", _scan(500, 64, 512, 16, 2, "f32", False, 50, True)),
        # training on two long sequences: few channels, so time itself has to be split
        ("scan_train_t16384_b2", _scan(16384, 2, 1000, 16, 1, "bf16", True, -1, True)),
        # one decoding step of a single request: the weights are what moves
        ("feed_step_b1", _feed(1, 1024, 2816, "bf16", "silu", True, False)),
        # one decoding step for 64 requests
        ("feed_step_b64", _feed(64, 1024, 4096, "bf16", "silu", True, False)),
        # reading one prompt of 333 steps
        ("feed_prompt", _feed(333, 1024, 2816, "bf16", "gelu_tanh", True, False)),
        # training in fp32 on a packed variable-length batch: as many rows as it has tokens
        ("feed_train_packed", _feed(19334, 512, 1368, "f32", "silu", False, True)),
        # training on 32 sequences of 1000 steps
        ("feed_train_t1000_b32", _feed(32000, 1024, 2816, "bf16", "silu", True, True)),
    ]
    out = []
    for name, case in named:
        case["name"] = name
        out.append(case)
    return out


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi, share=0.7):
    """A size over [lo, hi], a multiple of 8 in `share` of the draws."""
    n = _log_int(rng, lo, hi)
    return max(8, n // 8 * 8) if rng.random() < share else n


def draw(rng):
    """One more case: sizes log-uniform over what the listed ones span, odd
    sizes among them, bounded by the largest listed case of their operator."""
    op = rng.choice(["conv", "scan", "feed"])
    dtype = rng.choice(["f32", "bf16"])
    train = rng.random() < 0.5
    if op == "conv":
        T, B, C = _log_int(rng, 1, 16384), _log_int(rng, 1, 64), _width(rng, 16, 4096)
        while T * B * C > 60_000_000:
            T, B = max(1, T // 2), max(1, B - B // 4)
        return _conv(T, B, C, rng.choice([2, 3, 4]), dtype, rng.random() < 0.5, rng.choice([-1, 0, T // 4]), train)
    if op == "scan":
        groups = rng.choice([1, 1, 2, 4])
        T, B, H = _log_int(rng, 1, 16384), _log_int(rng, 1, 64), groups * _width(rng, 16, 2048 // groups)
        N = rng.choice([4, 8, 12, 16, 16, 16, 32, 64])
        while T * B * H * N > 520_000_000:
            T, B = max(1, T // 2), max(1, B - B // 4)
        return _scan(T, B, H, N, groups, dtype, rng.random() < 0.5, rng.choice([-1, 0, T // 4]), train)
    n, F = _width(rng, 64, 2048), _width(rng, 64, 8192)
    rows = _log_int(rng, 1, 32000)
    limit = 0.9 * 32000 * 1024 * 2816 * (0.15 if dtype == "f32" else 1.0)
    while rows * n * F > limit:
        rows = max(1, rows - rows // 4)
    return _feed(rows, n, F, dtype, rng.choice(["silu", "silu", "gelu_tanh", "sigmoid"]), rng.random() < 0.5, train)


def _lengths(lo, T, B):
    """The row lengths of a ragged batch: evenly spread over [lo, T] (what is
    drawn by the seed is their order), or None."""
    if lo < 0:
        return None
    if B == 1:
        return [T]
    return [lo + (T - lo) * j // (B - 1) for j in range(B)]


def work(case):
    e = ESIZE[case["dtype"]]
    if case["op"] == "feed":
        rows, n, F = case["rows"], case["n"], case["F"]
        weights, io = 3 * n * F, (3 if case["residual"] else 2) * rows * n
        if not case["train"]:
            return {"bytes": (weights + io) * e, "flops": 6 * rows * n * F}
        return {"bytes": (2 * weights + io + 2 * rows * n) * e, "flops": 18 * rows * n * F}
    T, B = case["T"], case["B"]
    lens = _lengths(case["lo"], T, B)
    tok = T * B if lens is None else sum(lens)
    if case["op"] == "conv":
        C, W = case["C"], case["W"]
        small = 2 * (W - 1) * B * C * e + C * (W + 1) * e
        if not case["train"]:
            return {"bytes": (tok + T * B) * C * e + small, "flops": 2 * W * tok * C}
        return {"bytes": (2 * tok + 2 * T * B) * C * e + 2 * small + C * (W + 1) * 4, "flops": 6 * W * tok * C}
    H, N, G = case["H"], case["N"], case["groups"]
    ins = 3 if case["gate"] else 2
    state = 8 * B * H * N
    params = 4 * H * (N + 2)
    if not case["train"]:
        return {"bytes": (ins * tok + T * B) * H * e + 2 * tok * G * N * e + state + params, "flops": 7 * tok * H * N}
    moved = ((ins + 1) * tok + (ins + 1) * T * B) * H * e + (2 * tok + 2 * T * B) * G * N * e
    return {"bytes": moved + 2 * state + 2 * params, "flops": 26 * tok * H * N}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, dtype, mean=0.0, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std + mean).to(dtype)


def _length_tensor(case, T, seed):
    lens = _lengths(case["lo"], T, case["B"])
    if lens is None:
        return None
    random.Random(seed).shuffle(lens)
    return torch.tensor(lens, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g, dt = _generator(seed), TYPES[case["dtype"]]
    st = dict(case)
    if case["op"] == "conv":
        T, B, C, W = case["T"], case["B"], case["C"], case["W"]
        # the branch that the convolution reads and the one that gates later, as one projection writes them
        st["xz"] = _normal(g, (T, B, 2, C), dt)
        st["w"] = _normal(g, (C, W), dt, 0.0, W ** -0.5)
        st["b"] = _normal(g, (C,), dt, 0.0, 0.2)
        st["state"] = _normal(g, (W - 1, B, C), dt)
        st["lengths"] = _length_tensor(case, T, seed)
        if case["train"]:
            st["dy"] = _normal(g, (T, B, C), dt)
            st["dstate"] = _normal(g, (W - 1, B, C), dt)
    elif case["op"] == "scan":
        T, B, H, N, G = (case[k] for k in ("T", "B", "H", "N", "groups"))
        st["x"] = _normal(g, (T, B, H), dt)
        st["dt"] = _normal(g, (T, B, H), dt, 0.0, 0.7)
        st["bc"] = _normal(g, (T, B, 2, G, N), dt)
        st["z"] = _normal(g, (T, B, H), dt) if case["gate"] else None
        # decays of 1 to N a unit of time, steps of 0.001 to 0.1, as such layers are set up
        spread = torch.rand((H,), generator=g, device=DEV)
        step = torch.exp(spread * (math.log(0.1) - math.log(0.001)) + math.log(0.001))
        st["dt_bias"] = step + torch.log(-torch.expm1(-step))
        st["A"] = -(torch.arange(1, N + 1, device=DEV, dtype=torch.float32)
                    * torch.exp(0.1 * torch.randn((H, N), generator=g, device=DEV)))
        st["D"] = _normal(g, (H,), torch.float32, 1.0, 0.2)
        st["h0"] = _normal(g, (B, H, N), torch.float32, 0.0, 0.5)
        st["lengths"] = _length_tensor(case, T, seed)
        if case["train"]:
            st["dy"] = _normal(g, (T, B, H), dt)
            st["dhn"] = _normal(g, (B, H, N), torch.float32, 0.0, 0.5)
    else:
        rows, n, F = case["rows"], case["n"], case["F"]
        st["x"] = _normal(g, (rows, n), dt)
        st["w_in"] = _normal(g, (2 * F, n), dt, 0.0, n ** -0.5)
        st["w_out"] = _normal(g, (n, F), dt, 0.0, F ** -0.5)
        st["r"] = _normal(g, (rows, n), dt, 0.0, 2.0) if case["residual"] else None
        if case["train"]:
            st["dy"] = _normal(g, (rows, n), dt)
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)[state["op"]](state)


# -- the library's operators --

def _own_conv(s):
    import gru_sequence_scan_amd as gss
    x, act = s["xz"][:, :, 0], "silu" if s["silu"] else None
    if not s["train"]:
        return gss.causal_conv(x, s["w"], s["b"], state=s["state"], lengths=s["lengths"], activation=act)
    (y, last), ctx = gss.causal_conv_train(x, s["w"], s["b"], state=s["state"], lengths=s["lengths"], activation=act)
    return (y, last) + gss.causal_conv_backward(ctx, s["dy"], s["dstate"])


def _own_scan(s):
    import gru_sequence_scan_amd as gss
    args = (s["x"], s["dt"], s["A"], s["bc"][:, :, 0], s["bc"][:, :, 1], s["D"])
    kw = {"z": s["z"], "dt_bias": s["dt_bias"], "h0": s["h0"], "lengths": s["lengths"]}
    if not s["train"]:
        return gss.selective_scan(*args, **kw)
    (y, hn), ctx = gss.selective_scan_train(*args, **kw)
    g = gss.selective_scan_backward(ctx, s["dy"], s["dhn"])
    out = (y, hn, g["x"], g["dt"], g["A"], g["B"], g["C"], g["D"], g["dt_bias"], g["h0"])
    return out + ((g["z"],) if s["gate"] else ())


def _own_feed(s):
    import gru_sequence_scan_amd as gss
    kw = {"residual": s["r"], "activation": s["activation"]}
    if not s["train"]:
        return gss.feed_forward(s["x"], s["w_in"], s["w_out"], **kw)
    y, ctx = gss.feed_forward_train(s["x"], s["w_in"], s["w_out"], **kw)
    return (y,) + gss.feed_forward_backward(ctx, s["dy"])


# -- their plain form --

def _live(s):
    """Whether row b has a step t, [T, B, 1]."""
    t = torch.arange(s["T"], device=DEV)[:, None]
    L = torch.full((1, s["B"]), s["T"], device=DEV) if s["lengths"] is None else s["lengths"].long()[None]
    return (t < L)[:, :, None]


def _plain_conv(s):
    x, w, b = s["xz"][:, :, 0], s["w"].float(), s["b"].float()
    dt, T, B, W = x.dtype, s["T"], s["B"], s["W"]
    live = _live(s)
    full = torch.cat([s["state"].float(), torch.where(live, x.float(), torch.zeros((), device=DEV))])
    p = b + sum(w[:, k] * full[k:k + T] for k in range(W))
    sig = torch.sigmoid(p)
    y = torch.where(live, p * sig if s["silu"] else p, torch.zeros_like(p))
    L = live[:, :, 0].sum(0)
    at = (L[None] + torch.arange(W - 1, device=DEV)[:, None])[:, :, None].expand(W - 1, B, s["C"])
    last = torch.gather(full, 0, at)
    if not s["train"]:
        return y.to(dt), last.to(dt)
    dp = torch.where(live, s["dy"].float(), torch.zeros_like(p))
    if s["silu"]:
        dp = dp * (sig + p * sig * torch.sigmoid(-p))
    dfull = torch.zeros_like(full)
    for k in range(W):
        dfull[k:k + T] += w[:, k] * dp
    dfull.scatter_add_(0, at, s["dstate"].float())
    dw = torch.stack([(dp * full[k:k + T]).sum((0, 1)) for k in range(W)], 1)
    dx = torch.where(live, dfull[W - 1:], torch.zeros_like(p))
    return y.to(dt), last.to(dt), dx.to(dt), dw, dp.sum((0, 1)), dfull[:W - 1].to(dt)


def _linear_scan(a, u):
    """h_t = a_t h_{t-1} + u_t over dimension 0 from h = 0, by doubling."""
    d, T = 1, a.shape[0]
    while d < T:
        u = torch.cat([u[:d], u[d:] + a[d:] * u[:-d]])
        a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return u


def _plain_scan(s):
    T, B, H, N, G = (s[k] for k in ("T", "B", "H", "N", "groups"))
    dt, live = s["x"].dtype, _live(s)
    x, A, D, h0 = s["x"].float(), s["A"], s["D"], s["h0"]
    raw = s["dt"].float() + s["dt_bias"]
    delta = torch.clamp(raw, min=0.0) + torch.log1p(torch.exp(-raw.abs()))
    delta = torch.where(live, delta, torch.zeros_like(delta))
    Bm, Cm = (s["bc"][:, :, i].float()[:, :, :, None] for i in (0, 1))    # [T, B, G, 1, N]
    a = torch.exp(delta[..., None] * A)                                   # 1 past a row's end
    u = ((delta * x).view(T, B, G, H // G, 1) * Bm).view(T, B, H, N)
    u[0] += a[0] * h0
    h = _linear_scan(a, u)
    del u
    hn = h[-1].clone()
    y = (h.view(T, B, G, H // G, N) * Cm).sum(-1).view(T, B, H) + D * x
    zero = torch.zeros_like(y)
    if s["gate"]:
        z = s["z"].float()
        sig = torch.sigmoid(z)
        gate = z * sig
    out = torch.where(live, y * gate if s["gate"] else y, zero).to(dt)
    if not s["train"]:
        return out, hn
    dout = torch.where(live, s["dy"].float(), zero)
    dY = dout * gate if s["gate"] else dout
    dv = dY.view(T, B, G, H // G, 1)
    dC = (dv * h.view(T, B, G, H // G, N)).sum(3)
    g = (dv * Cm).view(T, B, H, N)
    g[-1] += s["dhn"]
    back = torch.cat([torch.ones_like(a[:1]), a[1:].flip(0)])
    g = _linear_scan(back, g.flip(0)).flip(0)
    del back
    dh0 = a[0] * g[0]
    w = a * g * torch.cat([h0[None], h[:-1]])
    del a, h
    dA = (w * delta[..., None]).sum((0, 1))
    ddelta = (w * A).sum(-1)
    del w
    gv = g.view(T, B, G, H // G, N)
    gB = (gv * Bm).sum(-1).view(T, B, H)
    dB = (gv * (delta * x).view(T, B, G, H // G, 1)).sum(3)
    ddelta = ddelta + x * gB
    dx = torch.where(live, delta * gB + D * dY, zero)
    ddt = torch.where(live, ddelta * torch.sigmoid(raw), zero)
    grads = (dx.to(dt), ddt.to(dt), dA, dB.to(dt), dC.to(dt), (dY * x).sum((0, 1)), ddt.sum((0, 1)), dh0)
    if not s["gate"]:
        return (out, hn) + grads
    dz = dout * y * (sig + z * sig * torch.sigmoid(-z))
    return (out, hn) + grads + (torch.where(live, dz, zero).to(dt),)


def _activation(g, kind):
    """act(g) and its derivative."""
    if kind == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    sig, no = torch.sigmoid(g), torch.sigmoid(-g)
    if kind == "sigmoid":
        return sig, sig * no
    return g * sig, sig + g * sig * no


def _plain_feed(s):
    dt, F = s["x"].dtype, s["F"]
    x, w_in, w_out = s["x"].float(), s["w_in"].float(), s["w_out"].float()
    p = torch.matmul(x, w_in.t())
    g, u = p[:, :F], p[:, F:]
    act, slope = _activation(g, s["activation"])
    h = act * u
    y = torch.matmul(h, w_out.t())
    if s["residual"]:
        y = y + s["r"].float()
    if not s["train"]:
        return y.to(dt)
    dy = s["dy"].float()
    dh = torch.matmul(dy, w_out)
    dp = torch.cat([dh * u * slope, dh * act], 1)
    dx = torch.matmul(dp, w_in)
    return y.to(dt), dx.to(dt), torch.matmul(dp.t(), x).to(dt), torch.matmul(dy.t(), h).to(dt)


_run_own = {"conv": _own_conv, "scan": _own_scan, "feed": _own_feed}
_run_plain = {"conv": _plain_conv, "scan": _plain_scan, "feed": _plain_feed}


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "feed": _exact_feed}[case["op"]](s)


def _row_lengths(s):
    return [s["T"]] * s["B"] if s["lengths"] is None else s["lengths"].tolist()


def _exact_conv(s):
    """Row by row, as a correlation of the row with its history in front;
    gradients by differentiation."""
    T, B, C, W = s["T"], s["B"], s["C"], s["W"]
    x, w, b, state = (t.double().requires_grad_(s["train"]) for t in (s["xz"][:, :, 0], s["w"], s["b"], s["state"]))
    y, last = [], []
    for row, L in enumerate(_row_lengths(s)):
        seq = torch.cat([state[:, row], x[:L, row]])
        p = seq.unfold(0, W, 1).mul(w).sum(-1) + b if L else torch.zeros(0, C, dtype=torch.float64, device=DEV)
        if s["silu"]:
            p = p / (1 + torch.exp(-p))
        y.append(torch.cat([p, torch.zeros(T - L, C, dtype=torch.float64, device=DEV)]))
        last.append(seq[L:])
    y, last = torch.stack(y, 1), torch.stack(last, 1)
    if not s["train"]:
        return y, last
    loss = (y * s["dy"].double()).sum() + (last * s["dstate"].double()).sum()
    return (y.detach(), last.detach()) + torch.autograd.grad(loss, (x, w, b, state))


def _exact_scan(s):
    """The recurrence one step at a time, and its chain rule likewise."""
    T, B, H, N, G = (s[k] for k in ("T", "B", "H", "N", "groups"))
    A, D, bias = s["A"].double(), s["D"].double(), s["dt_bias"].double()
    L = torch.tensor(_row_lengths(s), device=DEV)
    heads = torch.arange(H, device=DEV) // (H // G)

    def at(t):
        on = (t < L)[:, None]
        raw = s["dt"][t].double() + bias
        delta = torch.where(raw > 0, raw + torch.log1p(torch.exp(-raw.abs())), torch.log1p(torch.exp(-raw.abs())))
        b, c = s["bc"][t, :, 0].double()[:, heads], s["bc"][t, :, 1].double()[:, heads]   # [B, H, N]
        z = s["z"][t].double() if s["gate"] else None
        return on, raw, delta, s["x"][t].double(), b, c, torch.exp(delta[..., None] * A), z

    h = s["h0"].double()
    states = torch.zeros((T if s["train"] else 0, B, H, N), dtype=torch.float64, device=DEV)
    out = torch.zeros((T, B, H), dtype=torch.float64, device=DEV)
    for t in range(T):
        on, _, delta, x, b, c, a, z = at(t)
        if s["train"]:
            states[t] = h
        h = torch.where(on[..., None], a * h + (delta * x)[..., None] * b, h)
        y = (h * c).sum(-1) + D * x
        out[t] = torch.where(on, y if z is None else y * z / (1 + torch.exp(-z)), torch.zeros_like(y))
    if not s["train"]:
        return out, h
    grads = [torch.zeros_like(out) for _ in range(3 if s["gate"] else 2)]
    dB, dC = torch.zeros((2, T, B, G, N), dtype=torch.float64, device=DEV)
    dA, dD, dbias = torch.zeros_like(A), torch.zeros_like(D), torch.zeros_like(bias)
    carry = s["dhn"].double()
    for t in range(T - 1, -1, -1):
        on, raw, delta, x, b, c, a, z = at(t)
        before = states[t]
        now = a * before + (delta * x)[..., None] * b
        do = torch.where(on, s["dy"][t].double(), torch.zeros_like(x))
        if s["gate"]:
            sig = 1 / (1 + torch.exp(-z))
            grads[2][t] = do * ((now * c).sum(-1) + D * x) * sig * (1 + z * (1 - sig))
            do = do * z * sig
        dC[t].index_add_(1, heads, do[..., None] * now)
        total = carry + do[..., None] * c
        total_on = torch.where(on[..., None], total, torch.zeros_like(total))
        dB[t].index_add_(1, heads, total_on * (delta * x)[..., None])
        decay = total_on * a * before
        through = (total_on * b).sum(-1)
        dA += (decay * delta[..., None]).sum(0)
        grads[0][t] = delta * through + D * do
        ddt = ((decay * A).sum(-1) + x * through) / (1 + torch.exp(-raw))
        grads[1][t] = ddt
        dbias += ddt.sum(0)
        dD += (do * x).sum(0)
        carry = torch.where(on[..., None], a * total, carry)
    return (out, h, grads[0], grads[1], dA, dB, dC, dD, dbias, carry) + tuple(grads[2:])


def _exact_feed(s):
    F = s["F"]
    leaf = [s[k].double().requires_grad_(s["train"]) for k in ("x", "w_in", "w_out")]
    x, w_in, w_out = leaf
    g, u = x @ w_in[:F].t(), x @ w_in[F:].t()
    if s["activation"] == "silu":
        g = g / (1 + torch.exp(-g))
    elif s["activation"] == "sigmoid":
        g = 1 / (1 + torch.exp(-g))
    else:
        g = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    y = (g * u) @ w_out.t()
    if s["residual"]:
        y = y + s["r"].double()
    if not s["train"]:
        return y
    return (y.detach(),) + torch.autograd.grad(y, leaf, s["dy"].double())
