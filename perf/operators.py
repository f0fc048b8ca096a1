"""What the decoder operators are measured on: layer norm, the gated linear
scan and cross attention, each beside its plain form.

A recurrent decoder block uses them in turn: norm, gated scan over the target
sequence, residual add and norm, cross attention to the states of a
(bidirectional, variable-length) encoder. Tensors are time-major, [T, B, ...],
as the library's padded layout has them.
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

def _norm(rows, n, dtype, residual, train):
    return {"op": "norm", "rows": rows, "n": n, "dtype": dtype, "residual": residual, "train": train}


def _scan(T, B, H, dtype, input_gate, reverse, lo, train):
    # lo: the shortest row of a ragged batch; -1: every row has T steps
    return {"op": "scan", "T": T, "B": B, "H": H, "dtype": dtype, "input_gate": input_gate, "reverse": reverse,
            "lo": lo, "train": train}


def _attend(Tq, Tk, B, heads, kv_heads, D, dtype, lo, train):
    # lo: the shortest encoder row of a ragged batch; -1: every row has Tk states
    return {"op": "attend", "Tq": Tq, "Tk": Tk, "B": B, "heads": heads, "kv_heads": kv_heads, "D": D, "dtype": dtype,
            "lo": lo, "train": train}


def listed():
    named = [
        # the norm of a narrow belief state between two steps of a 50-row unroll: pure latency, an odd width
        ("norm_step_b50", _norm(50, 200, "f32", False, False)),
        # the residual add and norm of one decoding step for 64 requests
        ("norm_step_b64", _norm(64, 1024, "bf16", True, False)),
        # training on a packed variable-length batch: as many rows as it has tokens
        ("norm_train_packed", _norm(19334, 512, "f32", False, True)),
        # training a residual stack, 32 sequences of 1000 steps
        ("norm_train_t1000_b32", _norm(32000, 1024, "bf16", True, True)),
        # one decoding step of the recurrence for 64 requests
        ("scan_step_b64", _scan(1, 64, 1024, "bf16", False, False, -1, False)),
        # reading 32 prompts of 1000 steps
        ("scan_forward_t1000_b32", _scan(1000, 32, 1024, "bf16", False, False, -1, False)),
        # training the reverse direction on 64 ragged sequences, with a gate of its own for the input
        ("scan_train_varlen_b64", _scan(500, 64, 512, "f32", True, True, 50, True)),
        # training on two long sequences: few channels, so time itself has to be split
        ("scan_train_t16384_b2", _scan(16384, 2, 1000, "bf16", False, False, -1, True)),
        # one decoding step of 64 requests over the encoder's states, ragged, one slot idle
        ("attend_step_b64", _attend(1, 500, 64, 8, 8, 64, "bf16", 0, False)),
        # one decoding step of a single request over a long document, shared key and value heads
        ("attend_step_long", _attend(1, 32773, 1, 16, 2, 128, "bf16", -1, False)),
        # training in fp32 on 32 ragged pairs, 80 target steps
        ("attend_train_f32", _attend(80, 500, 32, 4, 4, 64, "f32", 50, True)),
        # training in bf16 on 32 ragged pairs of up to 1000 steps each side, shared key and value heads
        ("attend_train_t1000_b32", _attend(1000, 1000, 32, 8, 2, 128, "bf16", 100, True)),
    ]
    out = []
    for name, case in named:
        case["name"] = name
        out.append(case)
    return out


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case: sizes log-uniform over what the listed ones span, odd
    sizes as likely as round ones, bounded by the largest listed case."""
    op = rng.choice(["norm", "scan", "attend"])
    dtype = rng.choice(["f32", "bf16"])
    train = rng.random() < 0.5
    if op == "norm":
        n = _log_int(rng, 16, 4096)
        if rng.random() < 0.5:
            n = max(16, n // 8 * 8)
        rows = min(_log_int(rng, 1, 40000), 32_000_000 // n)
        return _norm(rows, n, dtype, rng.random() < 0.5, train)
    if op == "scan":
        T, B, H = _log_int(rng, 1, 16384), _log_int(rng, 1, 64), _log_int(rng, 16, 2048)
        if rng.random() < 0.7:
            H = max(16, H // 8 * 8)
        while T * B * H > 32_000_000:
            T, B = max(1, T // 2), max(1, B - B // 4)
        lo = rng.choice([-1, 0, T // 4])
        return _scan(T, B, H, dtype, rng.random() < 0.5, rng.random() < 0.5, lo, train)
    D = rng.choice([32, 40, 64, 72, 80, 96, 100, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 1, 2, 4])
    B = _log_int(rng, 1, 64)
    Tq = 1 if not train and rng.random() < 0.5 else _log_int(rng, 2, 1000)
    Tk = _log_int(rng, 8, 4000)
    limit = 0.9 * 32 * 1000 * 550 * 8 * 128 * (0.1 if dtype == "f32" else 1.0)
    while B * Tq * Tk * heads * D > limit:
        Tq, B, Tk = max(1, Tq - Tq // 4), max(1, B - B // 4), max(8, Tk - Tk // 8)
    lo = rng.choice([-1, 0, Tk // 8])
    return _attend(Tq, Tk, B, heads, kv_heads, D, dtype, lo, train)


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
    if case["op"] == "norm":
        n = case["rows"] * case["n"]
        tensors = 2 + (2 if case["residual"] else 0)
        if case["train"]:
            tensors += 2 + (1 if case["residual"] else 0)  # dy (and the sum's gradient) in, dx out
        small = case["n"] * (2 * e + (8 if case["train"] else 0))
        return {"bytes": tensors * n * e + small, "flops": (24 if case["train"] else 9) * n}
    if case["op"] == "scan":
        T, B, H = case["T"], case["B"], case["H"]
        lens = _lengths(case["lo"], T, B)
        tok = T * B if lens is None else sum(lens)
        gates = 3 if case["input_gate"] else 2
        state = 8 * B * H
        if not case["train"]:
            return {"bytes": (gates * tok + T * B) * H * e + state, "flops": 10 * tok * H}
        return {"bytes": ((gates + 1) * tok + (gates + 1) * T * B) * H * e + 2 * state, "flops": 30 * tok * H}
    Tq, Tk, B, D = case["Tq"], case["Tk"], case["B"], case["D"]
    lens = _lengths(case["lo"], Tk, B)
    keys = Tk * B if lens is None else sum(lens)
    q, kv = Tq * B * case["heads"] * D, keys * case["kv_heads"] * D
    pairs = Tq * keys * case["heads"] * D
    if not case["train"]:
        return {"bytes": (2 * q + 2 * kv) * e, "flops": 4 * pairs}
    whole = Tk * B * case["kv_heads"] * D
    return {"bytes": (4 * q + 2 * kv + 2 * whole) * e, "flops": 14 * pairs}


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
    if case["op"] == "norm":
        rows, n = case["rows"], case["n"]
        # a residual stream: an offset per channel, and values of another size than the branch that is added
        st["x"] = _normal(g, (rows, n), dt, 0.0, 0.7)
        st["r"] = (_normal(g, (rows, n), torch.float32, 0.0, 2.0) + _normal(g, (n,), torch.float32)).to(dt) if case["residual"] else None
        st["w"] = _normal(g, (n,), dt, 1.0, 0.2)
        st["b"] = _normal(g, (n,), dt, 0.0, 0.2)
        if case["train"]:
            st["dy"] = _normal(g, (rows, n), dt)
            st["ds"] = _normal(g, (rows, n), dt) if case["residual"] else None
    elif case["op"] == "scan":
        shape = (case["T"], case["B"], case["H"])
        # the gates and the candidate as one projection writes them: thirds (halves) of its rows
        parts = 3 if case["input_gate"] else 2
        p = torch.randn(shape[:2] + (parts, shape[2]), generator=g, device=DEV)
        p[:, :, 0] = p[:, :, 0] * 1.5 + 2.0   # forget gates that mostly keep
        p = p.to(dt)
        st["proj"] = p
        st["h0"] = _normal(g, shape[1:], torch.float32, 0.0, 0.5)
        st["lengths"] = _length_tensor(case, case["T"], seed)
        if case["train"]:
            st["dy"] = _normal(g, shape, dt)
            st["dhn"] = _normal(g, shape[1:], torch.float32)
    else:
        B, D = case["B"], case["D"]
        st["q"] = _normal(g, (case["Tq"], B, case["heads"], D), dt)
        # keys and values as one projection of the encoder's states writes them
        st["kv"] = _normal(g, (case["Tk"], B, 2, case["kv_heads"], D), dt)
        st["lengths"] = _length_tensor(case, case["Tk"], seed)
        if case["train"]:
            st["do"] = _normal(g, (case["Tq"], B, case["heads"], D), dt)
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)[state["op"]](state)


# -- the library's operators --

def _own_norm(s):
    import gru_sequence_scan_amd as gss
    if not s["train"]:
        return gss.layer_norm(s["x"], s["w"], s["b"], residual=s["r"])
    (y, total), ctx = gss.layer_norm_train(s["x"], s["w"], s["b"], residual=s["r"])
    dx, dw, db = gss.layer_norm_backward(ctx, s["dy"], s["ds"])
    return (y, total, dx, dw, db) if s["residual"] else (y, dx, dw, db)


def _own_scan(s):
    import gru_sequence_scan_amd as gss
    p = s["proj"]
    gate = p[:, :, 2] if s["input_gate"] else None
    if not s["train"]:
        return gss.gated_scan(p[:, :, 1], p[:, :, 0], gate, h0=s["h0"], lengths=s["lengths"], reverse=s["reverse"])
    (y, hn), ctx = gss.gated_scan_train(p[:, :, 1], p[:, :, 0], gate, h0=s["h0"], lengths=s["lengths"],
                                        reverse=s["reverse"])
    dx, df, di, dh0 = gss.gated_scan_backward(ctx, s["dy"], s["dhn"])
    return (y, hn, dx, df, dh0) + ((di,) if s["input_gate"] else ())


def _own_attend(s):
    import gru_sequence_scan_amd as gss
    k, v = s["kv"][:, :, 0], s["kv"][:, :, 1]
    if not s["train"]:
        return gss.cross_attention(s["q"], k, v, lengths=s["lengths"])
    o, ctx = gss.cross_attention_train(s["q"], k, v, lengths=s["lengths"])
    return (o,) + gss.cross_attention_backward(ctx, s["do"])


# -- their plain form --

def _plain_norm(s, eps=1e-5):
    dt = s["x"].dtype
    total = s["x"]
    if s["residual"]:
        total = (s["x"].float() + s["r"].float()).to(dt)  # an output of its own: the stream as the next block reads it
    z, w, b = total.float(), s["w"].float(), s["b"].float()
    z = z - z.mean(-1, keepdim=True)
    rstd = torch.rsqrt((z * z).mean(-1, keepdim=True) + eps)
    xh = z * rstd
    y = (xh * w + b).to(dt)
    if not s["train"]:
        return (y, total) if s["residual"] else y
    dy = s["dy"].float()
    gw = dy * w
    dx = rstd * (gw - gw.mean(-1, keepdim=True) - xh * (gw * xh).mean(-1, keepdim=True))
    if s["residual"]:
        dx = dx + s["ds"].float()
    out = (dx.to(dt), (dy * xh).sum(0), dy.sum(0))
    return ((y, total) if s["residual"] else (y,)) + out


def _linear_scan(a, u):
    """h_t = a_t h_{t-1} + u_t over dimension 0 from h = 0, by doubling."""
    d, T = 1, a.shape[0]
    while d < T:
        u = torch.cat([u[:d], u[d:] + a[d:] * u[:-d]])
        a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return u


def _time_index(s):
    """Row t of [T, B]: the time that step t of each batch row reads, and
    whether the row is that long."""
    T, B = s["T"], s["B"]
    t = torch.arange(T, device=DEV)[:, None]
    L = torch.full((1, B), T, device=DEV) if s["lengths"] is None else s["lengths"].long()[None]
    live = t < L
    return (torch.where(live, L - 1 - t, t) if s["reverse"] else t.expand(T, B)), live, L


def _plain_scan(s):
    p = s["proj"].float()
    dt, T = s["proj"].dtype, s["T"]
    idx, live, L = _time_index(s)
    turn = s["reverse"]
    live = live[:, :, None]
    whole = s["lengths"] is None and not turn
    order = None if not turn else idx[:, :, None].expand(T, s["B"], s["H"])

    def steps(v):  # time order -> step order (its own inverse)
        return v if order is None else torch.gather(v, 0, order)

    f, x = steps(p[:, :, 0]), steps(p[:, :, 1])
    a, h0 = torch.sigmoid(f), s["h0"]
    keep = torch.sigmoid(-f)
    s_in = torch.sigmoid(steps(p[:, :, 2])) if s["input_gate"] else keep
    if whole:
        aa, u = a, s_in * x
    else:  # steps past the end keep the state
        aa, u = torch.where(live, a, torch.ones_like(a)), torch.where(live, s_in * x, torch.zeros_like(a))
    u = torch.cat([u[:1] + aa[:1] * h0, u[1:]])
    h = _linear_scan(aa, u)
    hn = h[-1].clone()
    y = steps(h * live).to(dt)
    if not s["train"]:
        return y, hn
    dy = steps(s["dy"].float()) * live
    dy = torch.cat([dy[:-1], dy[-1:] + s["dhn"]])
    # g_t = dy_t + a_{t+1} g_{t+1}: the same scan from the far end
    back = torch.cat([torch.ones_like(aa[:1]), aa[1:].flip(0)])
    g = _linear_scan(back, dy.flip(0)).flip(0)
    dh0 = aa[0] * g[0]
    hp = torch.cat([h0[None], h[:-1]])
    g = g * live
    if s["input_gate"]:
        df, di, dx = g * hp * a * keep, g * x * s_in * torch.sigmoid(-steps(p[:, :, 2])), g * s_in
        return y, hn, steps(dx).to(dt), steps(df).to(dt), dh0, steps(di).to(dt)
    df, dx = g * (hp - x) * a * keep, g * keep
    return y, hn, steps(dx).to(dt), steps(df).to(dt), dh0


def _plain_attend(s):
    dt = s["q"].dtype
    Tq, B, Hq, D = s["q"].shape
    Tk, Hk = s["kv"].shape[0], s["kv_heads"]
    G, scale = Hq // Hk, 1.0 / math.sqrt(D)

    def rows(t):  # [Tq, B, Hq, D] -> [B, Hk, G Tq, D]
        return t.float().view(Tq, B, Hk, G, D).permute(1, 2, 3, 0, 4).reshape(B, Hk, G * Tq, D)

    def unrows(t):
        return t.view(B, Hk, G, Tq, D).permute(3, 0, 1, 2, 4).reshape(Tq, B, Hq, D).to(dt)

    q = rows(s["q"])
    k = s["kv"][:, :, 0].float().permute(1, 2, 0, 3).contiguous()
    v = s["kv"][:, :, 1].float().permute(1, 2, 0, 3).contiguous()
    p = torch.matmul(q, k.transpose(-1, -2).contiguous()) * scale
    if s["lengths"] is not None:
        off = (torch.arange(Tk, device=DEV)[None] >= s["lengths"][:, None])[:, None, None]
        p = p.masked_fill(off, float("-inf"))
    m = p.amax(-1, keepdim=True)
    p = torch.exp(p - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    p = p / torch.where(l > 0, l, torch.ones_like(l))
    o = torch.matmul(p, v)
    if not s["train"]:
        return unrows(o)
    do = rows(s["do"])
    dp = torch.matmul(do, v.transpose(-1, -2).contiguous())
    ds = p * (dp - (do * o).sum(-1, keepdim=True)) * scale
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2).contiguous(), q)
    dv = torch.matmul(p.transpose(-1, -2).contiguous(), do)
    back = [t.permute(2, 0, 1, 3).contiguous().to(dt) for t in (dk, dv)]
    return unrows(o), unrows(dq), back[0], back[1]


_run_own = {"norm": _own_norm, "scan": _own_scan, "attend": _own_attend}
_run_plain = {"norm": _plain_norm, "scan": _plain_scan, "attend": _plain_attend}


# ---------------------------------------------------------------------------
# 64 bits, from the definitions
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "scan": _exact_scan, "attend": _exact_attend}[case["op"]](s)


def _exact_norm(s):
    total = s["x"]
    if s["residual"]:
        total = (s["x"].double() + s["r"].double()).to(s["x"].dtype)  # the stream is what is stored of the sum
    leaf = [t.double().requires_grad_(s["train"]) for t in (total, s["w"], s["b"])]
    z, w, b = leaf
    y = (z - z.mean(-1, keepdim=True)) / torch.sqrt(z.var(-1, unbiased=False, keepdim=True) + 1e-5) * w + b
    if not s["train"]:
        return (y, total.double()) if s["residual"] else y
    dx, dw, db = torch.autograd.grad(y, leaf, s["dy"].double())
    if s["residual"]:
        return y.detach(), total.double(), dx + s["ds"].double(), dw, db
    return y.detach(), dx, dw, db


def _exact_scan(s):
    """The recurrence one step at a time, and its chain rule likewise."""
    p = s["proj"].double()
    T, B, H = s["T"], s["B"], s["H"]
    L = torch.full((B,), T, device=DEV) if s["lengths"] is None else s["lengths"].long()
    gate = s["input_gate"]
    a, x = torch.sigmoid(p[:, :, 0]), p[:, :, 1]
    w = torch.sigmoid(p[:, :, 2]) if gate else 1.0 - a
    order = range(T - 1, -1, -1) if s["reverse"] else range(T)
    live = torch.arange(T, device=DEV)[:, None] < L[None]
    live = live[:, :, None]
    h = s["h0"].double()
    before = torch.zeros(T, B, H, dtype=torch.float64, device=DEV)
    y = torch.zeros_like(before)
    for t in order:
        before[t] = h
        h = torch.where(live[t], a[t] * h + w[t] * x[t], h)
        y[t] = h
    y = y * live
    if not s["train"]:
        return y, h
    g = s["dhn"].double()
    dy = s["dy"].double()
    at = torch.zeros_like(before)
    for t in reversed(order):
        total = g + dy[t]
        at[t] = total
        g = torch.where(live[t], a[t] * total, g)
    at = at * live
    da = at * before - (0.0 if gate else at * x)
    df, dx = da * a * (1 - a), at * w
    if gate:
        return y, h, dx, df, g, at * x * w * (1 - w)
    return y, h, dx, df, g


def _exact_attend(s):
    Tq, B, Hq, D = s["q"].shape
    Tk, Hk = s["kv"].shape[0], s["kv_heads"]
    if Tq * Tk * B * Hq * D * (7 if s["train"] else 2) > 2e12:
        return None
    G = Hq // Hk
    o = torch.zeros(Tq, B, Hq, D, dtype=torch.float64, device=DEV)
    dq = torch.zeros_like(o)
    dk = torch.zeros(Tk, B, Hk, D, dtype=torch.float64, device=DEV)
    dv = torch.zeros_like(dk)
    for b in range(B):
        n = Tk if s["lengths"] is None else int(s["lengths"][b])
        if n == 0:
            continue
        for h in range(Hk):
            heads = slice(h * G, (h + 1) * G)
            leaf = [t.double().contiguous().requires_grad_(s["train"]) for t in (
                s["q"][:, b, heads].reshape(Tq * G, D), s["kv"][:n, b, 0, h], s["kv"][:n, b, 1, h])]
            out = torch.softmax(leaf[0] @ leaf[1].t() / math.sqrt(D), -1) @ leaf[2]
            o[:, b, heads] = out.detach().view(Tq, G, D)
            if s["train"]:
                gq, gk, gv = torch.autograd.grad(out, leaf, s["do"][:, b, heads].double().reshape(Tq * G, D))
                dq[:, b, heads] = gq.view(Tq, G, D)
                dk[:n, b, h], dv[:n, b, h] = gk, gv
    return (o, dq, dk, dv) if s["train"] else o
