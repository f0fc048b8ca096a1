"""The state-space block's operators on the CPU: the float64 definitions
against torch and against differences, and the refusals of the C entry points
and of the Python calls, which all come before anything touches a device."""

import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import oracle

gss = pytest.importorskip("gru_sequence_scan_amd")
ops = gss.block_ops

OK, E_NULL, E_SHAPE, E_UNSUPPORTED, E_WORKSPACE, E_ALIGN, E_DEVICE = 0, -1, -2, -3, -5, -6, -7
ADDR = 4096
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _differences(fn, v, eps=1e-6):
    """d fn / d v by central differences, fn a scalar function."""
    g = np.zeros_like(v)
    for k in np.ndindex(v.shape):
        keep = v[k]
        v[k] = keep + eps
        up = fn()
        v[k] = keep - eps
        down = fn()
        v[k] = keep
        g[k] = (up - down) / (2 * eps)
    return g


def _layouts(tmp_path, names):
    """The structs' sizes and offsets in C are those of their ctypes mirrors."""
    lines = [f'  printf("%zu", sizeof({n}));' + "".join(f' printf(" %zu", offsetof({n}, {f[0]}));'
                                                       for f in getattr(gss, n)._fields_) + ' printf("\\n");' for n in names]
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"rnn.h\"\nint main(void) {\n" + "\n".join(lines) +
                   "\n  return 0;\n}\n")
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "layout")], check=True)
    out = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout.splitlines()
    for n, line in zip(names, out):
        t = getattr(gss, n)
        assert [int(v) for v in line.split()] == [ctypes.sizeof(t)] + [getattr(t, f[0]).offset for f in t._fields_]




@pytest.mark.parametrize("pack,name", [
    ("_CONV_DESC", "RnnCausalConvDesc"), ("_CONV_IO", "RnnCausalConvIO"), ("_CONV_GRADS", "RnnCausalConvGrads"),
    ("_SCAN_DESC", "RnnSelectiveScanDesc"), ("_SCAN_IO", "RnnSelectiveScanIO"), ("_SCAN_GRADS", "RnnSelectiveScanGrads"),
    ("_FEED_DESC", "RnnFeedForwardDesc"), ("_FEED_IO", "RnnFeedForwardIO"), ("_FEED_GRADS", "RnnFeedForwardGrads"),
])
def test_packed_structs_are_the_ctypes_ones(pack, name):
    t = getattr(gss, name)
    data = getattr(gss.state_block_ops, pack)(*range(1, len(t._fields_) + 1))
    assert len(data) == ctypes.sizeof(t)
    s = t.from_buffer_copy(data)
    assert [getattr(s, f[0]) for f in t._fields_] == list(range(1, len(t._fields_) + 1))


# ---------------------------------------------------------------------------
# Causal convolution
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("activation", [None, "silu"])
@pytest.mark.parametrize("W", [2, 4, 5])
def test_causal_conv_definition(W, activation):
    rng = np.random.default_rng(1)
    T, B, C = 5, 4, 3
    x, dy = rng.standard_normal((2, T, B, C))
    w, b = rng.standard_normal((C, W)), rng.standard_normal(C)
    state, ds = rng.standard_normal((2, W - 1, B, C))
    lens = [5, 0, 1, 4]
    y, last = oracle.causal_conv(x, w, b, state, lens, activation)
    ref = torch.nn.functional.conv1d(torch.tensor(np.concatenate([state, x])).permute(1, 2, 0), torch.tensor(w)[:, None],
                                     torch.tensor(b), groups=C).permute(2, 0, 1)
    ref = torch.nn.functional.silu(ref) if activation else ref
    for row, L in enumerate(lens):
        assert np.allclose(y[:L, row], ref[:L, row].numpy(), atol=1e-12) and (y[L:, row] == 0).all()
        assert np.array_equal(last[:, row], np.concatenate([state[:, row], x[:L, row]])[L:])

    def loss():
        y, last = oracle.causal_conv(x, w, b, state, lens, activation)
        return float((y * dy).sum() + (last * ds).sum())

    grads = oracle.causal_conv_backward(x, w, b, dy, ds, state, lens, activation)
    for got, v in zip(grads, (x, w, b, state)):
        assert np.allclose(got, _differences(loss, v), atol=1e-7)


def test_causal_conv_in_parts_is_the_whole():
    rng = np.random.default_rng(2)
    x, w = rng.standard_normal((9, 2, 3)), rng.standard_normal((3, 4))
    whole, last = oracle.causal_conv(x, w)
    state, parts = None, []
    for a, b in ((0, 1), (1, 6), (6, 9)):
        y, state = oracle.causal_conv(x[a:b], w, None, state)
        parts.append(y)
    assert np.allclose(np.concatenate(parts), whole, atol=1e-13) and np.array_equal(state, last)


def test_conv_layout(tmp_path):
    _layouts(tmp_path, ["RnnCausalConvDesc", "RnnCausalConvIO", "RnnCausalConvGrads"])


def _conv(**kw):
    v = dict(dtype=0, T=30, B=4, C=8, W=4, activation=1, x_t=32, x_b=8)
    v.update(kw)
    return gss.RnnCausalConvDesc(*v.values())


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), ({"dtype": 1}, OK), ({"W": 2}, OK), ({"W": 8}, OK), ({"activation": 0}, OK), ({"x_b": 0}, OK),
    ({"dtype": 2}, E_UNSUPPORTED), ({"W": 1}, E_UNSUPPORTED), ({"W": 9}, E_UNSUPPORTED), ({"W": 0}, E_SHAPE),
    ({"activation": 2}, E_UNSUPPORTED), ({"activation": -1}, E_UNSUPPORTED),
    ({"T": 0}, E_SHAPE), ({"B": 0}, E_SHAPE), ({"C": 0}, E_SHAPE), ({"x_t": -1}, E_SHAPE), ({"x_b": -8}, E_SHAPE),
    ({"T": 2147483647}, E_SHAPE), ({"T": 160000, "B": 1 << 19, "C": 4096}, E_SHAPE),
    ({"T": 1 << 20, "B": 1 << 10, "C": 63}, OK), ({"T": 1 << 20, "B": 1 << 10, "C": 64}, E_SHAPE),
    ({"T": 1, "B": 1, "C": 2147483647}, E_SHAPE), ({"T": 8, "B": 2147483647, "C": 1}, E_SHAPE),
])
def test_conv_desc(kw, expect):
    n = ctypes.c_size_t(0)
    assert ops._lib().rnn_causal_conv_backward_workspace_bytes(ctypes.byref(_conv(**kw)), ctypes.byref(n)) == expect
    if expect == OK:
        assert n.value >= 5 * 4 or kw.get("W") == 2


def test_conv_pointers():
    L = ops._lib()
    d = ctypes.byref(_conv())
    n = ctypes.c_size_t(0)
    assert L.rnn_causal_conv_backward_workspace_bytes(d, ctypes.byref(n)) == OK
    assert L.rnn_causal_conv_backward_workspace_bytes(d, None) == E_NULL

    def io(**kw):
        v = dict(x=ADDR, weight=ADDR, bias=ADDR, lengths=None, state=None, y=ADDR, state_n=ADDR)
        v.update(kw)
        return gss.RnnCausalConvIO(*v.values())

    def fwd(desc=d, **kw):
        return L.rnn_causal_conv(desc, ctypes.byref(io(**kw)), None)

    assert fwd(desc=None) == E_NULL and L.rnn_causal_conv(d, None, None) == E_NULL
    for k in ("x", "weight", "y"):
        assert fwd(**{k: None}) == E_NULL, k
    for k in ("x", "weight", "bias", "lengths", "state", "y", "state_n"):
        assert fwd(**{k: ADDR + 2}) == E_ALIGN, k

    def bwd(ws=ADDR, size=n.value, **kw):
        v = dict(dy=ADDR, dstate_n=None, dx=ADDR, dweight=ADDR, dbias=ADDR, dstate=None)
        v.update(kw)
        return L.rnn_causal_conv_backward(d, ctypes.byref(io()), ctypes.byref(gss.RnnCausalConvGrads(*v.values())), ws, size,
                                          None)

    for k in ("dy", "dx", "dweight"):
        assert bwd(**{k: None}) == E_NULL, k
    for k in ("dy", "dstate_n", "dx", "dweight", "dbias", "dstate"):
        assert bwd(**{k: ADDR + 1}) == E_ALIGN, k
    assert bwd(ws=None) == E_WORKSPACE and bwd(size=n.value - 1) == E_WORKSPACE and bwd(ws=ADDR + 4) == E_ALIGN
    assert L.rnn_causal_conv_backward(d, ctypes.byref(io()), None, ADDR, n.value, None) == E_NULL
    if not torch.cuda.is_available():
        assert fwd() == E_DEVICE and fwd(state_n=None, bias=None) == E_DEVICE and bwd() == E_DEVICE
        assert bwd(dbias=None) == E_DEVICE


def test_conv_python_refusals():
    x, w = torch.zeros(4, 2, 8, dtype=torch.float32), torch.zeros(8, 4, dtype=torch.float32)
    with pytest.raises(ValueError, match="GPU tensor"):
        gss.causal_conv(x, w)
    with pytest.raises(ValueError, match="activation"):
        gss.causal_conv(x, w, activation="gelu_tanh")
    with pytest.raises(ValueError, match="dimensions"):
        gss.causal_conv(x[0], w)
    with pytest.raises(ValueError, match="dtype"):
        gss.causal_conv(x.half(), w)


# ---------------------------------------------------------------------------
# Selective scan
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("G", [1, 2])
@pytest.mark.parametrize("full", [True, False])
def test_selective_scan_definition(full, G):
    rng = np.random.default_rng(4)
    T, B, H, N = 4, 3, 4, 3
    x, dt, z, dy = rng.standard_normal((4, T, B, H))
    Bm, Cm = rng.standard_normal((2, T, B, G, N))
    A = -np.exp(rng.standard_normal((H, N)))
    D, bias = rng.standard_normal((2, H))
    h0, dhn = rng.standard_normal((2, B, H, N))
    lens = [4, 0, 2]
    opt = dict(z=z, dt_bias=bias, soft=True) if full else dict(z=None, dt_bias=None, soft=False)
    D = D if full else None

    def loss():
        y, hn, _ = oracle.selective_scan(x, dt, A, Bm, Cm, D, h0=h0, lengths=lens, **opt)
        return float((y * dy).sum() + (hn * dhn).sum())

    g = oracle.selective_scan_backward(x, dt, A, Bm, Cm, D, dy, dhn, h0=h0, lengths=lens, **opt)
    # A difference of two losses of size |loss|, each rounded to 2^-53 of its
    # terms, over 2 eps = 2e-6 is off by up to |loss| 2^-52 / 2e-6 and as much
    # again for the sums' own roundings. (Steps may be negative here without
    # softplus: a state that grows by exp(-d A) reaches 1e9.)
    noise = abs(loss()) * 2.0 ** -52 / 1e-6
    for name, v in (("x", x), ("dt", dt), ("A", A), ("B", Bm), ("C", Cm), ("D", D), ("z", opt["z"]),
                    ("dt_bias", opt["dt_bias"]), ("h0", h0)):
        if v is not None:
            assert np.allclose(g[name], _differences(loss, v), atol=2e-7 + noise), name
    # a row without steps passes its state and its gradient through
    assert np.array_equal(oracle.selective_scan(x, dt, A, Bm, Cm, D, h0=h0, lengths=lens, **opt)[1][1], h0[1])
    assert np.array_equal(g["h0"][1], dhn[1])


def test_selective_scan_of_one_state_is_a_gated_scan():
    """N = 1, A = -1, B = C = 1 and unit-free inputs: h = a h + u with
    a = sigma(f) for d = -log sigma(f), u = (1 - sigma(f)) x."""
    rng = np.random.default_rng(5)
    T, B, H = 6, 2, 3
    x, f = rng.standard_normal((2, T, B, H))
    d = np.log1p(np.exp(-f))
    one = np.ones((T, B, 1, 1))
    u = x * (1 - np.exp(-d)) / d
    assert np.allclose(oracle.selective_scan(u, d, -np.ones((H, 1)), one, one, soft=False)[0],
                       oracle.gated_scan(x, f)[0], atol=1e-12)


def test_selective_layout(tmp_path):
    _layouts(tmp_path, ["RnnSelectiveScanDesc", "RnnSelectiveScanIO", "RnnSelectiveScanGrads"])


def _selective(**kw):
    v = dict(dtype=0, T=300, B=4, H=8, N=16, G=2, softplus=1, gate=1, x_t=32, x_b=8, dt_t=32, dt_b=8, z_t=32, z_b=8,
             B_t=128, B_b=32, B_g=16, C_t=128, C_b=32, C_g=16)
    v.update(kw)
    return gss.RnnSelectiveScanDesc(*v.values())


_SEL_SIZES = ("rnn_selective_scan_workspace_bytes", "rnn_selective_scan_reserve_bytes",
              "rnn_selective_scan_backward_workspace_bytes")


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), ({"dtype": 1}, OK), ({"N": 1}, OK), ({"N": 64}, OK), ({"G": 8}, OK), ({"softplus": 0, "gate": 0}, OK),
    ({"gate": 0, "z_t": -1}, OK), ({"x_b": 0}, OK),
    ({"dtype": 3}, E_UNSUPPORTED), ({"N": 65}, E_UNSUPPORTED), ({"N": 0}, E_SHAPE), ({"G": 3}, E_SHAPE), ({"G": 0}, E_SHAPE),
    ({"softplus": 2}, E_SHAPE), ({"gate": -1}, E_SHAPE), ({"z_t": -1}, E_SHAPE), ({"B_g": -1}, E_SHAPE), ({"C_t": -8}, E_SHAPE),
    ({"x_t": -1}, E_SHAPE), ({"dt_b": -1}, E_SHAPE), ({"T": 0}, E_SHAPE), ({"B": 0}, E_SHAPE), ({"H": 0}, E_SHAPE),
    ({"T": 2147483647}, E_SHAPE), ({"B": 1 << 20, "H": 4096, "G": 1}, E_SHAPE), ({"B": 2147483647}, E_SHAPE),
    ({"B": 1, "H": 1 << 26, "G": 1, "N": 64}, E_SHAPE), ({"T": 1 << 24, "B": 4, "G": 2}, E_SHAPE),
    ({"T": 2147483000, "H": 2147483640, "G": 1, "B": 2147483647}, E_SHAPE),
])
def test_selective_desc(kw, expect):
    n = ctypes.c_size_t(0)
    for fn in _SEL_SIZES:
        assert getattr(ops._lib(), fn)(ctypes.byref(_selective(**kw)), ctypes.byref(n)) == expect
    if expect == OK:
        for fn in _SEL_SIZES:
            assert getattr(ops._lib(), fn)(ctypes.byref(_selective(**kw)), None) == E_NULL


def test_selective_sizes():
    def size(fn, **kw):
        n = ctypes.c_size_t(0)
        assert getattr(ops._lib(), fn)(ctypes.byref(_selective(**kw)), ctypes.byref(n)) == OK
        return n.value

    # the reserve: a state (N rounded up to 4, 8, 16, 32 or 64) at every 16th step
    assert size(_SEL_SIZES[1]) == 19 * 4 * 8 * 16 * 4 and size(_SEL_SIZES[1], T=16, N=17) == 4 * 8 * 32 * 4
    # one tile of channels over a long time is cut into segments; a few steps are not
    assert size(_SEL_SIZES[0], T=20000) > 0 and size(_SEL_SIZES[0], T=100) == 0
    assert size(_SEL_SIZES[0], T=20000, B=64, H=2048, G=1) == 0


def test_selective_pointers():
    L = ops._lib()
    d = _selective(T=20000)
    sizes = []
    for fn in _SEL_SIZES:
        n = ctypes.c_size_t(0)
        assert getattr(L, fn)(ctypes.byref(d), ctypes.byref(n)) == OK and n.value > 0
        sizes.append(n.value)
    ws, rs, bs = sizes

    def io(**kw):
        v = dict(x=ADDR, dt=ADDR, z=ADDR, Bm=ADDR, Cm=ADDR, A=ADDR, D=ADDR, dt_bias=ADDR, lengths=None, h0=None, y=ADDR,
                 h_n=ADDR)
        v.update(kw)
        return ctypes.byref(gss.RnnSelectiveScanIO(*v.values()))

    def fwd(ptr=ADDR, size=ws, **kw):
        return L.rnn_selective_scan(ctypes.byref(d), io(**kw), ptr, size, None)

    for k in ("x", "dt", "z", "Bm", "Cm", "A", "y"):
        assert fwd(**{k: None}) == E_NULL, k
    for k in ("x", "dt", "z", "Bm", "Cm", "A", "D", "dt_bias", "lengths", "h0", "y", "h_n"):
        assert fwd(**{k: ADDR + 2}) == E_ALIGN, k
    assert fwd(ptr=None) == E_WORKSPACE and fwd(size=ws - 1) == E_WORKSPACE and fwd(ptr=ADDR + 8) == E_ALIGN
    assert L.rnn_selective_scan(ctypes.byref(d), None, ADDR, ws, None) == E_NULL
    assert L.rnn_selective_scan(None, io(), ADDR, ws, None) == E_NULL

    def train(ptr=ADDR, size=rs):
        return L.rnn_selective_scan_train(ctypes.byref(d), io(), ptr, size, ADDR, ws, None)

    assert train(ptr=None) == E_WORKSPACE and train(size=rs - 1) == E_WORKSPACE

    def bwd(ptr=ADDR, size=bs, rptr=ADDR, rsize=rs, **kw):
        v = dict(dy=ADDR, dh_n=None, dx=ADDR, ddt=ADDR, dz=ADDR, dB=ADDR, dC=ADDR, dA=ADDR, dD=ADDR, ddt_bias=ADDR, dh0=ADDR)
        v.update(kw)
        return L.rnn_selective_scan_backward(ctypes.byref(d), io(), ctypes.byref(gss.RnnSelectiveScanGrads(*v.values())), rptr,
                                             rsize, ptr, size, None)

    for k in ("dy", "dx", "ddt", "dz", "dB", "dC", "dA"):
        assert bwd(**{k: None}) == E_NULL, k
    for k in ("dy", "dh_n", "dx", "ddt", "dz", "dB", "dC", "dA", "dD", "ddt_bias", "dh0"):
        assert bwd(**{k: ADDR + 1}) == E_ALIGN, k
    assert bwd(ptr=None) == E_WORKSPACE and bwd(size=bs - 1) == E_WORKSPACE and bwd(rsize=rs - 1) == E_WORKSPACE
    assert L.rnn_selective_scan_backward(ctypes.byref(d), io(), None, ADDR, rs, ADDR, bs, None) == E_NULL
    if not torch.cuda.is_available():
        assert fwd() == E_DEVICE and train() == E_DEVICE and bwd() == E_DEVICE
        assert bwd(dD=None, ddt_bias=None, dh0=None) == E_DEVICE and fwd(D=None, dt_bias=None, h_n=None) == E_DEVICE


def test_selective_python_refusals():
    x, A, B = torch.zeros(4, 2, 8, dtype=torch.float32), torch.zeros(8, 4, dtype=torch.float32), torch.zeros(4, 2, 1, 4, dtype=torch.float32)
    with pytest.raises(ValueError, match="GPU tensor"):
        gss.selective_scan(x, x, A, B, B)
    with pytest.raises(ValueError, match="dimensions"):
        gss.selective_scan(x[0], x, A, B, B)
    with pytest.raises(ValueError, match="must be a tensor"):
        gss.selective_scan(None, x, A, B, B)


# ---------------------------------------------------------------------------
# Gated feed-forward
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["silu", "gelu_tanh", "sigmoid"])
def test_feed_forward_definition(kind):
    rng = np.random.default_rng(7)
    rows, n, F, n_out = 4, 3, 5, 2
    x, w_in, w_out = rng.standard_normal((rows, n)), rng.standard_normal((2 * F, n)), rng.standard_normal((n_out, F))
    r, dy = rng.standard_normal((2, rows, n_out))
    y = oracle.feed_forward(x, w_in, w_out, r, kind)
    t = torch.tensor(x @ w_in[:F].T)
    act = {"silu": torch.nn.functional.silu(t), "sigmoid": torch.sigmoid(t),
           "gelu_tanh": torch.nn.functional.gelu(t, approximate="tanh")}[kind].numpy()
    assert np.allclose(y, (act * (x @ w_in[F:].T)) @ w_out.T + r, atol=1e-12)
    loss = lambda: float((oracle.feed_forward(x, w_in, w_out, r, kind) * dy).sum())  # noqa: E731
    for got, v in zip(oracle.feed_forward_backward(x, w_in, w_out, dy, kind), (x, w_in, w_out)):
        assert np.allclose(got, _differences(loss, v), atol=1e-7)


def test_feed_layout(tmp_path):
    _layouts(tmp_path, ["RnnFeedForwardDesc", "RnnFeedForwardIO", "RnnFeedForwardGrads"])


def _feed(**kw):
    v = dict(dtype=1, activation=1, rows=300, N=64, F=96, N_out=64, aligned=1, x_ld=64, in_ld=64, out_ld=96, residual_ld=64)
    v.update(kw)
    return gss.RnnFeedForwardDesc(*v.values())


_FEED_SIZES = tuple(f"rnn_feed_forward_{k}_bytes" for k in ("workspace", "train_workspace", "backward_workspace", "reserve"))


def _feed_size(fn, **kw):
    n = ctypes.c_size_t(0)
    assert getattr(ops._lib(), fn)(ctypes.byref(_feed(**kw)), ctypes.byref(n)) == OK
    return n.value


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), ({"dtype": 0}, OK), ({"activation": 2}, OK), ({"activation": 3}, OK), ({"aligned": 0}, OK), ({"rows": 1}, OK),
    ({"N": 1, "F": 1, "N_out": 1}, OK), ({"x_ld": 1 << 40}, OK), ({"residual_ld": 0}, OK), ({"rows": 1 << 20}, OK),
    ({"dtype": 2}, E_UNSUPPORTED), ({"activation": 0}, E_UNSUPPORTED), ({"activation": 4}, E_UNSUPPORTED),
    ({"rows": 0}, E_SHAPE), ({"rows": -1}, E_SHAPE), ({"N": 0}, E_SHAPE), ({"F": 0}, E_SHAPE), ({"N_out": 0}, E_SHAPE),
    ({"aligned": 2}, E_SHAPE), ({"x_ld": 63}, E_SHAPE), ({"in_ld": 63}, E_SHAPE), ({"out_ld": 95}, E_SHAPE),
    ({"rows": 1 << 40}, E_SHAPE), ({"F": 2147483647, "out_ld": 1 << 40}, E_SHAPE),
    ({"rows": 1 << 30, "F": 1 << 20, "out_ld": 1 << 20}, E_SHAPE), ({"N": 2147483647, "x_ld": 1 << 40, "in_ld": 1 << 40}, E_SHAPE),
])
def test_feed_desc(kw, expect):
    n = ctypes.c_size_t(0)
    for fn in _FEED_SIZES:
        assert getattr(ops._lib(), fn)(ctypes.byref(_feed(**kw)), ctypes.byref(n)) == expect
        if expect == OK:
            assert getattr(ops._lib(), fn)(ctypes.byref(_feed(**kw)), None) == E_NULL


def test_feed_sizes():
    # the reserve: two fp32 numbers and a hidden value each, F in whole steps of 128 bytes
    assert _feed_size(_FEED_SIZES[3]) == 300 * 128 * (2 * 4 + 2)
    assert _feed_size(_FEED_SIZES[3], dtype=0) == 300 * 96 * 3 * 4
    # few rows keep the hidden values alone, whatever the alignment
    assert _feed_size(_FEED_SIZES[0], rows=64) == _feed_size(_FEED_SIZES[0], rows=64, aligned=0, x_ld=65) == 64 * 128 * 2
    # operands whose rows are not whole 16 bytes are copied
    for kw, more in (({"x_ld": 65}, 300 * 64 * 2), ({"in_ld": 65}, 2 * 96 * 64 * 2), ({"out_ld": 97}, 64 * 96 * 2),
                     ({"aligned": 0}, (300 * 64 + 2 * 96 * 64 + 64 * 96) * 2)):
        for fn in _FEED_SIZES[:2]:
            assert _feed_size(fn, **kw) == _feed_size(fn) + more, kw
    assert _feed_size(_FEED_SIZES[2], aligned=0) > _feed_size(_FEED_SIZES[2])


def test_training_of_few_rows_copies_nothing_forward():
    """Nor does it lay out tiles of 128 rows for them: no workspace but the
    divided sums' (none here)."""
    for rows in (1, 32, 64):
        assert _feed_size(_FEED_SIZES[1], rows=rows) == _feed_size(_FEED_SIZES[1], rows=rows, aligned=0, x_ld=65, in_ld=65) == 0
    assert _feed_size(_FEED_SIZES[1], rows=65, x_ld=65) > _feed_size(_FEED_SIZES[1], rows=65)
    big = dict(N=2048, N_out=2048, x_ld=2048, in_ld=2048, residual_ld=2048, aligned=0)
    few, many = dict(big, F=8192, out_ld=8192, rows=32), dict(big, F=8192, out_ld=8192, rows=33)
    assert _feed_size(_FEED_SIZES[1], **few) < 1 << 24 < _feed_size(_FEED_SIZES[1], **many)     # the weights' copies
    assert _feed_size(_FEED_SIZES[1], **dict(big, F=4096, out_ld=4096, rows=64)) < 1 << 24


def test_feed_pointers():
    L = ops._lib()
    d = _feed(aligned=0)
    ws, ts, bs, rs = (_feed_size(fn, aligned=0) for fn in _FEED_SIZES)

    def io(**kw):
        v = dict(x=ADDR, w_in=ADDR, w_out=ADDR, residual=ADDR, y=ADDR)
        v.update(kw)
        return ctypes.byref(gss.RnnFeedForwardIO(*v.values()))

    def fwd(ptr=ADDR, size=ws, desc=d, **kw):
        return L.rnn_feed_forward(ctypes.byref(desc), io(**kw), ptr, size, None)

    for k in ("x", "w_in", "w_out", "y"):
        assert fwd(**{k: None}) == E_NULL, k
    for k in ("x", "w_in", "w_out", "residual", "y"):
        assert fwd(**{k: ADDR + 1}) == E_ALIGN, k
    for k in ("x", "w_in", "w_out"):       # promised to be multiples of 16 bytes
        assert fwd(desc=_feed(), **{k: ADDR + 2}) == E_ALIGN, k
    assert fwd(desc=_feed(residual_ld=63)) == E_SHAPE
    assert fwd(ptr=None) == E_WORKSPACE and fwd(size=ws - 1) == E_WORKSPACE and fwd(ptr=ADDR + 8) == E_ALIGN
    assert L.rnn_feed_forward(ctypes.byref(d), None, ADDR, ws, None) == E_NULL
    assert L.rnn_feed_forward(None, io(), ADDR, ws, None) == E_NULL

    def train(ptr=ADDR, size=rs, wptr=ADDR, wsize=ts):
        return L.rnn_feed_forward_train(ctypes.byref(d), io(), ptr, size, wptr, wsize, None)

    assert train(ptr=None) == E_WORKSPACE and train(size=rs - 1) == E_WORKSPACE and train(wsize=ts - 1) == E_WORKSPACE

    def bwd(ptr=ADDR, size=bs, rsize=rs, desc=d, **kw):
        v = dict(dy=ADDR, dx=ADDR, dw_in=ADDR, dw_out=ADDR)
        v.update(kw)
        return L.rnn_feed_forward_backward(ctypes.byref(desc), io(), ctypes.byref(gss.RnnFeedForwardGrads(*v.values())), ADDR,
                                           rsize, ptr, size, None)

    for k in ("dy", "dx", "dw_in", "dw_out"):
        assert bwd(**{k: None}) == E_NULL, k
        assert bwd(**{k: ADDR + 1}) == E_ALIGN, k
    assert bwd(desc=_feed(), dy=ADDR + 2) == E_ALIGN
    assert bwd(ptr=None) == E_WORKSPACE and bwd(size=bs - 1) == E_WORKSPACE and bwd(rsize=rs - 1) == E_WORKSPACE
    assert L.rnn_feed_forward_backward(ctypes.byref(d), io(), None, ADDR, rs, ADDR, bs, None) == E_NULL
    if not torch.cuda.is_available():
        assert fwd() == E_DEVICE and fwd(residual=None) == E_DEVICE and train() == E_DEVICE and bwd() == E_DEVICE


def test_feed_python_refusals():
    x, w_in, w_out = torch.zeros(4, 8, dtype=torch.float32), torch.zeros(32, 8, dtype=torch.float32), torch.zeros(8, 16, dtype=torch.float32)
    with pytest.raises(ValueError, match="GPU tensor"):
        gss.feed_forward(x, w_in, w_out)
    with pytest.raises(ValueError, match="activation"):
        gss.feed_forward(x, w_in, w_out, activation=None)
    with pytest.raises(ValueError, match="tensor of at least one"):
        gss.feed_forward(None, w_in, w_out)
