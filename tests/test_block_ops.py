"""The decoder block's operators on the CPU: the float64 definitions against
torch and against differences, and the refusals of the C entry points and of
the Python calls, which all come before anything touches a device."""

import ctypes

import numpy as np
import pytest
import torch

import oracle

gss = pytest.importorskip("gru_sequence_scan_amd")
ops = gss.block_ops

OK, E_NULL, E_SHAPE, E_UNSUPPORTED, E_LENGTHS, E_WORKSPACE, E_ALIGN, E_DEVICE = 0, -1, -2, -3, -4, -5, -6, -7
ADDR = 4096


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


# -- the definitions --

def test_layer_norm_definition():
    rng = np.random.default_rng(1)
    s, w, b, dy, ds = rng.standard_normal((5, 7)), *rng.standard_normal((2, 7)), *rng.standard_normal((2, 5, 7))
    y = oracle.layer_norm(s, w, b)[0]
    ref = torch.nn.functional.layer_norm(torch.tensor(s), (7,), torch.tensor(w), torch.tensor(b))
    assert np.allclose(y, ref.numpy(), atol=1e-12)
    loss = lambda: float((oracle.layer_norm(s, w, b)[0] * dy).sum() + (s * ds).sum())  # noqa: E731
    dx, dw, db = oracle.layer_norm_backward(s, w, dy, ds)
    for got, v in ((dx, s), (dw, w), (db, b)):
        assert np.allclose(got, _differences(loss, v), atol=1e-7)


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("reverse", [False, True])
def test_gated_scan_definition(gate, reverse):
    rng = np.random.default_rng(2)
    T, B, H = 4, 3, 2
    x, f, i, dy = rng.standard_normal((4, T, B, H))
    h0, dhn = rng.standard_normal((2, B, H))
    i = i if gate else None
    lens = [4, 0, 2]

    def loss():
        y, hn, _ = oracle.gated_scan(x, f, i, h0, lens, reverse)
        return float((y * dy).sum() + (hn * dhn).sum())

    dx, df, di, dh0 = oracle.gated_scan_backward(x, f, i, dy, dhn, h0, lens, reverse)
    for got, v in ((dx, x), (df, f), (di, i), (dh0, h0)):
        if v is not None:
            assert np.allclose(got, _differences(loss, v), atol=1e-8)
    # a row without steps passes its state and its gradient through
    assert np.array_equal(oracle.gated_scan(x, f, i, h0, lens, reverse)[1][1], h0[1])
    assert np.array_equal(dh0[1], dhn[1])


def test_cross_attention_definition():
    rng = np.random.default_rng(3)
    Tq, Tk, B, heads, kv, D = 3, 5, 3, 4, 2, 3
    q, do = rng.standard_normal((2, Tq, B, heads, D))
    k, v = rng.standard_normal((2, Tk, B, kv, D))
    lens = [5, 0, 2]
    o = oracle.cross_attention(q, k, v, lens)
    t = [torch.tensor(x) for x in (q, k, v)]
    for b, n in ((0, 5), (2, 2)):
        ref = torch.nn.functional.scaled_dot_product_attention(
            t[0][:, b].transpose(0, 1), t[1][:n, b].transpose(0, 1).repeat_interleave(2, 0),
            t[2][:n, b].transpose(0, 1).repeat_interleave(2, 0))
        assert np.allclose(o[:, b], ref.transpose(0, 1).numpy(), atol=1e-12)
    assert (o[:, 1] == 0).all()
    loss = lambda: float((oracle.cross_attention(q, k, v, lens, 0.7) * do).sum())  # noqa: E731
    for got, x in zip(oracle.cross_attention_backward(q, k, v, do, lens, 0.7), (q, k, v)):
        assert np.allclose(got, _differences(loss, x), atol=1e-8)
    # the bounds scale with the unit and cover a rounded probability's effect
    small, large = (oracle.attention_bounds(q, k, v, do, lens, 0.7, u) for u in (1e-3, 2e-3))
    for a, b in zip(small, large):
        assert np.allclose(2 * a, b) and (a >= 0).all()


# -- layouts of the ctypes mirrors --

def test_ctypes_layout_matches_c(tmp_path):
    import os
    import subprocess
    names = ["RnnNormDesc", "RnnGatedScanDesc", "RnnGatedScanIO", "RnnGatedScanGrads",
             "RnnAttentionDesc", "RnnAttentionIO", "RnnAttentionGrads"]
    lines = [f'  printf("%zu", sizeof({n}));' + "".join(f' printf(" %zu", offsetof({n}, {f[0]}));'
                                                       for f in getattr(gss, n)._fields_) + ' printf("\\n");' for n in names]
    src = tmp_path / "layout.c"
    src.write_text("#include <stdio.h>\n#include <stddef.h>\n#include \"rnn.h\"\nint main(void) {\n" + "\n".join(lines) +
                   "\n  return 0;\n}\n")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["gcc", "-std=c99", "-I", include, str(src), "-o", str(tmp_path / "layout")], check=True)
    out = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True).stdout.splitlines()
    for n, line in zip(names, out):
        t = getattr(gss, n)
        assert [int(v) for v in line.split()] == [ctypes.sizeof(t)] + [getattr(t, f[0]).offset for f in t._fields_]


# -- refusals of the C entry points --

def _norm(**kw):
    v = dict(dtype=0, N=8, rows=4, x_ld=8, residual_ld=8, eps=1e-5, reserved=0)
    v.update(kw)
    return gss.RnnNormDesc(*v.values())


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), ({"dtype": 1}, OK), ({"N": 16384, "x_ld": 16384}, OK), ({"eps": 0.0}, OK),
    ({"dtype": 2}, E_UNSUPPORTED), ({"N": 16385, "x_ld": 20000}, E_UNSUPPORTED),
    ({"N": 0}, E_SHAPE), ({"rows": 0}, E_SHAPE), ({"rows": 1 << 40}, E_SHAPE), ({"x_ld": 7}, E_SHAPE),
    ({"eps": -1.0}, E_SHAPE), ({"eps": float("nan")}, E_SHAPE), ({"eps": float("inf")}, E_SHAPE), ({"reserved": 1}, E_SHAPE),
])
def test_norm_desc(kw, expect):
    n = ctypes.c_size_t(0)
    assert ops._lib().rnn_layer_norm_backward_workspace_bytes(ctypes.byref(_norm(**kw)), ctypes.byref(n)) == expect
    if expect == OK:
        assert n.value > 0


def test_norm_pointers():
    L = ops._lib()
    d = ctypes.byref(_norm())

    def fwd(x=ADDR, r=None, w=ADDR, b=ADDR, y=ADDR, s=None, stats=None, desc=d):
        return L.rnn_layer_norm(desc, x, r, w, b, y, s, stats, None)

    assert fwd(desc=None) == E_NULL and fwd(x=None) == E_NULL and fwd(y=None) == E_NULL
    assert fwd(r=ADDR) == E_NULL                       # a residual needs somewhere for the sum
    assert fwd(r=ADDR, s=ADDR, desc=ctypes.byref(_norm(residual_ld=7))) == E_SHAPE
    for k in ("x", "w", "b", "y", "stats"):
        assert fwd(**{k: ADDR + 2}) == E_ALIGN, k
    n = ctypes.c_size_t(0)
    assert L.rnn_layer_norm_backward_workspace_bytes(d, ctypes.byref(n)) == OK
    assert L.rnn_layer_norm_backward_workspace_bytes(d, None) == E_NULL

    def bwd(s=ADDR, stats=ADDR, dy=ADDR, ds=None, dx=ADDR, dw=ADDR, db=ADDR, ws=ADDR, size=n.value):
        return L.rnn_layer_norm_backward(d, s, ADDR, stats, dy, ds, dx, dw, db, ws, size, None)

    for k in ("s", "stats", "dy", "dx", "dw", "db"):
        assert bwd(**{k: None}) == E_NULL, k
        assert bwd(**{k: ADDR + 1}) == E_ALIGN, k
    assert bwd(ws=None) == E_WORKSPACE and bwd(size=n.value - 1) == E_WORKSPACE and bwd(ws=ADDR + 4) == E_ALIGN
    if not torch.cuda.is_available():
        assert fwd() == E_DEVICE and bwd() == E_DEVICE
        assert bwd(dw=None, db=None, ws=None, size=0) == E_DEVICE   # no parameters, no workspace


def _scan(**kw):
    v = dict(dtype=0, T=300, B=4, H=8, reverse=0, input_gate=0, x_t=32, x_b=8, f_t=32, f_b=8, i_t=32, i_b=8)
    v.update(kw)
    return gss.RnnGatedScanDesc(*v.values())


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), ({"dtype": 1}, OK), ({"reverse": 1, "input_gate": 1}, OK), ({"f_b": 0}, OK),
    ({"dtype": -1}, E_UNSUPPORTED), ({"T": 0}, E_SHAPE), ({"B": 0}, E_SHAPE), ({"H": -1}, E_SHAPE),
    ({"reverse": 2}, E_SHAPE), ({"reverse": -1}, E_SHAPE), ({"input_gate": 3}, E_SHAPE),
    ({"x_t": -1}, E_SHAPE), ({"f_b": -8}, E_SHAPE), ({"input_gate": 1, "i_t": -1}, E_SHAPE), ({"i_t": -1}, OK),
    ({"T": 2147483647}, E_SHAPE), ({"B": 1 << 20, "H": 4096}, E_SHAPE),
    ({"T": 2000000000, "B": 2000000000}, E_SHAPE), ({"B": 2147483647, "H": 2147483647}, E_SHAPE),
])
def test_scan_desc(kw, expect):
    n = ctypes.c_size_t(0)
    for fn in ("rnn_gated_scan_workspace_bytes", "rnn_gated_scan_reserve_bytes"):
        assert getattr(ops._lib(), fn)(ctypes.byref(_scan(**kw)), ctypes.byref(n)) == expect
    if expect == OK:
        assert n.value >= 3 * 4 * 8 * 4      # the reserve: a state at each of three chunks
        # few channels over a long time are cut into segments, whose maps
        # take a workspace; one chunk of steps needs none
        for T, some in ((20000, True), (128, False)):
            assert ops._lib().rnn_gated_scan_workspace_bytes(ctypes.byref(_scan(**dict(kw, T=T))), ctypes.byref(n)) == OK
            assert (n.value > 0) == some


def test_scan_pointers():
    L = ops._lib()
    d = _scan(input_gate=1, T=20000)
    n, r = ctypes.c_size_t(0), ctypes.c_size_t(0)
    assert L.rnn_gated_scan_workspace_bytes(ctypes.byref(d), ctypes.byref(n)) == OK
    assert L.rnn_gated_scan_reserve_bytes(ctypes.byref(d), ctypes.byref(r)) == OK

    def io(**kw):
        v = dict(x=ADDR, f=ADDR, i=ADDR, lengths=None, h0=None, y=ADDR, h_n=ADDR)
        v.update(kw)
        return gss.RnnGatedScanIO(*v.values())

    def fwd(ws=ADDR, size=n.value, **kw):
        return L.rnn_gated_scan(ctypes.byref(d), ctypes.byref(io(**kw)), ws, size, None)

    assert L.rnn_gated_scan(None, ctypes.byref(io()), ADDR, n.value, None) == E_NULL
    assert L.rnn_gated_scan(ctypes.byref(d), None, ADDR, n.value, None) == E_NULL
    for k in ("x", "f", "i", "y"):
        assert fwd(**{k: None}) == E_NULL and fwd(**{k: ADDR + 2}) == E_ALIGN, k
    for k in ("lengths", "h0", "h_n"):
        assert fwd(**{k: ADDR + 1}) == E_ALIGN, k
    assert fwd(ws=None) == E_WORKSPACE and fwd(size=n.value - 1) == E_WORKSPACE and fwd(ws=ADDR + 8) == E_ALIGN
    assert L.rnn_gated_scan_train(ctypes.byref(d), ctypes.byref(io()), None, 0, ADDR, n.value, None) == E_WORKSPACE

    def bwd(reserve=ADDR, rsize=r.value, ws=ADDR, **kw):
        v = dict(dy=ADDR, dh_n=None, dx=ADDR, df=ADDR, di=ADDR, dh0=None)
        v.update(kw)
        return L.rnn_gated_scan_backward(ctypes.byref(d), ctypes.byref(io(y=None, h_n=None)),
                                         ctypes.byref(gss.RnnGatedScanGrads(*v.values())), reserve, rsize, ws, n.value, None)

    for k in ("dy", "dx", "df", "di"):
        assert bwd(**{k: None}) == E_NULL and bwd(**{k: ADDR + 1}) == E_ALIGN, k
    assert bwd(dh0=ADDR + 2) == E_ALIGN and bwd(dh_n=ADDR + 2) == E_ALIGN
    assert bwd(reserve=None) == E_WORKSPACE and bwd(rsize=r.value - 1) == E_WORKSPACE and bwd(ws=None) == E_WORKSPACE
    if not torch.cuda.is_available():
        assert fwd() == E_DEVICE and bwd() == E_DEVICE


def _attend(**kw):
    v = dict(dtype=0, B=2, Tq=5, Tk=70, heads=4, kv_heads=2, D=8, scale=0.5, q_t=64, q_b=32, q_h=8, k_t=32, k_b=16, k_h=8,
             v_t=32, v_b=16, v_h=8)
    v.update(kw)
    return gss.RnnAttentionDesc(*v.values())


@pytest.mark.parametrize("kw,expect", [
    ({}, OK), ({"dtype": 1}, OK), ({"D": 128}, OK), ({"D": 1}, OK), ({"heads": 2}, OK), ({"k_b": 0}, OK),
    ({"dtype": 7}, E_UNSUPPORTED), ({"D": 129}, E_UNSUPPORTED),
    ({"B": 0}, E_SHAPE), ({"Tq": 0}, E_SHAPE), ({"Tk": -3}, E_SHAPE), ({"heads": 3}, E_SHAPE), ({"heads": 0}, E_SHAPE),
    ({"kv_heads": 0}, E_SHAPE), ({"heads": 1}, E_SHAPE), ({"D": 0}, E_SHAPE), ({"scale": float("nan")}, E_SHAPE),
    ({"scale": float("inf")}, E_SHAPE), ({"q_t": -1}, E_SHAPE), ({"k_h": -8}, E_SHAPE), ({"v_b": -1}, E_SHAPE),
    ({"B": 1 << 20, "Tq": 1}, OK), ({"B": 1 << 20, "Tk": 1 << 12}, E_SHAPE), ({"B": 1 << 20, "Tq": 1 << 12}, E_SHAPE),
    ({"Tk": 2147483647}, E_SHAPE), ({"Tq": 2000000000}, E_SHAPE), ({"B": 2000000000, "kv_heads": 4}, E_SHAPE),
])
def test_attention_desc(kw, expect):
    n = ctypes.c_size_t(0)
    for fn in ("rnn_cross_attention_workspace_bytes", "rnn_cross_attention_reserve_bytes",
               "rnn_cross_attention_backward_workspace_bytes"):
        assert getattr(ops._lib(), fn)(ctypes.byref(_attend(**kw)), ctypes.byref(n)) == expect
    if expect == OK:   # one fp32 value per query row; the reserve has o's rest too in bf16
        d = _attend(**kw)
        rows = d.B * d.heads * d.Tq
        assert n.value == rows * 4
        assert ops._lib().rnn_cross_attention_reserve_bytes(ctypes.byref(d), ctypes.byref(n)) == OK
        assert n.value == rows * 4 + (rows * d.D * 2 if d.dtype == 1 else 0)


def test_attention_split_workspace():
    """A call with few query rows splits the keys over workgroups, and its
    workspace holds a partial row per split; one that fills the device does
    not."""
    n = ctypes.c_size_t(0)
    fn = ops._lib().rnn_cross_attention_workspace_bytes
    assert fn(ctypes.byref(_attend(B=1, Tq=1, Tk=32768)), ctypes.byref(n)) == OK
    assert n.value >= 8 * 4 * (8 + 2) * 4
    assert fn(ctypes.byref(_attend(B=64, Tq=1000, Tk=1000, heads=8, kv_heads=8)), ctypes.byref(n)) == OK and n.value == 0


def test_attention_pointers():
    L = ops._lib()
    d = _attend(B=1, Tq=1, Tk=32768)
    n, r = ctypes.c_size_t(0), ctypes.c_size_t(0)
    assert L.rnn_cross_attention_workspace_bytes(ctypes.byref(d), ctypes.byref(n)) == OK
    assert L.rnn_cross_attention_reserve_bytes(ctypes.byref(d), ctypes.byref(r)) == OK

    def io(**kw):
        v = dict(q=ADDR, k=ADDR, v=ADDR, lengths=None, o=ADDR)
        v.update(kw)
        return gss.RnnAttentionIO(*v.values())

    def fwd(ws=ADDR, size=n.value, **kw):
        return L.rnn_cross_attention(ctypes.byref(d), ctypes.byref(io(**kw)), ws, size, None)

    assert L.rnn_cross_attention(None, ctypes.byref(io()), ADDR, n.value, None) == E_NULL
    assert L.rnn_cross_attention(ctypes.byref(d), None, ADDR, n.value, None) == E_NULL
    for k in ("q", "k", "v", "o"):
        assert fwd(**{k: None}) == E_NULL and fwd(**{k: ADDR + 2}) == E_ALIGN, k
    assert fwd(lengths=ADDR + 2) == E_ALIGN
    assert fwd(ws=None) == E_WORKSPACE and fwd(size=n.value - 1) == E_WORKSPACE and fwd(ws=ADDR + 8) == E_ALIGN
    assert L.rnn_cross_attention_train(ctypes.byref(d), ctypes.byref(io()), ADDR, r.value - 1, ADDR, n.value,
                                       None) == E_WORKSPACE

    def bwd(reserve=ADDR, ws=ADDR, size=r.value, **kw):
        v = dict(d_o=ADDR, dq=ADDR, dk=ADDR, dv=ADDR)
        v.update(kw)
        return L.rnn_cross_attention_backward(ctypes.byref(d), ctypes.byref(io()), ctypes.byref(gss.RnnAttentionGrads(*v.values())),
                                              reserve, r.value, ws, size, None)

    for k in ("d_o", "dq", "dk", "dv"):
        assert bwd(**{k: None}) == E_NULL and bwd(**{k: ADDR + 1}) == E_ALIGN, k
    assert bwd(reserve=None) == E_WORKSPACE and bwd(ws=None) == E_WORKSPACE and bwd(ws=ADDR + 4) == E_ALIGN
    if not torch.cuda.is_available():
        assert fwd() == E_DEVICE and bwd() == E_DEVICE


# -- refusals of the Python calls --

def test_python_refusals():
    x = torch.zeros(4, 3, 8)
    for call in (lambda: gss.layer_norm(x), lambda: gss.gated_scan(x, x), lambda: gss.gated_scan([1.0], x),
                 lambda: gss.cross_attention(x[None], x[None], x[None])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError, match="float32, bfloat16"):
        gss.layer_norm(x.half())
    with pytest.raises(ValueError, match="3 dimensions"):
        gss.gated_scan(x[0], x[0])
    with pytest.raises(ValueError, match="batch of 3"):
        ops._lengths([1, 2], 3, 4, torch.device("cpu"))
    for bad in ([0, 1, 5], [-1, 2, 3]):
        with pytest.raises(ValueError, match=r"\[0, 4\]"):
            ops._lengths(bad, 3, 4, torch.device("cpu"))


def test_rows_of_strided_tensors():
    t = torch.arange(2 * 3 * 4 * 8.0).reshape(2, 3, 4, 8)
    for v, ld in ((t, 8), (t[:, :, 0], 32), (t[..., 2:6], 8), (t[0, 0, 0], 8), (t[:, 1, 1:2], 96)):
        r, got = ops._rows(v)
        assert r is v and got == ld
    for v in (t[:, :2], t.transpose(0, 1), t[..., ::2], t[:1, :1, :1].expand(5, 1, 1, 8)):
        r, got = ops._rows(v)
        assert torch.equal(r, v) and r.is_contiguous() and got == v.shape[-1]
