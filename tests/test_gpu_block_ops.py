"""Layer norm and the gated scan on the GPU against the float64 definitions:
types, odd sizes, strides, alignment, lengths from none to whole, gradients."""

import numpy as np
import pytest
import torch

import oracle
from block_util import assert_near, draw, f64, shifted, strided
from gpu_util import log

pytestmark = pytest.mark.gpu

gss = pytest.importorskip("gru_sequence_scan_amd")

DTYPES = [torch.float32, torch.bfloat16]
IDS = ["f32", "bf16"]
PLACE = {"dense": lambda t: t.cuda(), "strided": strided, "shifted": shifted}


# ---------------------------------------------------------------------------
# Layer norm
# ---------------------------------------------------------------------------

NORM_CASES = [  # rows, N: every row team and its edges, odd widths, few and many rows
    (1, 1), (3, 2), (5, 16), (70, 127), (33, 128), (9, 129), (50, 200), (7, 512), (6, 513), (65, 1000), (5, 1024), (3, 2047),
    (4, 2048), (3, 2056), (2, 4097), (3, 8192), (2, 16377), (2, 16384), (5003, 24),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("rows,n", NORM_CASES)
@pytest.mark.parametrize("place", list(PLACE))
def test_layer_norm(rows, n, dtype, place):
    log(f"layer_norm rows {rows} n {n} {dtype} {place}")
    rng = np.random.default_rng(rows * 7 + n)
    put = PLACE[place]
    x, r = draw(rng, (rows, n), dtype, 1.0, 3.0), draw(rng, (rows, n), dtype, 2.0)
    w, b = draw(rng, (n,), dtype, 0.3, 1.0), draw(rng, (n,), dtype, 0.3)
    dy, ds = draw(rng, (rows, n), dtype), draw(rng, (rows, n), dtype)
    dense = shifted if place == "shifted" else (lambda t: t.cuda())
    # rstd of a short row can be large: errors of x (2^-24 of its size) are
    # multiplied by it, in y and, once more, in dx
    (y, total), ctx = gss.layer_norm_train(put(x), dense(w), dense(b), residual=put(r))
    s = (x.double() + r.double()).to(dtype)
    assert torch.equal(total.cpu(), (x.float() + r.float()).to(dtype))
    yr, _, rstd = oracle.layer_norm(f64(s), f64(w), f64(b))
    amp = (2.0 ** -22 * np.abs(f64(s)).max(-1, keepdims=True) * rstd[:, None])
    assert_near(y, yr, dtype, "y", amp * 4)
    dx, dw, db = gss.layer_norm_backward(ctx, dense(dy), dense(ds))
    dxr, dwr, dbr = oracle.layer_norm_backward(f64(s), f64(w), f64(dy), f64(ds))
    size = np.abs(f64(dy)).max() * np.abs(f64(w)).max()
    assert_near(dx, dxr, dtype, "dx", amp * 16 * size * rstd[:, None])
    # columns are sums over the rows: fp32 error of each term
    col = np.abs(f64(dy)).max() * amp.max() * rows + 2.0 ** -22 * rows ** 0.5
    assert_near(dw, dwr, torch.float32, "dw", col)
    assert_near(db, dbr, torch.float32, "db", 2.0 ** -20 * rows ** 0.5)
    plain = gss.layer_norm(put(x), dense(w), dense(b), residual=put(r))
    assert torch.equal(plain[0], y) and torch.equal(plain[1], total)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_layer_norm_without_parameters_or_residual(dtype):
    rng = np.random.default_rng(5)
    x, dy = draw(rng, (3, 11, 96), dtype), draw(rng, (3, 11, 96), dtype)
    y = gss.layer_norm(x.cuda())
    (yt, total), ctx = gss.layer_norm_train(x.cuda())
    assert total is None and torch.equal(y, yt) and y.shape == x.shape
    flat = f64(x).reshape(33, 96)
    assert_near(y.reshape(33, 96), oracle.layer_norm(flat)[0], dtype, "y")
    dx, dw, db = gss.layer_norm_backward(ctx, dy.cuda())
    assert dw is None and db is None
    assert_near(dx.reshape(33, 96), oracle.layer_norm_backward(flat, None, f64(dy).reshape(33, 96))[0], dtype, "dx")
    for name, kw in (("weight", {"weight": x[0, 0].cuda()}), ("bias", {"bias": x[0, 0].cuda()})):
        y = gss.layer_norm(x.cuda(), **kw)
        ref = oracle.layer_norm(flat, *[f64(kw[k]) if k in kw else None for k in ("weight", "bias")])[0]
        assert_near(y.reshape(33, 96), ref, dtype, name)
        _, ctx = gss.layer_norm_train(x.cuda(), **kw)
        assert gss.layer_norm_backward(ctx, dy.cuda())[1].shape == (96,)


def test_layer_norm_extreme_rows():
    """A constant row (variance 0), a row with a large mean, values near the
    type's largest, and rows with NaN or infinity, which stay in their row."""
    x = torch.randn(6, 64, generator=torch.Generator().manual_seed(3), dtype=torch.float32)
    x[1] = 7.0
    x[2] += 4096.0
    x[3] *= 1e18
    x[4, 5] = float("nan")
    x[5, 9] = float("inf")
    y = gss.layer_norm(x.cuda()).cpu()
    ref = oracle.layer_norm(f64(x[:4]))[0]
    assert np.all(f64(y[1]) == 0.0)
    assert_near(y[0], ref[0], torch.float32, "plain row")
    assert_near(y[2], ref[2], torch.float32, "large mean", 4096.0 * 2.0 ** -22)
    assert_near(y[3], ref[3], torch.float32, "large values")
    assert torch.isnan(y[4]).all() and torch.isnan(y[5]).any() and torch.isfinite(y[:4]).all()


# ---------------------------------------------------------------------------
# Gated scan
# ---------------------------------------------------------------------------

SCAN_CASES = [  # T, B, H: one step, chunk edges (128), several chunks, odd widths
    (1, 1, 1), (1, 5, 64), (2, 3, 8), (8, 2, 100), (31, 2, 4), (127, 2, 7), (128, 1, 68), (129, 3, 12), (257, 2, 65),
    (700, 3, 36), (1500, 1, 9), (3000, 1, 4),
]


def _scan_case(T, B, H, dtype, gate, seed):
    rng = np.random.default_rng(seed)
    x, dy = draw(rng, (T, B, H), dtype), draw(rng, (T, B, H), dtype)
    f = draw(rng, (T, B, H), dtype, 2.0, 2.0)
    i = draw(rng, (T, B, H), dtype) if gate else None
    h0, dhn = draw(rng, (B, H), torch.float32), draw(rng, (B, H), torch.float32)
    return x, f, i, h0, dy, dhn


def _check_scan(x, f, i, h0, dy, dhn, lengths, reverse, put, dev_lengths, what, keep=None):
    dtype = x.dtype
    T, B, H = x.shape
    L = np.full(B, T) if lengths is None else np.asarray(lengths)
    past = np.arange(T)[:, None] >= L[None]
    g = [None if t is None else put(t) for t in (x, f, i)]
    (y, hn), ctx = gss.gated_scan_train(*g, h0=None if h0 is None else h0.cuda(), lengths=dev_lengths, reverse=reverse)
    yr, hr, _ = oracle.gated_scan(f64(x), f64(f), f64(i), f64(h0), lengths, reverse)
    assert_near(y, yr, dtype, what + " y")
    assert_near(hn, hr, torch.float32, what + " h_n")
    assert (f64(y)[past] == 0).all()
    dense = shifted if put is shifted else (lambda t: t.cuda())
    dx, df, di, dh0 = gss.gated_scan_backward(ctx, dense(dy), None if dhn is None else dhn.cuda())
    rx, rf, ri, rh = oracle.gated_scan_backward(f64(x), f64(f), f64(i), f64(dy), f64(dhn), f64(h0), lengths, reverse)
    assert_near(dx, rx, dtype, what + " dx")
    assert_near(df, rf, dtype, what + " df")
    assert_near(dh0, rh, torch.float32, what + " dh0")
    if i is not None:
        assert_near(di, ri, dtype, what + " di")
    else:
        assert di is None
    for t in (dx, df):
        assert (f64(t)[past] == 0).all()
    y2, hn2 = gss.gated_scan(*g, h0=None if h0 is None else h0.cuda(), lengths=dev_lengths, reverse=reverse)
    assert torch.equal(y2, y) and torch.equal(hn2, hn)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("gate", [False, True], ids=["coupled", "gate"])
@pytest.mark.parametrize("T,B,H", SCAN_CASES)
def test_gated_scan(T, B, H, gate, dtype):
    log(f"gated_scan T {T} B {B} H {H} gate {gate} {dtype}")
    case = _scan_case(T, B, H, dtype, gate, T * 131 + H)
    reverse = (T + B) % 2 == 1
    _check_scan(*case, None, reverse, PLACE["dense"], None, "dense")
    _check_scan(*case[:3], None, case[4], None, None, not reverse, PLACE["dense"], None, "no states")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("reverse", [False, True], ids=["forward", "reverse"])
@pytest.mark.parametrize("place", ["strided", "shifted"])
def test_gated_scan_ragged(place, reverse, dtype):
    """Ragged rows, rows without steps among them; NaN past each row's end
    must not matter; strided and unaligned inputs."""
    T, lengths = 300, [300, 0, 1, 127, 128, 129, 255, 256, 257, 0]
    for gate, H in ((False, 72), (True, 40)):
        log(f"gated_scan ragged {place} reverse {reverse} gate {gate} {dtype}")
        x, f, i, h0, dy, dhn = _scan_case(T, len(lengths), H, dtype, gate, 17 + gate)
        dev = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        clean = (x, f, i, h0, dy, dhn)

        def dirty(t):
            out = PLACE[place](t)
            if t.dim() == 3 and t.shape[0] == T:
                for b, L in enumerate(lengths):
                    out[L:, b] = float("nan")
            return out

        _check_scan(*clean, lengths, reverse, dirty, dev, place)
        # host lengths, and lengths out of range, which clamp
        a = gss.gated_scan(x.cuda(), f.cuda(), None if i is None else i.cuda(), lengths=lengths, reverse=reverse)
        wild = torch.tensor([v if v not in (0, T) else (-5 if v == 0 else T + 9) for v in lengths], dtype=torch.int64)
        b = gss.gated_scan(x.cuda(), f.cuda(), None if i is None else i.cuda(), lengths=wild.cuda(), reverse=reverse)
        c = gss.gated_scan(x.cuda(), f.cuda(), None if i is None else i.cuda(), lengths=wild.int().cuda(), reverse=reverse)
        for p, q, r in zip(a, b, c):
            assert torch.equal(p, q) and torch.equal(p, r)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("reverse", [False, True], ids=["forward", "reverse"])
def test_gated_scan_ragged_segments(reverse, dtype):
    """Few channels over a long time: segments of the time axis, with rows
    that end before, at and inside a segment and a chunk."""
    T, lengths = 1700, [1700, 0, 1, 255, 256, 257, 1024, 1300, 1536]
    for gate, H, place in ((False, 8, "dense"), (True, 5, "strided")):
        log(f"gated_scan segments reverse {reverse} gate {gate} {dtype}")
        case = _scan_case(T, len(lengths), H, dtype, gate, 23 + gate)

        def dirty(t):
            out = PLACE[place](t)
            if t.dim() == 3 and t.shape[0] == T:
                for b, L in enumerate(lengths):
                    out[L:, b] = float("nan")
            return out

        _check_scan(*case, lengths, reverse, dirty, torch.tensor(lengths, dtype=torch.int32, device="cuda"), place)


def test_gated_scan_nan_in_unread_gradients():
    """What lies past a row's end in dy is not read either."""
    T, lengths = 140, [3, 140, 0]
    x, f, i, h0, dy, dhn = _scan_case(T, 3, 16, torch.float32, True, 4)
    (y, hn), ctx = gss.gated_scan_train(x.cuda(), f.cuda(), i.cuda(), h0=h0.cuda(), lengths=lengths)
    ref = gss.gated_scan_backward(ctx, dy.cuda(), dhn.cuda())
    for b, L in enumerate(lengths):
        dy[L:, b] = float("nan")
    got = gss.gated_scan_backward(ctx, dy.cuda(), dhn.cuda())
    for p, q in zip(ref, got):
        assert torch.equal(p, q)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_gated_scan_saturated_gates(dtype):
    """Gates far into both tails, the types' largest values and infinities:
    a and 1 - a stay exact 0 and 1, and no 0 * inf arises."""
    big = torch.finfo(dtype).max
    vals = [0.0, 40.0, -40.0, 90.0, -90.0, 200.0, -200.0, big, -big, float("inf"), -float("inf")]
    f = torch.tensor(vals, dtype=dtype)[None, None].repeat(6, 2, 1)
    rng = np.random.default_rng(9)
    x, dy = draw(rng, f.shape, dtype), draw(rng, f.shape, dtype)
    i = torch.flip(f, (2,)).contiguous()
    with np.errstate(over="ignore"):
        for gate in (None, i):
            _check_scan(x, f, gate, draw(rng, f.shape[1:], torch.float32), dy, None, None, False, PLACE["dense"], None, "tails")


@pytest.mark.parametrize("reverse", [False, True])
def test_gated_scan_in_pieces(reverse):
    """Running a sequence in pieces, one step at a time at the end, is the
    whole run: the state that passes between the calls is fp32."""
    x, f, i, h0, _, _ = (None if t is None else t.cuda() for t in _scan_case(200, 3, 24, torch.bfloat16, True, 8))
    y, hn = gss.gated_scan(x, f, i, h0=h0, reverse=reverse)
    h, out = h0, []
    cuts = [(0, 150), (150, 197), (197, 198), (198, 199), (199, 200)]
    for lo, hi in (reversed(cuts) if reverse else cuts):
        part, h = gss.gated_scan(x[lo:hi], f[lo:hi], i[lo:hi], h0=h, reverse=reverse)
        out.append(part)
    whole = torch.cat(out[::-1] if reverse else out)
    assert_near(whole, f64(y), torch.bfloat16, "y")
    assert_near(h, f64(hn), torch.float32, "h_n")


def test_block_ops_capture_and_streams():
    """Calls on a side stream, and captured in a graph that is replayed on new
    inputs, give what eager calls give."""
    x, f, _, h0, dy, _ = (None if t is None else t.cuda() for t in _scan_case(300, 4, 64, torch.bfloat16, False, 12))
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")

    def step():
        n, nctx = gss.layer_norm_train(x, w)
        (y, hn), ctx = gss.gated_scan_train(n[0], f, h0=h0)
        dx, df, _, dh0 = gss.gated_scan_backward(ctx, dy)
        return (y, hn, df, dh0) + gss.layer_norm_backward(nctx, dx)[:2]

    eager = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    for a, b in zip(eager, other):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(3):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(k)).to(x.dtype))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(step(), held):
            assert torch.equal(a, b)


def test_layer_norm_more_rows_than_a_launch():
    """More rows than one launch has teams for: the last rows are normalised
    too, and with the same values as the same rows alone."""
    rows = (1 << 27) + 5003          # 2^23 workgroups of 16 rows, and some
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB of free device memory")
    x = torch.zeros(rows, 8, dtype=torch.bfloat16, device="cuda")
    tail = draw(np.random.default_rng(2), (6000, 8), torch.bfloat16).cuda()
    x[-6000:] = tail
    y = gss.layer_norm(x)
    assert torch.equal(y[-6000:], gss.layer_norm(tail))
    assert not y[:6000].any()
