"""The gated feed-forward on the GPU against its float64 definition: types,
activations, rows from one to many, odd sizes, strides, alignment, tiles of
both sizes, split sums, gradients, a captured graph."""

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
KINDS = ["silu", "gelu_tanh", "sigmoid"]
BF16_HALF_ULP = 2.0 ** -8


def _case(rows, n, F, n_out, dtype, seed):
    rng = np.random.default_rng(seed)
    return {"x": draw(rng, (rows, n), dtype), "w_in": draw(rng, (2 * F, n), dtype, n ** -0.5),
            "w_out": draw(rng, (n_out, F), dtype, F ** -0.5), "r": draw(rng, (rows, n_out), dtype, 2.0),
            "dy": draw(rng, (rows, n_out), dtype)}


def _bounds(x, w_in, w_out, dy, kind, act):
    """What one rounding of h, dg and du (2^-8 of each in bf16) moves y, dx,
    dw_in and dw_out by at most. numpy or torch arrays."""
    F = w_out.shape[1]
    u = x @ w_in[F:].T
    a, slope = act(x @ w_in[:F].T, kind)
    h, dh = a * u, dy @ w_out
    dg, du = abs(dh * u * slope), abs(dh * a)
    ax, ai, ao, ady = abs(x), abs(w_in), abs(w_out), abs(dy)
    cat = np.concatenate if isinstance(x, np.ndarray) else torch.cat
    dp = cat([dg, du], 1)
    return [BF16_HALF_ULP * v for v in (abs(h) @ ao.T, dp @ ai, dp.T @ ax, ady.T @ abs(h))]


def _rms_off(got, ref):
    """The error's 2-norm over the result's."""
    d = got.double() - ref
    return float(d.norm() / ref.norm())


def _check(c, kind, place="dense", residual=True, what=""):
    put = PLACE[place]
    dense = shifted if place == "shifted" else (lambda t: t.cuda())
    dtype = c["x"].dtype
    x, w_in, w_out, dy = put(c["x"]), put(c["w_in"]), put(c["w_out"]), dense(c["dy"])
    r = put(c["r"]) if residual else None
    y, ctx = gss.feed_forward_train(x, w_in, w_out, residual=r, activation=kind)
    got = (y,) + gss.feed_forward_backward(ctx, dy)
    v = {k: f64(t) for k, t in c.items()}
    ref = (oracle.feed_forward(v["x"], v["w_in"], v["w_out"], v["r"] if residual else None, kind),) + \
        oracle.feed_forward_backward(v["x"], v["w_in"], v["w_out"], v["dy"], kind)
    from oracle.state_block import activation
    extra = [0.0] * 4 if dtype == torch.float32 else _bounds(v["x"], v["w_in"], v["w_out"], v["dy"], kind, activation)
    for g, t, b, name in zip(got, ref, extra, ("y", "dx", "dw_in", "dw_out")):
        assert_near(g, t, dtype, f"{what} {name}", b)
    # serving: the same operator without what training keeps (few rows: kernels of their own)
    y2 = gss.feed_forward(x, w_in, w_out, residual=r, activation=kind)
    if c["x"].shape[0] > 64:
        assert torch.equal(y2, y)
    else:
        assert_near(y2, ref[0], dtype, f"{what} y served", extra[0])
    return got


SIZES = [  # rows, N, F, N_out: single rows, edges of the tiles (16, 128) and steps (32, 64), widths not of 16 bytes
    (1, 1, 1, 1), (1, 64, 32, 8), (2, 7, 5, 3), (15, 24, 40, 24), (16, 72, 64, 17), (17, 100, 130, 100), (33, 8, 8, 520),
    (63, 65, 33, 64), (64, 128, 264, 128), (65, 64, 64, 64), (128, 520, 96, 128), (129, 136, 200, 264), (257, 33, 129, 31),
    (300, 512, 1000, 512), (700, 40, 70, 300),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("rows,n,F,n_out", SIZES)
def test_feed_forward(rows, n, F, n_out, dtype):
    log(f"feed_forward rows {rows} n {n} F {F} n_out {n_out} {dtype}")
    c = _case(rows, n, F, n_out, dtype, rows + n + F)
    _check(c, KINDS[(rows + F) % 3], residual=(n + F) % 2 == 0, what="dense")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("place", ["strided", "shifted"])
@pytest.mark.parametrize("rows", [3, 200])
def test_places(rows, place, kind, dtype):
    log(f"feed_forward {place} {kind} rows {rows} {dtype}")
    _check(_case(rows, 72, 136, 88, dtype, 3), kind, place, what=place)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("n,F", [(64, 96), (63, 97), (33, 6), (3, 2), (72, 39), (5, 260)])
@pytest.mark.parametrize("rows", [1, 17, 64])
def test_few_rows_at_any_address(rows, n, F, dtype):
    """Few rows read each operand 16 bytes at a time wherever it begins: every
    one alone off its alignment, rows of any length, with what lies around
    them not a number, and the same bits as from aligned tensors."""
    log(f"feed_forward any address rows {rows} n {n} F {F} {dtype}")
    c = _case(rows, n, F, 24, dtype, rows + n * F)

    def off(t, by):
        wide = torch.full((t.shape[0] * (t.shape[1] + 5) + 16,), float("nan"), dtype=dtype, device="cuda")
        out = wide[by:by + t.shape[0] * (t.shape[1] + 5)].view(t.shape[0], -1)[:, :t.shape[1]]
        out.copy_(t)
        return out

    x, w_in, w_out = (c[k].cuda() for k in ("x", "w_in", "w_out"))
    y = gss.feed_forward(x, w_in, w_out)
    v = {k: f64(t) for k, t in c.items()}
    from oracle.state_block import activation
    extra = 0.0 if dtype == torch.float32 else _bounds(v["x"], v["w_in"], v["w_out"], v["dy"], "silu", activation)[0]
    assert_near(y, oracle.feed_forward(v["x"], v["w_in"], v["w_out"]), dtype, "y", extra)
    for by in (0, 1, 2, 3, 7):
        for args in ((off(x, by), w_in, w_out), (x, off(w_in, by), w_out), (x, w_in, off(w_out, by)),
                     (off(x, by), off(w_in, by + 1), off(w_out, by + 2))):
            assert torch.equal(gss.feed_forward(*args), y), by


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("rows,n,F,n_out", [(1, 264, 1030, 96), (17, 33, 70, 520), (32, 520, 2056, 130), (33, 200, 1000, 64),
                                            (64, 130, 97, 7), (40, 2056, 4104, 2056)])
def test_training_of_few_rows(rows, n, F, n_out, dtype):
    """Up to 64 rows (up to 32 with large weights: the last case is in tiles)
    training takes serving's kernels forward and keeps the projections."""
    log(f"feed_forward few rows training {rows} n {n} F {F} n_out {n_out} {dtype}")
    c = _case(rows, n, F, n_out, dtype, rows)
    y = _check(c, "gelu_tanh", what="few")[0]
    served = gss.feed_forward(*(c[k].cuda() for k in ("x", "w_in", "w_out")), residual=c["r"].cuda(), activation="gelu_tanh")
    if n < 2000:
        assert torch.equal(y, served)


@pytest.mark.parametrize("which", ["x", "w_in", "w_out", "dy"])
def test_one_operand_off_its_alignment_copies_no_other(which, monkeypatch):
    """What is not an operand's copy stays as it was in the workspace: with x
    alone off its alignment no weight is copied, and so on."""
    rows, n, F, n_out = 200, 72, 136, 88
    c = _case(rows, n, F, n_out, torch.bfloat16, 12)
    put = {k: (shifted if k == which else lambda t: t.cuda())(c[k]) for k in ("x", "w_in", "w_out", "dy")}
    sizes = {"x": rows * n * 2, "w_in": 2 * F * n * 2, "w_out": n_out * F * 2, "dy": rows * n_out * 2}
    made = []

    def buffer(size, device):
        made.append(torch.full((size,), 0xA5, dtype=torch.uint8, device=device))
        return made[-1]

    monkeypatch.setattr(gss.state_block_ops, "_buffer", buffer)
    y, ctx = gss.feed_forward_train(put["x"], put["w_in"], put["w_out"])
    got = (y,) + gss.feed_forward_backward(ctx, put["dy"])
    forward, _, backward = made
    monkeypatch.undo()
    aligned = {k: c[k].cuda() for k in put}
    y, ctx = gss.feed_forward_train(aligned["x"], aligned["w_in"], aligned["w_out"])
    assert all(torch.equal(a, b) for a, b in zip(got, (y,) + gss.feed_forward_backward(ctx, aligned["dy"])))
    for ws, room in ((forward, ("x", "w_in", "w_out")), (backward, ("x", "w_in", "w_out", "dy"))):
        if ws is forward and which == "dy":
            continue                                      # nothing is off its alignment there
        assert int((ws == 0xA5).sum()) >= sum(sizes[k] for k in room if k != which)


def _torch_act(g, kind):
    if kind == "gelu_tanh":
        c = (2 / np.pi) ** 0.5
        t = torch.tanh(c * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    s = torch.sigmoid(g)
    return (s, s * torch.sigmoid(-g)) if kind == "sigmoid" else (g * s, s + g * s * torch.sigmoid(-g))


@pytest.mark.parametrize("dtype,rows,n,F,n_out", [
    (torch.bfloat16, 16389, 520, 2056, 520), (torch.bfloat16, 5000, 2048, 2816, 1000), (torch.bfloat16, 20011, 129, 700, 264),
    (torch.float32, 9001, 516, 1368, 512), (torch.float32, 3000, 1000, 2052, 1028),
], ids=str)
def test_many_rows(dtype, rows, n, F, n_out):
    """Large tiles with edges, several tiles a workgroup, sums over many rows
    split and joined; the definition in float64 on the GPU."""
    log(f"feed_forward many rows {rows} n {n} F {F} n_out {n_out} {dtype}")
    c = {k: v.cuda() for k, v in _case(rows, n, F, n_out, dtype, 9).items()}
    y, ctx = gss.feed_forward_train(c["x"], c["w_in"], c["w_out"], residual=c["r"])
    got = (y,) + gss.feed_forward_backward(ctx, c["dy"])
    x, w_in, w_out, dy = (c[k].double() for k in ("x", "w_in", "w_out", "dy"))
    act, slope = _torch_act(x @ w_in[:F].T, "silu")
    u = x @ w_in[F:].T
    dh = dy @ w_out
    dp = torch.cat([dh * u * slope, dh * act], 1)
    ref = ((act * u) @ w_out.T + c["r"].double(), dp @ w_in, dp.T @ x, dy.T @ (act * u))
    bounds = _bounds(x, w_in, w_out, dy, "silu", _torch_act)
    # a rounding's mean square is at most (2^-8)^2 / 3 of the value's: two of them
    most = 2.0 ** 0.5 * BF16_HALF_ULP / 3.0 ** 0.5 if dtype == torch.bfloat16 else 4e-6
    for g, t, b, name in zip(got, ref, bounds, ("y", "dx", "dw_in", "dw_out")):
        assert _rms_off(g, t) < most, name
        limit = 1e-4 * t.abs() + 1e-5 * t.abs().max()
        if dtype == torch.bfloat16:
            limit = limit + b
            limit = limit + BF16_HALF_ULP * (t.abs() + limit)
        assert bool(((g.double() - t).abs() <= limit).all()), name
    assert torch.equal(gss.feed_forward(c["x"], c["w_in"], c["w_out"], residual=c["r"]), y)


@pytest.mark.parametrize("rows", [5, 150])
def test_not_a_number_stays_in_its_row(rows):
    """A row that is not a number, or infinite, changes no other row."""
    c = {k: v.cuda() for k, v in _case(rows, 40, 72, 24, torch.bfloat16, 1).items()}
    y = gss.feed_forward(c["x"], c["w_in"], c["w_out"])
    x = c["x"].clone()
    x[2] = float("nan")
    x[4, 3] = float("inf")
    y2, ctx = gss.feed_forward_train(x, c["w_in"], c["w_out"])
    served = gss.feed_forward(x, c["w_in"], c["w_out"])
    keep = torch.ones(rows, dtype=torch.bool)
    keep[2] = keep[4] = False
    assert torch.equal(served[keep], y[keep]) and torch.isnan(y2[2]).all() and not torch.isfinite(y2[4]).any()
    clean = gss.feed_forward_train(c["x"], c["w_in"], c["w_out"])[1]
    assert torch.equal(gss.feed_forward_backward(ctx, c["dy"])[0][keep], gss.feed_forward_backward(clean, c["dy"])[0][keep])


def test_large_gates():
    """act(g) and its slope where the exponential overflows or vanishes."""
    c = _case(70, 16, 32, 16, torch.float32, 6)
    c["w_in"][:32] *= 60.0
    for kind in KINDS:
        _check(c, kind, what=kind)


@pytest.mark.parametrize("kind", KINDS)
def test_gates_whose_square_no_fp32_number_holds(kind):
    """Gates of 1e20 either way: the slope is 0 or 1 (the sigmoid's 0), and
    what is not a number stays that in its gradient."""
    rows, n, F = 70, 16, 32
    c = _case(rows, n, F, 16, torch.float32, 8)
    c["x"][:, 0] = 1.0
    c["w_in"][:16] = 0.0
    c["w_in"][:8, 0], c["w_in"][8:16, 0] = 1e20, -1e20
    c["dy"] *= 1e-20                                      # so that dw_in's parts are of one size
    c["r"] *= 1e20
    _check(c, kind, what=kind)
    x = c["x"].cuda()
    x[3, 1] = float("nan")
    ctx = gss.feed_forward_train(x, c["w_in"].cuda(), c["w_out"].cuda(), activation=kind)[1]
    assert torch.isnan(gss.feed_forward_backward(ctx, c["dy"].cuda())[0][3]).all()


def test_leading_dimensions():
    c = _case(6 * 5, 24, 40, 16, torch.float32, 2)
    x, w_in, w_out, r = (c[k].cuda() for k in ("x", "w_in", "w_out", "r"))
    y = gss.feed_forward(x, w_in, w_out, residual=r)
    y3 = gss.feed_forward(x.view(6, 5, 24), w_in, w_out, residual=r.view(6, 5, 16))
    assert y3.shape == (6, 5, 16) and torch.equal(y3.view(30, 16), y)
    one = gss.feed_forward(x[0], w_in, w_out, residual=r[0])
    assert one.shape == (16,) and torch.equal(one, y[0])
    t = x.view(6, 5, 24).transpose(0, 1)
    assert torch.equal(gss.feed_forward(t, w_in, w_out), gss.feed_forward(x, w_in, w_out).view(6, 5, 16).transpose(0, 1))


@pytest.mark.parametrize("rows", [7, 400])
def test_captured_replayed_and_on_another_stream(rows):
    c = {k: v.cuda() for k, v in _case(rows, 128, 192, 128, torch.bfloat16, 4).items()}

    def run():
        y, ctx = gss.feed_forward_train(c["x"], c["w_in"], c["w_out"], residual=c["r"])
        return (y, gss.feed_forward(c["x"], c["w_in"], c["w_out"])) + gss.feed_forward_backward(ctx, c["dy"])

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for _ in range(4):
        c["x"].copy_(torch.randn_like(c["x"]))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, run()):
            assert torch.equal(a, b)


def test_refusals():
    c = {k: v.cuda() for k, v in _case(5, 8, 16, 8, torch.float32, 1).items()}
    gss.feed_forward(c["x"], c["w_in"], c["w_out"])
    for args, match in (((c["x"], c["w_in"][:31], c["w_out"]), "w_in"), ((c["x"], c["w_in"].bfloat16(), c["w_out"]), "w_in"),
                        ((c["x"], c["w_in"], c["w_out"][:, :15]), "w_in"), ((c["x"], c["w_in"], c["w_out"].cpu()), "w_out")):
        with pytest.raises(ValueError, match=match):
            gss.feed_forward(*args)
    with pytest.raises(ValueError, match="residual"):
        gss.feed_forward(c["x"], c["w_in"], c["w_out"], residual=c["r"][:4])
    with pytest.raises(gss.RnnError):
        gss.feed_forward(c["x"][:0], c["w_in"], c["w_out"])
    y, ctx = gss.feed_forward_train(c["x"], c["w_in"], c["w_out"])
    with pytest.raises(ValueError, match="dy"):
        gss.feed_forward_backward(ctx, c["dy"][:4])
