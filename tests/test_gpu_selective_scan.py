"""The selective scan on the GPU against its float64 definition: types, state
lengths, groups, odd sizes, strides, alignment, lengths from none to whole,
cut time, gradients, token by token, large and zero steps, a captured graph."""

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
NAMES = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0")


def _case(T, B, H, N, G, dtype, seed):
    rng = np.random.default_rng(seed)
    c = {k: draw(rng, (T, B, H), dtype) for k in ("x", "z", "dy")}
    c["dt"] = draw(rng, (T, B, H), dtype, 0.7, -2.0)
    c["B"], c["C"] = draw(rng, (T, B, G, N), dtype), draw(rng, (T, B, G, N), dtype)
    c["A"] = -torch.exp(draw(rng, (H, N), torch.float32, 0.5))
    c["D"], c["dt_bias"] = draw(rng, (H,), torch.float32), draw(rng, (H,), torch.float32, 0.5)
    c["h0"], c["dh_n"] = draw(rng, (B, H, N), torch.float32), draw(rng, (B, H, N), torch.float32)
    return c


def _run(c, put, dense, lengths, softplus=True):
    opt = {k: None if c[k] is None else dense(c[k]) for k in ("dt_bias", "h0")}
    z = None if c["z"] is None else put(c["z"])
    args = (put(c["x"]), put(c["dt"]), dense(c["A"]), put(c["B"]), put(c["C"]), None if c["D"] is None else dense(c["D"]))
    (y, hn), ctx = gss.selective_scan_train(*args, z=z, softplus=softplus, lengths=lengths, **opt)
    g = gss.selective_scan_backward(ctx, dense(c["dy"]), None if c["dh_n"] is None else dense(c["dh_n"]))
    y2, hn2 = gss.selective_scan(*args, z=z, softplus=softplus, lengths=lengths, **opt)
    assert torch.equal(y2, y) and torch.equal(hn2, hn)
    return y, hn, g


def _reference(c, lengths, softplus=True):
    v = {k: f64(t) for k, t in c.items()}
    kw = dict(z=v["z"], dt_bias=v["dt_bias"], soft=softplus, h0=v["h0"], lengths=lengths)
    y, hn, _ = oracle.selective_scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], **kw)
    return y, hn, oracle.selective_scan_backward(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], v["dy"], v["dh_n"], **kw)


def _check(c, lengths, place="dense", softplus=True, what=""):
    put = PLACE[place]
    dense = shifted if place == "shifted" else (lambda t: t.cuda())
    dtype = c["x"].dtype
    dev = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    y, hn, g = _run(c, put, dense, dev, softplus)
    yr, hr, gr = _reference(c, lengths, softplus)
    assert_near(y, yr, dtype, what + " y")
    assert_near(hn, hr, torch.float32, what + " h_n")
    for k in NAMES:
        if k in ("D", "z", "dt_bias") and c[k] is None:
            assert g[k] is None
            continue
        assert_near(g[k], gr[k], dtype if k in ("x", "dt", "z", "B", "C") else torch.float32, f"{what} d{k}")
    if lengths is not None:
        past = np.arange(c["x"].shape[0])[:, None] >= np.asarray(lengths)[None]
        for t in (y, g["x"], g["dt"], g["B"], g["C"]) + (() if g["z"] is None else (g["z"],)):
            assert (f64(t)[past] == 0).all()
    return y, hn, g


CASES = [  # T, B, H, N, G: one step, tile edges (16, 32 steps, 64 channels), every state length, odd widths
    (1, 1, 1, 1, 1), (1, 5, 64, 16, 1), (2, 3, 8, 3, 2), (8, 2, 72, 16, 1), (9, 2, 24, 4, 1), (16, 1, 64, 16, 2),
    (17, 2, 65, 5, 1), (31, 1, 128, 8, 1), (33, 3, 40, 12, 4), (48, 1, 200, 16, 1), (65, 2, 7, 16, 1), (20, 1, 8, 17, 1),
    (40, 2, 68, 32, 1), (25, 1, 12, 33, 1), (35, 2, 70, 64, 2), (100, 2, 130, 16, 2),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T,B,H,N,G", CASES)
def test_selective_scan(T, B, H, N, G, dtype):
    log(f"selective_scan T {T} B {B} H {H} N {N} G {G} {dtype}")
    c = _case(T, B, H, N, G, dtype, T * 31 + H + N)
    _check(c, None, what="all")
    for k in ("z", "D", "dt_bias", "h0", "dh_n"):
        c[k] = None
    c["dt"] = torch.nn.functional.softplus(c["dt"].float()).to(dtype)
    _check(c, None, softplus=False, what="least")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("N", [4, 16, 20, 64])
@pytest.mark.parametrize("place", ["dense", "strided", "shifted"])
def test_ragged(place, N, dtype):
    """Lengths of none, one, around the tiles' edges; what lies past a row's
    end is NaN and changes nothing."""
    T, B, H, G = 50, 9, 48, 2
    lengths = [0, 1, 15, 16, 17, 32, 33, 49, 50]
    log(f"selective_scan ragged {place} N {N} {dtype}")
    c = _case(T, B, H, N, G, dtype, 5)
    past = torch.arange(T)[:, None] >= torch.tensor(lengths)[None]
    for k in ("x", "dt", "z", "dy", "B", "C"):
        c[k][past] = 0.0
    y, hn, g = _check(c, lengths, place, what=place)
    for k in ("x", "dt", "z", "dy", "B", "C"):
        c[k] = c[k].clone()
        c[k][past] = float("nan")
    dense = shifted if place == "shifted" else (lambda t: t.cuda())
    y2, hn2, g2 = _run(c, PLACE[place], dense, torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    assert torch.equal(y, y2) and torch.equal(hn, hn2)
    for k in NAMES:
        assert torch.equal(g[k], g2[k]), k


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T,B,H,N,lengths", [(1000, 1, 8, 16, None), (700, 3, 20, 8, [700, 130, 0]), (513, 2, 4, 64, [64, 512])])
def test_cut_time(T, B, H, N, lengths, dtype):
    """Few channels over a long time: its segments run at once."""
    log(f"selective_scan cut T {T} B {B} H {H} N {N} {dtype}")
    c = _case(T, B, H, N, 1, dtype, 17)
    d = gss.RnnSelectiveScanDesc(0, T, B, H, N, 1, 1, 1, *([0] * 12))
    assert gss.block_ops._bytes("rnn_selective_scan_workspace_bytes", d) > 0
    _check(c, lengths, what="cut")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("T,B,H,N,lengths", [(2100, 1, 8, 16, None), (1500, 2, 20, 8, [1500, 1025]), (1100, 1, 70, 32, None),
                                             (1153, 3, 5, 64, [1153, 1088, 1089])])
def test_many_segments(T, B, H, N, lengths, dtype):
    """More segments than the launch between them takes at once, rows that end
    at and beside a segment's edge."""
    log(f"selective_scan segments T {T} B {B} H {H} N {N} {dtype}")
    _check(_case(T, B, H, N, 1, dtype, 23), lengths, what="segments")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("N,G", [(16, 1), (9, 2)])
def test_token_by_token(N, G, dtype):
    """A prompt of 40 steps at once, and step by step with the state carried."""
    T, B, H = 40, 3, 72
    c = {k: v.cuda() for k, v in _case(T, B, H, N, G, dtype, 8).items()}
    kw = dict(dt_bias=c["dt_bias"])
    whole, hn = gss.selective_scan(c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"], z=c["z"], h0=c["h0"], **kw)
    h, out = c["h0"], []
    for t in range(T):
        s = slice(t, t + 1)
        y, h = gss.selective_scan(c["x"][s], c["dt"][s], c["A"], c["B"][s], c["C"][s], c["D"], z=c["z"][s], h0=h, **kw)
        out.append(y)
    assert_near(torch.cat(out), f64(whole), dtype, "y", 0.0 if dtype == torch.float32 else float(whole.abs().max()) * 2.0 ** -8)
    assert_near(h, f64(hn), torch.float32, "h_n")


@pytest.mark.parametrize("soft", [True, False])
def test_steps_from_nothing_to_huge(soft):
    """Steps that are zero keep the state, huge ones forget it; tiny softplus
    steps keep their own relative accuracy."""
    T, B, H, N = 24, 1, 16, 4
    c = _case(T, B, H, N, 1, torch.float32, 21)
    raw = torch.linspace(-80, 80, T, dtype=torch.float32)[:, None, None].expand(T, B, H).contiguous() if soft else \
        torch.tensor([0.0] * 8 + [1e4] * 8 + [1e-6] * 8, dtype=torch.float32)[:, None, None].expand(T, B, H).contiguous()
    c["dt"], c["dt_bias"], c["z"], c["D"] = raw, None, None, None
    # large steps make large inputs: compare where the state is of order one
    c["x"] = c["x"] / (1 + raw.clamp(min=0))
    y, hn, g = _check(c, None, softplus=soft, what="steps")
    if soft:  # the first step is exp(-80) long: y's input part alone, from a zero state
        c["h0"] = None
        one = {k: (v[:1] if k in ("x", "dt", "B", "C", "dy") and v is not None else v) for k, v in c.items()}
        one["dh_n"] = None
        y, _, _ = _run(one, PLACE["dense"], PLACE["dense"], None)
        ref, _, _ = _reference(one, None)
        assert np.abs(f64(y) - ref).max() <= 2e-5 * np.abs(ref).max() and np.abs(ref).max() < 1e-30


def test_growing_states_and_positive_A():
    c = _case(30, 2, 24, 8, 1, torch.float32, 4)
    c["A"] = 0.3 * c["A"].abs()
    _check(c, None, what="positive A")


def _growing(T, H, N, grow):
    """A channel that grows by exp(128) over each 64 steps of `grow`, hardly
    elsewhere, from a state of zero."""
    c = _case(T, 1, H, N, 1, torch.float32, 29)
    c["A"] = 0.9 + 0.1 * torch.rand((H, N), generator=torch.Generator().manual_seed(3), dtype=torch.float32)
    c["dt"] = torch.full((T, 1, H), 1e-3, dtype=torch.float32)
    c["dt"][grow] = 2.2
    c["x"][grow] = 0.0
    c["dt_bias"] = c["h0"] = c["dh_n"] = None
    d = gss.RnnSelectiveScanDesc(0, T, 1, H, N, 1, 0, 1, *([0] * 12))
    assert gss.block_ops._bytes("rnn_selective_scan_workspace_bytes", d) > 0    # cut
    return c


@pytest.mark.parametrize("H,N", [(8, 16), (20, 5)])
def test_cut_time_keeps_a_state_of_zero_over_any_growth(H, N):
    """A segment's factor that no fp32 number holds leaves a state of zero at
    zero, as the walk step by step does, forward and backward."""
    T = 1000
    c = _growing(T, H, N, slice(0, 700))
    args = [c[k].cuda() for k in ("x", "dt", "A", "B", "C", "D")]
    y, hn = gss.selective_scan(*args, z=c["z"].cuda(), softplus=False)
    v = {k: f64(t) for k, t in c.items()}
    yr, hr, _ = oracle.selective_scan(v["x"], v["dt"], v["A"], v["B"], v["C"], v["D"], z=v["z"], soft=False)
    assert_near(y, yr, torch.float32, "y")
    assert_near(hn, hr, torch.float32, "h_n")
    # backward the same from the other end: no state, and gradients before the growth alone
    c = _growing(T, H, N, slice(300, T))
    c["x"][:] = 0.0
    c["dy"][300:] = 0.0
    y, hn, g = _run(c, PLACE["dense"], PLACE["dense"], None, softplus=False)
    yr, hr, gr = _reference(c, None, softplus=False)
    assert not hn.any() and not hr.any()
    for k in NAMES:
        if k != "dt_bias":
            assert_near(g[k], gr[k], torch.float32, f"d{k}")
    assert float(g["x"].abs().max()) > 1.0


def test_cut_time_grows_a_small_state_past_one_factor():
    """From 2^-100 by exp(104), about 2^150, in one segment: that factor is no fp32 number, the state is."""
    T, H, N = 640, 8, 16
    c = _growing(T, H, N, slice(64, 128))
    c["A"][:] = 1.0
    c["dt"][64:128] = 104.0 / 64
    c["dt"][:64] = c["dt"][128:] = 0.0
    c["x"][:] = 0.0
    c["h0"] = torch.full((1, H, N), 2.0 ** -100, dtype=torch.float32)
    _, hn = gss.selective_scan(*[c[k].cuda() for k in ("x", "dt", "A", "B", "C")], h0=c["h0"].cuda(), softplus=False)
    # the steps and their sum are exact; log2(e), its product with the sum, a third and the product with that are
    # rounded: 104 (2^-25 + 2^-24 + 2^-25 + 2^-24), and three times an exponential (2^-23) and a product: 1.9e-5 in all
    assert np.abs(f64(hn) / (2.0 ** -100 * np.exp(104.0)) - 1).max() < 2e-5


def test_gradient_of_shared_inputs():
    """B and C of one group gather the gradients of all its channels, however
    many tiles of 64 they make."""
    c = _case(18, 2, 520, 16, 1, torch.float32, 6)
    _check(c, [18, 7], what="shared")


def test_deterministic_and_on_another_stream():
    c = _case(200, 4, 256, 16, 1, torch.bfloat16, 2)
    put = PLACE["dense"]
    y, hn, g = _run(c, put, put, None)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        y2, hn2, g2 = _run(c, put, put, None)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(hn, hn2) and all(torch.equal(g[k], g2[k]) for k in NAMES)


@pytest.mark.parametrize("T,H", [(1, 96), (70, 96), (1200, 8)])
def test_captured_and_replayed(T, H):
    c = {k: v.cuda() for k, v in _case(T, 3, H, 16, 1, torch.bfloat16, 12).items()}
    lens = torch.tensor([T, 0, (T + 1) // 2], dtype=torch.int32, device="cuda")

    def run():
        (y, hn), ctx = gss.selective_scan_train(c["x"], c["dt"], c["A"], c["B"], c["C"], c["D"], z=c["z"],
                                                dt_bias=c["dt_bias"], h0=c["h0"], lengths=lens)
        g = gss.selective_scan_backward(ctx, c["dy"], c["dh_n"])
        return [y, hn] + [g[k] for k in NAMES]

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for k in range(4):
        c["x"].copy_(torch.randn_like(c["x"]))
        lens.copy_(torch.tensor([T - k % 2, k % 2, (T + 1) // 2], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, run()):
            assert torch.equal(got, want)


def test_refusals():
    c = {k: v.cuda() for k, v in _case(5, 2, 8, 4, 2, torch.float32, 1).items()}
    args = [c[k] for k in ("x", "dt", "A", "B", "C", "D")]
    gss.selective_scan(*args)
    for i, bad, match in ((1, c["dt"][:, :, :4], "dt"), (2, c["A"][:, :3], "A"), (4, c["C"][:, :, :1], "C"),
                          (5, c["D"][:4], "D"), (1, c["dt"].bfloat16(), "dt"), (2, c["A"].double(), "A")):
        with pytest.raises(ValueError, match=match):
            gss.selective_scan(*(args[:i] + [bad] + args[i + 1:]))
    with pytest.raises(ValueError, match="h0"):
        gss.selective_scan(*args, h0=c["h0"][:1])
    with pytest.raises(ValueError, match="lengths"):
        gss.selective_scan(*args, lengths=[6, 1])
    big = torch.zeros(5, 2, 2, 65, device="cuda", dtype=torch.float32)
    with pytest.raises(gss.RnnError):
        gss.selective_scan(c["x"], c["dt"], torch.zeros(8, 65, device="cuda", dtype=torch.float32), big, big)
    with pytest.raises(gss.RnnError):      # 8 channels in 3 groups
        gss.selective_scan(c["x"], c["dt"], c["A"], *(torch.zeros(5, 2, 3, 4, device="cuda", dtype=torch.float32),) * 2)
