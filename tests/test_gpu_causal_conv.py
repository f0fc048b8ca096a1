"""The causal convolution on the GPU against its float64 definition: types,
filter lengths, odd sizes, strides, alignment, lengths from none to whole,
states, gradients, token by token, a captured graph."""

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


def _case(T, B, C, W, dtype, seed):
    rng = np.random.default_rng(seed)
    x, dy = draw(rng, (T, B, C), dtype), draw(rng, (T, B, C), dtype)
    w, b = draw(rng, (C, W), dtype, W ** -0.5), draw(rng, (C,), dtype, 0.3)
    state, ds = draw(rng, (W - 1, B, C), dtype), draw(rng, (W - 1, B, C), dtype)
    return x, w, b, state, dy, ds


def _check(case, lengths, activation, put, what, bias=True, states=True, dev_lengths=None):
    x, w, b, state, dy, ds = case
    dtype, (T, B, C) = x.dtype, x.shape
    b, state, ds = (b if bias else None), (state if states else None), (ds if states else None)
    dense = shifted if put is shifted else (lambda t: None if t is None else t.cuda())
    place = lambda t: None if t is None else dense(t)  # noqa: E731
    if dev_lengths is None and lengths is not None:
        dev_lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    (y, last), ctx = gss.causal_conv_train(put(x), dense(w), place(b), state=place(state), lengths=dev_lengths,
                                           activation=activation)
    yr, lr = oracle.causal_conv(f64(x), f64(w), f64(b), f64(state), lengths, activation)
    assert_near(y, yr, dtype, what + " y")
    assert np.array_equal(f64(last), lr), what + " state_n"     # copied
    dx, dw, db, dstate = gss.causal_conv_backward(ctx, dense(dy), place(ds))
    rx, rw, rb, rs = oracle.causal_conv_backward(f64(x), f64(w), f64(b), f64(dy), f64(ds), f64(state), lengths, activation)
    assert_near(dx, rx, dtype, what + " dx")
    assert_near(dstate, rs, dtype, what + " dstate")
    # sums over all tokens: each term carries a few fp32 roundings
    size = float(np.abs(f64(dy)).max() * np.abs(f64(x)).max()) * 2.0 ** -22 * (T * B) ** 0.5
    assert_near(dw, rw, torch.float32, what + " dweight", size)
    assert (db is None) == (not bias)
    if bias:
        assert_near(db, rb, torch.float32, what + " dbias", size)
    if lengths is not None:
        past = np.arange(T)[:, None] >= np.asarray(lengths)[None]
        assert (f64(y)[past] == 0).all() and (f64(dx)[past] == 0).all()
    y2, last2 = gss.causal_conv(put(x), dense(w), place(b), state=place(state), lengths=dev_lengths, activation=activation)
    assert torch.equal(y2, y) and torch.equal(last2, last)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("W", [2, 3, 4, 5, 7, 8])
@pytest.mark.parametrize("T,B,C", [(1, 1, 1), (1, 5, 64), (3, 2, 8), (8, 3, 40), (9, 2, 100), (16, 1, 520), (17, 3, 24),
                                   (33, 2, 7), (100, 4, 264)])
def test_causal_conv(T, B, C, W, dtype):
    log(f"causal_conv T {T} B {B} C {C} W {W} {dtype}")
    case = _case(T, B, C, W, dtype, T * 31 + C + W)
    _check(case, None, "silu" if (T + W) % 2 else None, PLACE["dense"], "dense")
    _check(case, None, None if (T + W) % 2 else "silu", PLACE["dense"], "no states", bias=False, states=False)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("W", [2, 3, 4, 6])
@pytest.mark.parametrize("place", ["dense", "strided", "shifted"])
def test_causal_conv_ragged(place, W, dtype):
    """Lengths of none, one, less than the filter, around a run's end; what
    lies past a row's end is NaN and never read."""
    T, B, C = 37, 8, 48
    lengths = [0, 1, 2, 15, 16, 17, 36, 37]
    log(f"causal_conv ragged {place} W {W} {dtype}")
    case = _case(T, B, C, W, dtype, 5)
    past = torch.arange(T)[:, None] >= torch.tensor(lengths)[None]
    nan = [t.clone() for t in (case[0], case[4])]
    for t in nan:
        t[past] = float("nan")
    clean = [t.clone() for t in (case[0], case[4])]
    for t in clean:
        t[past] = 0.0
    x, w, b, state, dy, ds = case
    _check((clean[0], w, b, state, clean[1], ds), lengths, "silu", PLACE[place], place)
    put = PLACE[place]
    dense = shifted if place == "shifted" else (lambda t: t.cuda())
    dev = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    outs = []
    for xx, dd in (clean[:2], nan[:2]):
        (y, last), ctx = gss.causal_conv_train(put(xx), dense(w), dense(b), state=dense(state), lengths=dev, activation="silu")
        outs.append((y, last) + gss.causal_conv_backward(ctx, dense(dd), dense(ds)))
    for a, c in zip(*outs):
        assert torch.equal(a, c)


def test_lengths_are_clamped_and_host_values_checked():
    x, w, b, state, dy, ds = (t.cuda() for t in _case(12, 3, 16, 4, torch.float32, 3))
    wild = torch.tensor([-5, 100, 7], dtype=torch.int32, device="cuda")
    y, last = gss.causal_conv(x, w, b, state=state, lengths=wild)
    y2, last2 = gss.causal_conv(x, w, b, state=state, lengths=[0, 12, 7])
    assert torch.equal(y, y2) and torch.equal(last, last2)
    with pytest.raises(ValueError, match="lengths"):
        gss.causal_conv(x, w, b, lengths=[0, 13, 7])
    for bad in (w[:8], None, w[:, :0], w.bfloat16()):
        with pytest.raises(ValueError, match="weight"):
            gss.causal_conv(x, bad, b)
    with pytest.raises(ValueError, match="state"):
        gss.causal_conv(x, w, b, state=state[:2])
    with pytest.raises(gss.RnnError):
        gss.causal_conv(x, w[:, :1].contiguous(), b)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_token_by_token(dtype):
    x, w, b, state, _, _ = (t.cuda() for t in _case(11, 3, 72, 4, dtype, 9))
    whole, last = gss.causal_conv(x, w, b, state=state, activation="silu")
    st, out = state, []
    for t in range(11):
        y, st = gss.causal_conv(x[t:t + 1], w, b, state=st, activation="silu")
        out.append(y)
    assert torch.equal(torch.cat(out), whole) and torch.equal(st, last)


def test_infinities_stay_in_their_window():
    """An infinite input reaches W outputs of its channel and no gradient but
    those of its window."""
    x, w, b, _, dy, _ = _case(40, 1, 16, 5, torch.float32, 4)
    x[20, 0, 3] = float("inf")
    (y, _), ctx = gss.causal_conv_train(x.cuda(), w.cuda(), b.cuda())
    bad = ~torch.isfinite(y.cpu())
    assert bad[20:25, 0, 3].all() and int(bad.sum()) == 5
    dx, dw, db, _ = gss.causal_conv_backward(ctx, dy.cuda())
    assert torch.isfinite(dx).all() and torch.isfinite(db).all()
    assert int((~torch.isfinite(dw)).any(1).sum()) == 1
    dy[20, 0, 5] = float("inf")     # reaches five inputs
    dx = gss.causal_conv_backward(ctx, dy.cuda())[0]
    bad = ~torch.isfinite(dx.cpu())
    assert bad[16:21, 0, 5].all() and int(bad.sum()) == 5


def test_captured_and_replayed():
    x, w, b, state, dy, ds = (t.cuda() for t in _case(50, 4, 64, 4, torch.bfloat16, 12))
    lens = torch.tensor([50, 0, 20, 33], dtype=torch.int32, device="cuda")

    def run():
        (y, last), ctx = gss.causal_conv_train(x, w, b, state=state, lengths=lens, activation="silu")
        return (y, last) + gss.causal_conv_backward(ctx, dy, ds)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for k in range(4):
        x.copy_(torch.randn_like(x))
        lens.copy_(torch.tensor([50 - k, k, 20, 33 + k], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(out, run()):
            assert torch.equal(got, want)


def test_on_another_stream():
    x, w, b, state, dy, ds = (t.cuda() for t in _case(200, 8, 512, 4, torch.float32, 2))
    (y, last), ctx = gss.causal_conv_train(x, w, b, state=state)
    want = (y, last) + gss.causal_conv_backward(ctx, dy, ds)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        (y, last), ctx = gss.causal_conv_train(x, w, b, state=state)
        got = (y, last) + gss.causal_conv_backward(ctx, dy, ds)
    side.synchronize()
    for a, c in zip(got, want):
        assert torch.equal(a, c)
