"""Every tile and split of the feed-forward's products on the GPU, at sizes
that the plan gives them, against the definition in float64."""

import pytest
import torch

from feed_plan_shapes import SHAPES
from gpu_util import log
from test_gpu_feed_forward import BF16_HALF_ULP, KINDS, _bounds, _rms_off, _torch_act

pytestmark = pytest.mark.gpu

gss = pytest.importorskip("gru_sequence_scan_amd")

EPS = 2.0 ** -24


@pytest.mark.parametrize("dtype,rows,n,F,n_out", SHAPES)
def test_every_tile_and_split(dtype, rows, n, F, n_out):
    log(f"feed_forward plan {dtype} rows {rows} n {n} F {F} n_out {n_out}")
    kind, bf = KINDS[(rows + F) % 3], dtype == "bf16"
    g = torch.Generator(device="cuda").manual_seed(rows + n + F)

    def normal(a, b, scale=1.0):
        return (torch.randn((a, b), generator=g, device="cuda", dtype=torch.float32) * scale).to(torch.bfloat16 if bf else torch.float32)

    x, r, dy = normal(rows, n), normal(rows, n_out, 2.0), normal(rows, n_out)
    w_in, w_out = normal(2 * F, n, n ** -0.5), normal(n_out, F, F ** -0.5)
    y, ctx = gss.feed_forward_train(x, w_in, w_out, residual=r, activation=kind)
    got = (y,) + gss.feed_forward_backward(ctx, dy)
    served = gss.feed_forward(x, w_in, w_out, residual=r, activation=kind)
    del ctx
    x, w_in, w_out, dy, r = (t.double() for t in (x, w_in, w_out, dy, r))
    act, slope = _torch_act(x @ w_in[:F].T, kind)
    u = x @ w_in[F:].T
    dh = dy @ w_out
    dp = torch.cat([dh * u * slope, dh * act], 1)
    ref = ((act * u) @ w_out.T + r, dp @ w_in, dp.T @ x, dy.T @ (act * u))
    bounds = _bounds(x, w_in, w_out, dy, kind, _torch_act) if bf else (0.0,) * 4
    # A sum of K products of random signs, term by term: partial sums of k terms are sqrt(k) of one term's size and each
    # is rounded by at most EPS of itself, sqrt(K / 2) EPS of the result in all (2-norms). g and u have that of N and
    # dh that of N_out as factors, the activation and its slope a few EPS. bf16: one rounding of the terms and one of
    # the result, each of mean square at most a third of half an ulp's.
    inner = 2 * (n / 2) ** 0.5 + (n_out / 2) ** 0.5 + 8
    for got_t, t, b, terms, name in zip(got, ref, bounds, (F, 2 * F, rows, rows), ("y", "dx", "dw_in", "dw_out")):
        most = EPS * ((terms / 2) ** 0.5 + inner) + ((2.0 / 3.0) ** 0.5 * BF16_HALF_ULP if bf else 0.0)
        assert _rms_off(got_t, t) < most, name
        limit = 1e-4 * t.abs() + 1e-5 * t.abs().max()
        if bf:
            limit = limit + b
            limit = limit + BF16_HALF_ULP * (t.abs() + limit)
        assert bool(((got_t.double() - t).abs() <= limit).all()), name
    assert torch.equal(served, y)
