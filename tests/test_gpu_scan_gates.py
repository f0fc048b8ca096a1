"""The gated scan's gradients at gates far in their tails, element by element:
sigma' = s (1 - s) is as small as 1e-26 there, and has its own relative
accuracy."""

import numpy as np
import pytest
import torch

import oracle
from block_util import BF16_HALF_ULP, F32_REL, f64, shifted
from gpu_util import log

pytestmark = pytest.mark.gpu

gss = pytest.importorskip("gru_sequence_scan_amd")

DTYPES = [torch.float32, torch.bfloat16]
IDS = ["f32", "bf16"]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("reverse", [False, True], ids=["forward", "reverse"])
@pytest.mark.parametrize("T,H,place", [(1, 16, "dense"), (5, 33, "dense"), (300, 24, "dense"), (300, 24, "shifted"),
                                       (1700, 8, "dense")])
def test_gradients_of_saturated_gates(T, H, place, reverse, dtype):
    """Every gate between 4 and 60 (a column has one sign), x and the incoming
    gradients positive, so that no sum cancels and each element is within the
    storage type's rounding and 1e-4 of its own size: the exponential of a
    rounded product carries 60 * 2^-24 = 4e-6, sums of T positive terms in
    fp32 less than T 2^-24 = 1e-4 at T = 1700."""
    log(f"saturated gates T {T} H {H} {place} reverse {reverse} {dtype}")
    rng = np.random.default_rng(T + H)

    def positive(*shape):
        return torch.from_numpy(rng.uniform(0.5, 1.5, shape).astype(np.float32))

    B = 3
    x, dy = positive(T, B, H).to(dtype), positive(T, B, H).to(dtype)
    h0, dhn = positive(B, H), positive(B, H)
    sign = np.where(np.arange(H) % 2 == 0, 1.0, -1.0)
    f = torch.from_numpy((rng.uniform(4.0, 60.0, (T, B, H)) * sign).astype(np.float32)).to(dtype)
    i = torch.from_numpy((rng.uniform(4.0, 60.0, (T, B, H)) * np.roll(sign, H // 2)).astype(np.float32)).to(dtype)
    put = shifted if place == "shifted" else (lambda t: t.cuda())
    _, ctx = gss.gated_scan_train(put(x), put(f), put(i), h0=h0.cuda(), reverse=reverse)
    got = gss.gated_scan_backward(ctx, put(dy), dhn.cuda())
    ref = oracle.gated_scan_backward(f64(x), f64(f), f64(i), f64(dy), f64(dhn), f64(h0), None, reverse)
    for name, a, r in zip(("dx", "df", "di", "dh0"), got, ref):
        rel = 2 * F32_REL + (BF16_HALF_ULP if dtype == torch.bfloat16 and name != "dh0" else 0.0)
        # fp32 has no 24 bits below 2^-126, bf16 storage none of its 8 bits
        worst = np.abs(f64(a) - r) - rel * np.abs(r) - 2.0 ** -130
        at = np.unravel_index(int(worst.argmax()), r.shape)
        assert worst[at] <= 0.0, f"{name} at {at}: {f64(a)[at]:.6g} for {r[at]:.6g}"
        if name == "di":
            assert (f64(a) != 0.0).all()
