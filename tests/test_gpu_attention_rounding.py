"""What bf16 attention rounds and what it does not: p, ds and o enter the sums
as the rounded value and the rest of its rounding, in o and dq always, in dk
and dv where the launch has at most as many workgroups as the device has
compute units. On the CPU: the bounds used here do not hold for sums of values
that are rounded only once."""

import numpy as np
import pytest
import torch

import oracle
from block_util import assert_near, draw, f64

gss = pytest.importorskip("gru_sequence_scan_amd")

DTYPE = torch.bfloat16
REST, ONCE = 2.0 ** -16, 2.0 ** -8   # a value with its rest: two roundings of 2^-8 at most; rounded once

# Tq, Tk, B, heads, kv_heads, D, whether dk and dv take the rest: tiles of 64 keys (heads of 64 and less) or 128, times
# B kv_heads, against 256 compute units
CASES = [
    (1, 40, 3, 4, 2, 64, True), (20, 150, 4, 4, 2, 64, True), (33, 70, 8, 4, 4, 40, True), (20, 300, 4, 4, 2, 128, True),
    (70, 200, 3, 4, 2, 96, True), (9, 1100, 1, 4, 1, 32, True), (50, 70, 64, 2, 2, 64, True),
    (50, 70, 70, 4, 4, 64, False), (37, 130, 70, 8, 4, 128, False), (20, 70, 100, 3, 3, 33, False),
]


def _case(Tq, Tk, B, heads, kv, D):
    rng = np.random.default_rng(Tq * 7 + Tk + D)
    q, do = draw(rng, (Tq, B, heads, D), DTYPE), draw(rng, (Tq, B, heads, D), DTYPE)
    k, v = draw(rng, (Tk, B, kv, D), DTYPE), draw(rng, (Tk, B, kv, D), DTYPE)
    # rows of few keys, where one rounding shows most, beside long ones and an empty one
    lengths = None if B < 3 else [(3, Tk, 0, 7, Tk // 2, 1)[b % 6] for b in range(B)]
    return q, k, v, do, lengths


def _fp32_unit(q, k):
    """Relative error of a probability in fp32: 2^-24 of the sum of a score's
    products' sizes at each of up to four steps, and 2^-22 for the rest."""
    size = max((np.abs(q[:, b, h]) @ np.abs(k[:, b, hk]).T).max() for b, h, hk, _ in oracle.block._pairs(q, k, None))
    return 2.0 ** -22 * (1.0 + float(size) * q.shape[-1] ** -0.5)


def _limits(q, k, v, do, lengths):
    fp32 = _fp32_unit(q, k)
    return [oracle.attention_bounds(q, k, v, do, lengths, None, fp32 + u) for u in (REST, ONCE)]


@pytest.mark.gpu
@pytest.mark.parametrize("Tq,Tk,B,heads,kv,D,rest", CASES)
def test_bf16_sums_keep_the_rest(Tq, Tk, B, heads, kv, D, rest):
    print(f"attention rounding Tq {Tq} Tk {Tk} B {B} heads {heads}/{kv} D {D}", flush=True)
    q, k, v, do, lengths = _case(Tq, Tk, B, heads, kv, D)
    args = [f64(t) for t in (q, k, v)]
    tight, once = _limits(*args, f64(do), lengths)
    o, ctx = gss.cross_attention_train(q.cuda(), k.cuda(), v.cuda(), lengths=lengths)
    assert_near(o, oracle.cross_attention(*args, lengths), DTYPE, "o", tight[0])
    got = gss.cross_attention_backward(ctx, do.cuda())
    ref = oracle.cross_attention_backward(*args, f64(do), lengths)
    assert_near(got[0], ref[0], DTYPE, "dq", tight[1])
    for n, name in ((1, "dk"), (2, "dv")):
        assert_near(got[n], ref[n], DTYPE, name, (tight if rest else once)[n + 1])


def _round(x):
    return torch.from_numpy(x).to(DTYPE).double().numpy()


def _emulated(q, k, v, do, lengths, rounded):
    """o, dq, dk, dv in float64 with the named values rounded once to bf16."""
    scale = q.shape[-1] ** -0.5
    o, dq, dk, dv = np.zeros_like(q), np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for b, h, hk, n in oracle.block._pairs(q, k, lengths):
        if not n:
            continue
        p = oracle.block._softmax(scale * q[:, b, h] @ k[:n, b, hk].T)
        pr = _round(p) if "p" in rounded else p
        o[:, b, h] = pr @ v[:n, b, hk]
        kept = _round(p @ v[:n, b, hk]) if "o" in rounded else p @ v[:n, b, hk]
        ds = p * (do[:, b, h] @ v[:n, b, hk].T - (do[:, b, h] * kept).sum(-1, keepdims=True))
        ds = (_round(ds) if "ds" in rounded else ds) * scale
        dq[:, b, h] = ds @ k[:n, b, hk]
        dk[:n, b, hk] += ds.T @ q[:, b, h]
        dv[:n, b, hk] += pr.T @ do[:, b, h]
    return [_round(t) for t in (o, dq, dk, dv)]


@pytest.mark.parametrize("Tq,Tk,B,heads,kv,D", [c[:6] for c in CASES if 3 <= c[2] <= 8])
def test_bounds_tell_the_rest(Tq, Tk, B, heads, kv, D):
    """On the cases with rows of few keys (over many, one rounding's errors
    average out below the output's own)."""
    q, k, v, do, lengths = _case(Tq, Tk, B, heads, kv, D)
    args = [f64(t) for t in (q, k, v, do)]
    tight, once = _limits(*args, lengths)
    ref = [oracle.cross_attention(*args[:3], lengths), *oracle.cross_attention_backward(*args, lengths)]
    names = ("o", "dq", "dk", "dv")
    for name, t, r, e in zip(names, _emulated(*args, lengths, ()), ref, tight):
        assert_near(t, r, DTYPE, name, e)
    for rounded, tells in (("p", ("o", "dv")), ("ds", ("dq", "dk")), ("o", ("dq", "dk"))):
        got = _emulated(*args, lengths, (rounded,))
        for name, t, r, e, loose in zip(names, got, ref, tight, once):
            assert_near(t, r, DTYPE, name, loose)
            if name in tells:
                with pytest.raises(AssertionError):
                    assert_near(t, r, DTYPE, name, e)
