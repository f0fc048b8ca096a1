"""Cross attention at large scores, forward and backward.

The scores are made exact: a query row holds (A, n, 0, ...), a key (1, off,
...), so that with scale 1 a score is A + n off, a number that fp32 holds (n
is a multiple of the spacing of fp32 below A). The softmax does not depend on
A, and a kernel that forms a score's distance from the row's maximum without
loss gives the probabilities to fp32 accuracy, however large A is."""

import numpy as np
import pytest
import torch

import oracle
from block_util import assert_near, draw, f64
from gpu_util import log

pytestmark = pytest.mark.gpu

gss = pytest.importorskip("gru_sequence_scan_amd")

DTYPES = [torch.float32, torch.bfloat16]
IDS = ["f32", "bf16"]

# the tiles of every kernel: one token and few rows (waves that divide the keys), long keys split over workgroups, wide
# tiles, heads of 64 and less, of up to 128, and sizes without 16-byte rows
SHAPES = [  # Tq, Tk, B, heads, kv_heads, D
    (1, 300, 2, 4, 2, 64), (3, 70, 2, 4, 2, 64), (5, 90, 2, 2, 1, 33), (1, 5000, 1, 8, 2, 128), (21, 200, 2, 2, 2, 100),
    (40, 1100, 1, 4, 2, 64), (50, 70, 70, 4, 4, 40), (37, 130, 70, 8, 4, 128), (70, 1030, 2, 2, 2, 96),
]


def _case(Tq, Tk, B, heads, kv, D, dtype, level, seed):
    """Every other row of queries has scores about `level`, the rest small
    ones. Offsets are mostly far below the row's maximum, with ties and near
    ties of it at both ends and in the middle of the keys."""
    rng = np.random.default_rng(seed)
    q = torch.zeros(Tq, B, heads, D, dtype=dtype)
    rows = torch.arange(Tq * heads).view(Tq, 1, heads)
    q[..., 0] = (rows % 2 * float(level)).to(dtype)
    q[..., 1] = ((1.0 + rows % 3) * max(1.0, level * 2.0 ** -24)).to(dtype)
    k, v, do = draw(rng, (Tk, B, kv, D), dtype), draw(rng, (Tk, B, kv, D), dtype), draw(rng, (Tq, B, heads, D), dtype)
    k[..., 0] = 1.0
    k[..., 1] = torch.from_numpy(-rng.integers(0, 9, (Tk, B, kv)).astype(np.float32)).to(dtype)
    return q, k, v, do


def _unit(dtype):
    """Relative error of a probability, beside what rounding p and ds to bf16
    for dk and dv costs: the score's distance from the maximum is exact; times
    log2 e, beside what the reference's rounding leaves (16 at most) and the
    log of the sum, it carries 2^-24 of 32 where the probability counts, the
    exponentials and the sum 2^-22. In bf16 a value and the rest of its
    rounding, each rounded by 2^-8 at most, hold it to 2^-16, p and ds in the
    sums and o in delta; half of that is allowed, since the errors of a sum's
    terms differ in sign."""
    return (2.0 ** -19 + 2.0 ** -17, 2.0 ** -8) if dtype == torch.bfloat16 else (2.0 ** -19, 0.0)


def _check_forward(case, lengths, dtype, what, scale=1.0):
    q, k, v, do = case
    args = (f64(q), f64(k), f64(v))
    bound = oracle.attention_bounds(*args, f64(do), lengths, scale, _unit(dtype)[0])[0]
    o = gss.cross_attention(*[t.cuda() for t in (q, k, v)], lengths=lengths, scale=scale)
    assert_near(o, oracle.cross_attention(*args, lengths, scale), dtype, what, bound)


def _check_backward(case, lengths, dtype, what, scale=1.0):
    q, k, v, do = case
    args = (f64(q), f64(k), f64(v))
    unit, rounding = _unit(dtype)
    exact = oracle.attention_bounds(*args, f64(do), lengths, scale, unit)
    loose = oracle.attention_bounds(*args, f64(do), lengths, scale, unit + rounding)
    o, ctx = gss.cross_attention_train(*[t.cuda() for t in (q, k, v)], lengths=lengths, scale=scale)
    dq, dk, dv = gss.cross_attention_backward(ctx, do.cuda())
    rq, rk, rv = oracle.cross_attention_backward(*args, f64(do), lengths, scale)
    assert_near(dq, rq, dtype, what + " dq", exact[1])
    # column 0 of dk carries the level: it and the others each against their own largest value
    dk = f64(dk)
    assert_near(dk[..., :1], rk[..., :1], dtype, what + " dk column 0", loose[2][..., :1])
    assert_near(dk[..., 1:], rk[..., 1:], dtype, what + " dk", loose[2][..., 1:])
    assert_near(dv, rv, dtype, what + " dv", loose[3])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("Tq,Tk,B,heads,kv,D", SHAPES)
def test_large_scores_forward(Tq, Tk, B, heads, kv, D, dtype):
    lengths = None if B < 3 else [(11 * b) % (Tk + 1) for b in range(B)]
    for power in (9, 13, 17, 20, 22, 25, 27):
        log(f"large scores 2^{power} Tq {Tq} Tk {Tk} B {B} heads {heads}/{kv} D {D} {dtype}")
        _check_forward(_case(Tq, Tk, B, heads, kv, D, dtype, 2 ** power, power + D), lengths, dtype, f"2^{power}")


def _moving(Tq, Tk, D, dtype, power, scale):
    """Scores that grow along the keys, so that the running maximum moves many
    times and each part of the keys has another one. Neighbours share the
    weight: steps of 1 / 128 (2^16 and less), else of 1 every 8 keys."""
    q, k, v, do = _case(Tq, Tk, 1, 4, 2, D, dtype, 2 ** power, power)
    n = torch.arange(Tk).float().view(Tk, 1, 1)
    fine = 64 if power <= 16 else 8
    k[..., 1] = 0.0
    k[..., 2] = ((n // fine) - Tk // fine).to(dtype)
    k[..., 3] = (n % fine).to(dtype)
    q[..., 1], q[..., 2], q[..., 3] = 0.0, 0.5 if power <= 16 else 1.0, 2.0 ** -7 if power <= 16 else 0.0
    return q if scale > 0 else -q, k, v, do


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("Tq,Tk", [(1, 1200), (1, 9000), (40, 1200)])
def test_maximum_that_moves_forward(Tq, Tk, dtype):
    """Up, down, and with a negative scale."""
    for power in (13, 16, 20, 22):
        for scale in (1.0, -1.0):
            q, k, v, do = _moving(Tq, min(Tk, 1200) if power <= 16 else Tk, 64, dtype, power, scale)
            for name, kk in (("up", k), ("down", k.flip(0))):
                log(f"maximum that moves {name} Tq {Tq} Tk {Tk} 2^{power} scale {scale} {dtype}")
                _check_forward((q, kk, v, do), None, dtype, f"{name} 2^{power}", scale)


LARGEST = [(2, 150, 1, 4, 2, 64), (1, 5000, 1, 2, 2, 64), (40, 1100, 1, 4, 2, 64), (37, 130, 70, 8, 4, 128)]


def _largest(Tq, Tk, B, heads, kv, D, dtype, score, where):
    """Keys `where` far above the others."""
    rng = np.random.default_rng(31)
    q = torch.zeros(Tq, B, heads, D, dtype=dtype)
    q[..., 0] = 1.0
    k, v, do = draw(rng, (Tk, B, kv, D), dtype), draw(rng, (Tk, B, kv, D), dtype), draw(rng, (Tq, B, heads, D), dtype)
    for n in where:
        k[n] = 0.0
        k[n, ..., 0] = score
    return q, k, v, do


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("Tq,Tk,B,heads,kv,D", LARGEST)
def test_largest_scores_forward(Tq, Tk, B, heads, kv, D, dtype):
    """One key far above the others, at scores up to the type's largest finite
    values, takes all the weight; two such keys share it; and so do all keys
    at the type's lowest value."""
    for score in (1e9, 3e37, 3e38):
        for where in ((Tk // 3,), (7, Tk - 2)):
            log(f"largest scores {score} keys {where} Tq {Tq} Tk {Tk} D {D} {dtype}")
            q, k, v, _ = _largest(Tq, Tk, B, heads, kv, D, dtype, score, where)
            o = gss.cross_attention(q.cuda(), k.cuda(), v.cuda(), scale=1.0)
            ref = torch.stack([v[n].double() for n in where]).mean(0).repeat_interleave(heads // kv, 1)
            assert_near(o, ref.expand(o.shape).numpy(), dtype, f"{score}", 2.0 ** -21)
    k[:] = 0.0
    k[..., 0] = float(torch.finfo(dtype).min)
    o = gss.cross_attention(q.cuda(), k.cuda(), v.cuda(), scale=1.0)
    ref = f64(v).mean(0).repeat(heads // kv, 1)
    assert_near(o, np.broadcast_to(ref, o.shape), dtype, "lowest", 2.0 ** -18)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("Tq,Tk,B,heads,kv,D", SHAPES)
def test_large_scores_backward(Tq, Tk, B, heads, kv, D, dtype):
    lengths = None if B < 3 else [(11 * b) % (Tk + 1) for b in range(B)]
    for power in (9, 13, 17, 20, 22, 25, 27):
        log(f"large scores 2^{power} Tq {Tq} Tk {Tk} B {B} heads {heads}/{kv} D {D} {dtype}")
        _check_backward(_case(Tq, Tk, B, heads, kv, D, dtype, 2 ** power, power + D), lengths, dtype, f"2^{power}")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("Tq,Tk", [(1, 1200), (1, 9000), (40, 1200)])
def test_maximum_that_moves_backward(Tq, Tk, dtype):
    """Up, down, and with a negative scale."""
    for power in (13, 16, 20, 22):
        for scale in (1.0, -1.0):
            q, k, v, do = _moving(Tq, min(Tk, 1200) if power <= 16 else Tk, 64, dtype, power, scale)
            for name, kk in (("up", k), ("down", k.flip(0))):
                log(f"maximum that moves {name} Tq {Tq} Tk {Tk} 2^{power} scale {scale} {dtype}")
                _check_backward((q, kk, v, do), None, dtype, f"{name} 2^{power}", scale)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("Tq,Tk,B,heads,kv,D", LARGEST)
def test_largest_scores_backward(Tq, Tk, B, heads, kv, D, dtype):
    """The value of a key that takes all the weight gets the sum of the rows'
    incoming gradients; two such keys, and all keys at the type's lowest
    score, share it."""
    def check(q, k, v, do, where):
        o, ctx = gss.cross_attention_train(q.cuda(), k.cuda(), v.cuda(), scale=1.0)
        _, dk, dv = gss.cross_attention_backward(ctx, do.cuda())
        per = f64(do).reshape(Tq, B, kv, heads // kv, D)
        want, size = np.zeros(dv.shape), np.zeros(dv.shape)
        want[where], size[where] = per.sum((0, 3)) / len(where), np.abs(per).sum((0, 3)) / len(where)
        # p is 1 / n: exact in fp32 and, where n is a power of two, in bf16
        exact = dtype == torch.float32 or len(where) & (len(where) - 1) == 0
        assert_near(dv, want, dtype, "dv", (2.0 ** -19 if exact else 2.0 ** -8) * size)
        return f64(dk)

    for score in (1e9, 3e37, 3e38):
        for where in ([Tk // 3], [7, Tk - 2]):
            log(f"largest scores backward {score} keys {where} Tq {Tq} Tk {Tk} D {D} {dtype}")
            q, k, v, do = _largest(Tq, Tk, B, heads, kv, D, dtype, score, where)
            dk = check(q, k, v, do, where)
            # the other keys have no weight at all
            assert np.isfinite(dk).all() and not dk[[n for n in range(Tk) if n not in where]].any()
    k[:] = 0.0
    k[..., 0] = float(torch.finfo(dtype).min)
    check(q, k, v, do, list(range(Tk)))
