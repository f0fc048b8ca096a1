"""Cross attention on the GPU against the float64 definition: types, head
layouts, lengths, odd sizes, strides, masked rows, gradients."""

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


def _case(Tq, Tk, B, heads, kv, D, dtype, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    q, do = draw(rng, (Tq, B, heads, D), dtype, spread), draw(rng, (Tq, B, heads, D), dtype)
    k, v = draw(rng, (Tk, B, kv, D), dtype), draw(rng, (Tk, B, kv, D), dtype)
    return q, k, v, do


def _check(q, k, v, do, lengths=None, scale=None, dev=None, put=lambda t: t.cuda(), put_grad=lambda t: t.cuda(), what="",
           train=True):
    """Forward and gradients within fp32 accuracy, plus, for bf16 storage, the
    bounds of one rounding (2^-8 at most) of each p, ds and o in the sums.
    The fp32 part carries the error of a score: 2^-22 of its size (products
    of D terms, then an exponential of the difference), relative to p."""
    dtype = q.dtype
    args = (f64(q), f64(k), f64(v))
    size = np.abs(args[0]).max() * np.abs(args[1]).max() * q.shape[-1] * (q.shape[-1] ** -0.5 if scale is None else abs(scale))
    unit = 2.0 ** -22 * (4.0 + size) + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
    bounds = oracle.attention_bounds(*args, f64(do), lengths, scale, unit)
    dev = lengths if dev is None else dev
    g = [put(t) for t in (q, k, v)]
    o = gss.cross_attention(*g, lengths=dev, scale=scale)
    assert_near(o, oracle.cross_attention(*args, lengths, scale), dtype, what + " o", bounds[0])
    if not train:
        return o
    o2, ctx = gss.cross_attention_train(*g, lengths=dev, scale=scale)
    assert torch.equal(o, o2)
    got = gss.cross_attention_backward(ctx, put_grad(do))
    for name, a, r, e in zip(("dq", "dk", "dv"), got, oracle.cross_attention_backward(*args, f64(do), lengths, scale), bounds[1:]):
        assert_near(a, r, dtype, f"{what} {name}", e)
    return (o,) + got


ATTEND_CASES = [  # Tq, Tk, B, heads, kv_heads, D: one token and one key, tile edges (16, 32, 64, 128), odd sizes, shared heads
    (1, 1, 1, 1, 1, 1), (1, 5, 3, 2, 1, 8), (1, 130, 2, 8, 8, 64), (1, 300, 1, 16, 2, 128), (2, 33, 2, 4, 4, 40),
    (5, 64, 2, 6, 2, 72), (16, 65, 1, 2, 2, 32), (17, 31, 3, 3, 1, 33), (63, 127, 1, 2, 1, 96), (65, 40, 2, 2, 2, 100),
    (129, 129, 1, 4, 1, 128), (130, 20, 1, 1, 1, 127), (40, 513, 1, 2, 2, 16), (3, 1100, 1, 4, 2, 80),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("Tq,Tk,B,heads,kv,D", ATTEND_CASES)
def test_cross_attention(Tq, Tk, B, heads, kv, D, dtype):
    log(f"cross_attention Tq {Tq} Tk {Tk} B {B} heads {heads}/{kv} D {D} {dtype}")
    _check(*_case(Tq, Tk, B, heads, kv, D, dtype, Tq * 100 + Tk), what="whole")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("Tq,heads,kv,D", [(1, 4, 4, 64), (1, 8, 2, 128), (9, 2, 1, 32), (70, 4, 2, 64), (70, 2, 2, 96)])
def test_cross_attention_ragged(Tq, heads, kv, D, dtype):
    """Row lengths from none to all, at tile edges; NaN and infinities in the
    states past them must not matter."""
    Tk, lengths = 150, [150, 0, 1, 15, 16, 17, 63, 64, 65, 128, 129, 0, 149]
    q, k, v, do = _case(Tq, Tk, len(lengths), heads, kv, D, dtype, Tq + D)
    dev = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    log(f"cross_attention ragged Tq {Tq} heads {heads}/{kv} D {D} {dtype}")

    def dirty(t):
        out = t.cuda()
        if t.shape[0] == Tk:
            for b, L in enumerate(lengths):
                out[L:, b] = [float("nan"), float("inf"), -float("inf")][b % 3]
        return out

    o, dq, dk, dv = _check(q, k, v, do, lengths, dev=dev, put=dirty, what="ragged")
    for b, L in enumerate(lengths):
        assert (f64(dk)[L:, b] == 0).all() and (f64(dv)[L:, b] == 0).all()
        if L == 0:
            assert (f64(o)[:, b] == 0).all() and (f64(dq)[:, b] == 0).all()
    host = gss.cross_attention(q.cuda(), k.cuda(), v.cuda(), lengths=lengths)
    wild = torch.tensor([Tk + 7 if n == Tk else (-3 if n == 0 else n) for n in lengths], device="cuda")
    for n in (wild, wild.int()):
        assert torch.equal(host, gss.cross_attention(q.cuda(), k.cuda(), v.cuda(), lengths=n))
    assert torch.equal(host, o)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("Tq,Tk,B,heads,kv,D", [
    (50, 70, 70, 4, 4, 64), (50, 70, 70, 4, 4, 40), (37, 130, 70, 8, 4, 128), (70, 33, 70, 4, 4, 96), (65, 40, 60, 4, 4, 33),
    (50, 65, 100, 4, 4, 32), (40, 1100, 1, 2, 1, 64), (70, 1030, 2, 2, 2, 128), (33, 1100, 1, 3, 1, 100),
])
def test_cross_attention_wide_tiles(Tq, Tk, B, heads, kv, D, dtype):
    """Enough rows, or keys, for the kernels that work on wide tiles of query
    rows, whole and ragged (a row without keys among them), and for long keys
    that are split over workgroups."""
    log(f"cross_attention wide Tq {Tq} Tk {Tk} B {B} heads {heads}/{kv} D {D} {dtype}")
    q, k, v, do = _case(Tq, Tk, B, heads, kv, D, dtype, D + B)
    _check(q, k, v, do, what="whole")
    if B > 2:
        lengths = [(7 * b) % (Tk + 1) for b in range(B)]
        lengths[1] = Tk
        dev = torch.tensor(lengths, dtype=torch.int32, device="cuda")

        def dirty(t):
            out = t.cuda()
            if t.shape[0] == Tk and t.shape[2] == kv:
                for b, L in enumerate(lengths):
                    out[L:, b] = float("nan")
            return out

        _check(q, k, v, do, lengths, dev=dev, put=dirty, what="ragged")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("D", [64, 24, 33])
@pytest.mark.parametrize("Tq", [1, 21])
def test_cross_attention_layouts(Tq, D, dtype):
    """Slices of one projection, batch-major tensors, rows apart and unaligned
    memory give what dense time-major tensors give."""
    Tk, B, heads, kv = 70, 3, 4, 2
    q, k, v, do = _case(Tq, Tk, B, heads, kv, D, dtype, 5)
    ref = _check(q, k, v, do, what="dense")
    fused = torch.cat([k, v], 2).cuda()
    ways = {
        "fused": (q.cuda(), fused[:, :, :kv], fused[:, :, kv:]),
        "batch_major": tuple(t.transpose(0, 1).contiguous().cuda().transpose(0, 1) for t in (q, k, v)),
        "head_major": tuple(t.permute(1, 2, 0, 3).contiguous().cuda().permute(2, 0, 1, 3) for t in (q, k, v)),
        "strided": tuple(strided(t) for t in (q, k, v)),
        "shifted": tuple(shifted(t) for t in (q, k, v)),
        "last_dim_apart": tuple(t.repeat_interleave(2, -1).cuda()[..., ::2] for t in (q, k, v)),
    }
    for name, g in ways.items():
        log(f"cross_attention layout {name} Tq {Tq} D {D} {dtype}")
        o, ctx = gss.cross_attention_train(*g)
        for a, b in zip((o,) + gss.cross_attention_backward(ctx, shifted(do) if name == "shifted" else do.cuda()), ref):
            assert torch.equal(a, b), name
    # a broadcast key head: stride 0
    one = k[:, :, :1].cuda().expand(Tk, B, heads, D)
    many = k[:, :, :1].expand(Tk, B, heads, D).contiguous().cuda()
    assert torch.equal(gss.cross_attention(q.cuda(), one, one), gss.cross_attention(q.cuda(), many, many))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_cross_attention_scales_and_peaks(dtype):
    """Nearly uniform scores, peaked ones, a negative and a zero scale."""
    for n, (spread, scale) in enumerate([(0.01, None), (12.0, None), (1.0, -0.3), (1.0, 0.0), (1.0, 2.0)]):
        log(f"cross_attention spread {spread} scale {scale} {dtype}")
        _check(*_case(19, 90, 2, 2, 1, 64, dtype, 40 + n, spread), scale=scale, what=f"spread {spread} scale {scale}")


def test_cross_attention_large_scores():
    """Scores of the size of 1e4 (a running maximum that moves far) and of the
    largest finite values stay finite where the softmax is."""
    q, k, v, _ = (t.cuda() for t in _case(4, 200, 1, 2, 2, 64, torch.float32, 77))
    o = gss.cross_attention(q * 1e4, k, v)
    assert torch.isfinite(o).all()
    # one key far above the others takes all the weight
    k[123] = 0.0
    k[123, :, :, 0] = 3e37
    q[..., 0] = 1.0
    o = gss.cross_attention(q, k, v, scale=1.0)
    assert torch.equal(o, v[123][None].expand_as(o))
    # the others' scores all at the type's lowest
    q[..., 0], q[..., 1:] = -1.0, 0.0
    k[:, :, :, 0] = torch.finfo(torch.float32).max
    k[7] = 0.0
    assert torch.equal(gss.cross_attention(q, k, v, scale=1.0), v[7][None].expand_as(o))


def test_cross_attention_nan_stays_in_its_row():
    q, k, v, do = (t.cuda() for t in _case(20, 40, 2, 2, 2, 32, torch.bfloat16, 3))
    ref = gss.cross_attention(q, k, v)
    q[3, 1, 0, 5] = float("nan")
    o = gss.cross_attention(q, k, v)
    assert torch.isnan(o[3, 1, 0]).all()
    o[3, 1, 0] = ref[3, 1, 0]
    assert torch.equal(o, ref)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_cross_attention_long_and_deterministic(dtype):
    """A long key axis, split over workgroups: right, and the same bits again."""
    q, k, v, do = _case(1, 9001, 2, 8, 2, 64, dtype, 9)
    log(f"cross_attention long {dtype}")
    o = _check(q, k, v, do, [9001, 4097], what="long", train=False)
    for _ in range(3):
        assert torch.equal(o, gss.cross_attention(q.cuda(), k.cuda(), v.cuda(), lengths=[9001, 4097]))


def test_cross_attention_offsets_past_32_bits():
    """Keys whose element offsets pass 2^31: the last rows of a view into a
    buffer of more than 2^31 elements are read where they are."""
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of free device memory")
    stride = 1 << 28   # elements between key steps: step 9 lies at 2.4e9
    buf = torch.empty(9 * stride + 4096, dtype=torch.bfloat16, device="cuda")
    q, k, v, _ = _case(1, 10, 1, 2, 2, 64, torch.bfloat16, 21)
    views = []
    for n, t in enumerate((k, v)):
        w = buf[n * 1024:].as_strided((10, 1, 2, 64), (stride, 128, 64, 1))
        w.copy_(t)
        views.append(w)
    o = gss.cross_attention(q.cuda(), *views)
    assert torch.equal(o, gss.cross_attention(q.cuda(), k.cuda(), v.cuda()))


def test_cross_attention_capture_and_streams():
    q, k, v, do = (t.cuda() for t in _case(33, 100, 2, 4, 2, 64, torch.bfloat16, 6))
    lengths = torch.tensor([100, 40], dtype=torch.int32, device="cuda")

    def step():
        o, ctx = gss.cross_attention_train(q, k, v, lengths=lengths)
        one = gss.cross_attention(q[:1], k, v, lengths=lengths)
        return (o, one) + gss.cross_attention_backward(ctx, do)

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
    for n in (100, 3, 0):
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(n)).to(q.dtype))
        lengths[0] = n
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(step(), held):
            assert torch.equal(a, b)
