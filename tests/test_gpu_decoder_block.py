"""The operators together: examples/decoder_block.py trains and decodes, and
its gradients are those of the plain block in float64."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from block_util import assert_near, f64
from gpu_util import log

pytestmark = pytest.mark.gpu

pytest.importorskip("gru_sequence_scan_amd")

_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_block.py")


def _example():
    spec = importlib.util.spec_from_file_location("decoder_block", _PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_example_trains_and_decodes(dtype):
    log(f"decoder block {dtype}")
    losses, apart = _example().main(dtype=dtype)
    assert all(np.isfinite(losses)) and losses[-1] < 0.9 * losses[0]
    # outputs of size about 4; the two runs round at the same places, and the
    # library's products may sum in another order for one row than for many
    assert apart < (1e-3 if dtype == torch.float32 else 0.25)


def _plain(w, x, enc, lengths, heads, kv_heads):
    """The block in float64 on the CPU, differentiable."""
    T, B, H = x.shape
    D = H // heads

    def norm(t, a, b):
        return torch.nn.functional.layer_norm(t, (H,), a, b)

    p = (norm(x, w["norm1"], w["bias1"]) @ w["scan"]).view(T, B, 2, H)
    a, state, hs = torch.sigmoid(p[:, :, 1]), torch.zeros(B, H, dtype=torch.float64), []
    for t in range(T):
        state = a[t] * state + (1 - a[t]) * p[t, :, 0]
        hs.append(state)
    s = x + torch.stack(hs) @ w["out"]
    q = (norm(s, w["norm2"], w["bias2"]) @ w["q"]).view(T, B, heads, D)
    kv = (enc @ w["kv"]).view(*enc.shape[:2], 2, kv_heads, D)
    rows = []
    for b in range(B):
        n = lengths[b]
        k, v = (kv[:n, b, i].repeat_interleave(heads // kv_heads, 1).transpose(0, 1) for i in (0, 1))
        att = torch.softmax(q[:, b].transpose(0, 1) @ k.transpose(1, 2) * D ** -0.5, -1) @ v
        rows.append(att.transpose(0, 1))
    return s + torch.stack(rows, 1).reshape(T, B, H) @ w["mix"]


def test_example_gradients():
    ex = _example()
    T, B, S, H, heads, kv = 9, 3, 14, 32, 4, 2
    lengths = [14, 1, 8]
    enc = ex.encoder(B, S, 8, 12, lengths, torch.float32)
    block = ex.DecoderBlock(H, 24, heads, kv, torch.float32, seed=3)
    g = torch.Generator().manual_seed(5)
    x, dy = torch.randn(2, T, B, H, generator=g, dtype=torch.float32)
    y, saved = block.train(x.cuda(), enc, lengths)
    grads, dx, denc = block.backward(saved, dy.cuda())
    w = {k: v.double().cpu().requires_grad_(True) for k, v in block.w.items()}
    xr, er = x.double().requires_grad_(True), enc.double().cpu().requires_grad_(True)
    ref = _plain(w, xr, er, lengths, heads, kv)
    ref.backward(dy.double())
    assert_near(y, f64(ref), torch.float32, "y")
    for name in w:
        assert_near(grads[name], f64(w[name].grad), torch.float32, name, 2e-5 * float(w[name].grad.abs().max()))
    assert_near(dx, f64(xr.grad), torch.float32, "dx", 2e-5 * float(xr.grad.abs().max()))
    assert_near(denc, f64(er.grad), torch.float32, "denc", 2e-5 * float(er.grad.abs().max()))
