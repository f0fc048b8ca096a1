"""A recurrent decoder block over a variable-length encoder.

The encoder is the library's bidirectional LSTM on padded rows of different
lengths (rnn_forward). The block is

    h = gated_scan(project(layer_norm(x)))
    s = x + project(h)
    y = s + project(cross_attention(project(layer_norm(s)), encoder states))

trained on whole sequences (layer_norm_train, gated_scan_train,
cross_attention_train and their backward calls) and then run token by token,
with the scan's state carried from call to call and the encoder's keys and
values projected once.

    python examples/decoder_block.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gru_sequence_scan_amd as gss  # noqa: E402


class DecoderBlock:
    """Weights of one block and its three ways to run: train, backward, step."""

    def __init__(self, width, enc_width, heads, kv_heads, dtype=torch.bfloat16, device="cuda:0", seed=0):
        g = torch.Generator().manual_seed(seed)
        self.heads, self.kv_heads, self.D = heads, kv_heads, width // heads

        def mat(n, m):
            return (torch.randn(n, m, generator=g) * n ** -0.5).to(device=device, dtype=dtype)

        self.w = {
            "scan": mat(width, 2 * width), "out": mat(width, width), "q": mat(width, heads * self.D),
            "kv": mat(enc_width, 2 * kv_heads * self.D), "mix": mat(heads * self.D, width),
            "norm1": torch.ones(width, device=device, dtype=dtype), "bias1": torch.zeros(width, device=device, dtype=dtype),
            "norm2": torch.ones(width, device=device, dtype=dtype), "bias2": torch.zeros(width, device=device, dtype=dtype),
        }

    def keys_values(self, enc):
        """The encoder states' keys and values, [S, B, 2, kv_heads, D]."""
        return (enc @ self.w["kv"]).view(*enc.shape[:2], 2, self.kv_heads, self.D)

    def train(self, x, enc, lengths):
        """y [T, B, width] of x [T, B, width], and what backward needs."""
        w, (T, B, H) = self.w, x.shape
        (n1, _), c1 = gss.layer_norm_train(x, w["norm1"], w["bias1"])
        p = (n1 @ w["scan"]).view(T, B, 2, H)
        (h, _), c2 = gss.gated_scan_train(p[:, :, 0], p[:, :, 1])
        (n2, s), c3 = gss.layer_norm_train(h @ w["out"], w["norm2"], w["bias2"], residual=x)
        q = (n2 @ w["q"]).view(T, B, self.heads, self.D)
        kv = self.keys_values(enc)
        a, c4 = gss.cross_attention_train(q, kv[:, :, 0], kv[:, :, 1], lengths=lengths)
        y = s + a.view(T, B, -1) @ w["mix"]
        return y, (n1, c1, h, c2, n2, c3, a, c4, enc)

    def backward(self, saved, dy):
        """Gradients of the weights, of x and of the encoder's states."""
        n1, c1, h, c2, n2, c3, a, c4, enc = saved
        w, (T, B, H) = self.w, dy.shape

        def rows(t):
            return t.reshape(T * B, -1)

        g = {"mix": rows(a).t() @ rows(dy)}
        dq, dk, dv = gss.cross_attention_backward(c4, (dy @ w["mix"].t()).view(a.shape))
        dkv = torch.stack([dk, dv], 2).view(*enc.shape[:2], -1)
        g["kv"] = enc.reshape(-1, enc.shape[-1]).t() @ dkv.reshape(-1, dkv.shape[-1])
        g["q"] = rows(n2).t() @ rows(dq)
        ds, g["norm2"], g["bias2"] = gss.layer_norm_backward(c3, dq.view(T, B, -1) @ w["q"].t(), dy)
        g["out"] = rows(h).t() @ rows(ds)
        dx, df, _, _ = gss.gated_scan_backward(c2, ds @ w["out"].t())
        dp = torch.stack([dx, df], 2).view(T, B, 2 * H)
        g["scan"] = rows(n1).t() @ rows(dp)
        dx, g["norm1"], g["bias1"] = gss.layer_norm_backward(c1, dp @ w["scan"].t(), ds)
        return g, dx, dkv @ w["kv"].t()

    def step(self, x, state, kv, lengths):
        """One token: x [1, B, width], the scan's fp32 state [B, width] (None
        at the start) -> y [1, B, width] and the next state."""
        w, (_, B, H) = self.w, x.shape
        p = (gss.layer_norm(x, w["norm1"], w["bias1"]) @ w["scan"]).view(1, B, 2, H)
        h, state = gss.gated_scan(p[:, :, 0], p[:, :, 1], h0=state)
        n2, s = gss.layer_norm(h @ w["out"], w["norm2"], w["bias2"], residual=x)
        q = (n2 @ w["q"]).view(1, B, self.heads, self.D)
        a = gss.cross_attention(q, kv[:, :, 0], kv[:, :, 1], lengths=lengths)
        return s + a.view(1, B, -1) @ w["mix"], state


def encoder(batch, steps, width, hidden, lengths, dtype, device="cuda:0", seed=1):
    """States [steps, batch, 2 hidden] of a bidirectional LSTM over rows of
    the given lengths."""
    g = torch.Generator().manual_seed(seed)

    def draw(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g) * scale).to(device=device, dtype=dtype)

    params = [{"w_ih": draw(4 * hidden, width, scale=width ** -0.5), "w_hh": draw(4 * hidden, hidden, scale=hidden ** -0.5),
               "b_ih": draw(4 * hidden, scale=0.1), "b_hh": draw(4 * hidden, scale=0.1)} for _ in range(2)]
    x = draw(steps, batch, width)
    y = torch.zeros(steps, batch, 2 * hidden, device=device, dtype=dtype)  # positions past a row's end stay as they are
    gss.rnn_forward("lstm", x, params, lengths=lengths, bidirectional=True, y_out=y)
    return y


def main(T=48, B=6, S=40, width=128, hidden=64, heads=4, kv_heads=2, dtype=torch.bfloat16, epochs=12):
    lengths = [S - 5 * b for b in range(B)]
    enc = encoder(B, S, 32, hidden, lengths, dtype)
    lens = torch.tensor(lengths, dtype=torch.int32, device=enc.device)
    block = DecoderBlock(width, 2 * hidden, heads, kv_heads, dtype)
    g = torch.Generator().manual_seed(7)
    x = torch.randn(T, B, width, generator=g).to(device=enc.device, dtype=dtype)
    target = torch.randn(T, B, width, generator=g).to(device=enc.device, dtype=dtype)
    losses = []
    for _ in range(epochs):
        y, saved = block.train(x, enc, lens)
        diff = y.float() - target.float()
        losses.append(float((diff * diff).mean()))
        grads, _, _ = block.backward(saved, (diff * (2.0 / B)).to(dtype))
        for name, v in block.w.items():
            v -= (0.004 * grads[name].float() / T).to(dtype)
    # the same outputs token by token
    y, _ = block.train(x, enc, lens)
    kv, state, out = block.keys_values(enc), None, []
    for t in range(T):
        one, state = block.step(x[t:t + 1], state, kv, lens)
        out.append(one)
    apart = float((torch.cat(out).float() - y.float()).abs().max())
    return losses, apart


if __name__ == "__main__":
    losses, apart = main()
    print("loss " + " ".join(f"{v:.4f}" for v in losses))
    print(f"token by token, largest difference from the whole run: {apart:.4f}")
