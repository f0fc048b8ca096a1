"""A state-space block: trained on whole sequences, then run on a prompt and
token by token.

    p, z = project(layer_norm(x))
    c = silu(causal_conv(p));  dt, B, C = project(c)
    s = x + project(selective_scan(c, dt, A, B, C, D) * silu(z))
    y = s + feed_forward(layer_norm(s))

Rows may have different lengths. Serving carries two states a row: the last
inputs of the convolution and the scan's fp32 state.

    python examples/state_space_block.py
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gru_sequence_scan_amd as gss  # noqa: E402


class StateSpaceBlock:
    """Weights of one block and its ways to run: train, backward, step (a
    prompt or a single token)."""

    def __init__(self, width, inner, state, taps, hidden, groups=1, dtype=torch.bfloat16, device="cuda:0", seed=0):
        g = torch.Generator().manual_seed(seed)
        self.width, self.inner, self.N, self.G = width, inner, state, groups

        def mat(n, m, scale=None):  # [out, in], as the library's weights are
            return (torch.randn(n, m, generator=g) * (m ** -0.5 if scale is None else scale)).to(device=device, dtype=dtype)

        def f32(t):
            return t.to(device=device, dtype=torch.float32)

        step = torch.exp(torch.rand(inner, generator=g) * 4.6 - 6.9)  # 0.001 to 0.1
        self.w = {
            "in": mat(2 * inner, width), "conv": mat(inner, taps, taps ** -0.5), "conv_bias": mat(1, inner, 0.1)[0],
            "bc": mat(2 * groups * state, inner), "dt": mat(inner, inner, 0.1 * inner ** -0.5), "out": mat(width, inner),
            "ff_in": mat(2 * hidden, width), "ff_out": mat(width, hidden),
            "norm1": torch.ones(width, device=device, dtype=dtype), "norm2": torch.ones(width, device=device, dtype=dtype),
            "A": f32(-torch.arange(1, state + 1).float().expand(inner, state).contiguous()),
            "D": f32(torch.ones(inner)), "dt_bias": f32(step + torch.log(-torch.expm1(-step))),
        }

    def _project(self, x, conv):
        """The scan's inputs but x: dt, B, C and the gate, given the projected
        input p, z and the convolved branch."""
        T, B, _ = x.shape
        bc = (conv @ self.w["bc"].t()).view(T, B, 2, self.G, self.N)
        return conv @ self.w["dt"].t(), bc

    def train(self, x, lengths=None):
        """y [T, B, width] of x, and what backward needs."""
        w, (T, B, _) = self.w, x.shape
        (n1, _), c1 = gss.layer_norm_train(x, w["norm1"])
        pz = (n1 @ w["in"].t()).view(T, B, 2, self.inner)
        (c, _), c2 = gss.causal_conv_train(pz[:, :, 0], w["conv"], w["conv_bias"], lengths=lengths, activation="silu")
        dt, bc = self._project(x, c)
        (h, _), c3 = gss.selective_scan_train(c, dt, w["A"], bc[:, :, 0], bc[:, :, 1], w["D"], z=pz[:, :, 1],
                                              dt_bias=w["dt_bias"], lengths=lengths)
        (n2, s), c4 = gss.layer_norm_train(h @ w["out"].t(), w["norm2"], residual=x)
        y, c5 = gss.feed_forward_train(n2, w["ff_in"], w["ff_out"], residual=s)
        return y, (n1, c1, c2, c, dt, bc, c3, h, c4, c5)

    def backward(self, saved, dy):
        """Gradients of the weights and of x."""
        n1, c1, c2, c, dt, bc, c3, h, c4, c5 = saved
        w, (T, B, _) = self.w, dy.shape
        g = {}

        def rows(t):
            return t.reshape(T * B, -1)

        dn2, g["ff_in"], g["ff_out"] = gss.feed_forward_backward(c5, dy)
        ds, g["norm2"], _ = gss.layer_norm_backward(c4, dn2, dy)
        g["out"] = rows(ds).t() @ rows(h)
        d = gss.selective_scan_backward(c3, ds @ w["out"])
        g["A"], g["D"], g["dt_bias"] = d["A"], d["D"], d["dt_bias"]
        dbc = torch.stack([d["B"], d["C"]], 2).view(T, B, -1)
        g["bc"], g["dt"] = rows(dbc).t() @ rows(c), rows(d["dt"]).t() @ rows(c)
        dp, g["conv"], g["conv_bias"], _ = gss.causal_conv_backward(c2, d["x"] + dbc @ w["bc"] + d["dt"] @ w["dt"])
        dpz = torch.stack([dp, d["z"]], 2).view(T, B, -1)
        g["in"] = rows(dpz).t() @ rows(n1)
        dx, g["norm1"], _ = gss.layer_norm_backward(c1, dpz @ w["in"], ds)
        return g, dx

    def step(self, x, states=(None, None), lengths=None):
        """A prompt or one token, x [T, B, width]: y and the two states to go on with."""
        w, (T, B, _) = self.w, x.shape
        pz = (gss.layer_norm(x, w["norm1"]) @ w["in"].t()).view(T, B, 2, self.inner)
        c, last = gss.causal_conv(pz[:, :, 0], w["conv"], w["conv_bias"], state=states[0], lengths=lengths, activation="silu")
        dt, bc = self._project(x, c)
        h, state = gss.selective_scan(c, dt, w["A"], bc[:, :, 0], bc[:, :, 1], w["D"], z=pz[:, :, 1], dt_bias=w["dt_bias"],
                                      h0=states[1], lengths=lengths)
        n2, s = gss.layer_norm(h @ w["out"].t(), w["norm2"], residual=x)
        return gss.feed_forward(n2, w["ff_in"], w["ff_out"], residual=s), (last, state)


def main(T=64, B=4, width=64, inner=128, state=16, taps=4, hidden=160, dtype=torch.bfloat16, epochs=10):
    block = StateSpaceBlock(width, inner, state, taps, hidden, dtype=dtype)
    dev = block.w["in"].device
    lengths = torch.tensor([T - 9 * b for b in range(B)], dtype=torch.int32, device=dev)
    live = (torch.arange(T, device=dev)[:, None] < lengths[None])[:, :, None]
    g = torch.Generator().manual_seed(7)
    x = torch.randn(T, B, width, generator=g).to(device=dev, dtype=dtype)
    target = torch.randn(T, B, width, generator=g).to(device=dev, dtype=dtype)
    losses = []
    for _ in range(epochs):
        y, saved = block.train(x, lengths)
        diff = (y.float() - target.float()) * live
        losses.append(float((diff * diff).mean()))
        grads, _ = block.backward(saved, (diff * (2.0 / B)).to(dtype))
        for name, v in block.w.items():
            v -= (0.002 * grads[name].float() / T).to(v.dtype)
    # the same outputs from a prompt of half the steps and one token at a time
    y, _ = block.train(x, lengths)
    half = T // 2
    out, states = block.step(x[:half], lengths=lengths.clamp(max=half))
    out = [out]
    for t in range(half, T):
        one, states = block.step(x[t:t + 1], states, lengths=(lengths - t).clamp(0, 1))
        out.append(one)
    apart = float((((torch.cat(out).float() - y.float()) * live).abs()).max())
    return losses, apart


if __name__ == "__main__":
    losses, apart = main()
    print("loss " + " ".join(f"{v:.4f}" for v in losses))
    print(f"prompt and tokens, largest difference from the whole run: {apart:.4f}")
