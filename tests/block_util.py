"""Tolerances and tensors shared by the tests of the decoder block's
operators."""

import numpy as np
import torch

# fp32: sums of up to a few thousand products of fp32-rounded factors, gates
# from hardware exp2 and reciprocal (1 ulp each): 1e-5 of the tensor's largest
# value and 1e-4 of the element, as for the recurrences. bf16 storage: one
# rounding to nearest at the end, half an ulp = up to 2^-8 of the element (8 significant bits), on top of
# the fp32 part.
F32_REL, F32_SCALE = 1e-4, 1e-5
BF16_HALF_ULP = 2.0 ** -8


def assert_near(got, ref, dtype, what, extra=0.0):
    """|got - ref| within the above; `extra`: a further absolute bound per
    element (a number or an array) that the caller derives."""
    got = got.detach().float().cpu().numpy().astype(np.float64) if isinstance(got, torch.Tensor) else got
    ref = np.asarray(ref, dtype=np.float64)
    assert got.shape == ref.shape, f"{what}: shape {got.shape} != {ref.shape}"
    if ref.size == 0:
        return
    assert np.isfinite(got).all(), f"{what}: non-finite values"
    limit = F32_REL * np.abs(ref) + F32_SCALE * max(float(np.abs(ref).max()), 1e-30) + extra
    if dtype == torch.bfloat16:
        limit = limit + BF16_HALF_ULP * (np.abs(ref) + limit)
    err = np.abs(got - ref)
    bad = err > limit
    at = np.unravel_index(int((err - limit).argmax()), ref.shape)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {ref.size} elements off, worst at {at}: "
                           f"{got[at]:.6g} for {ref[at]:.6g} (limit {np.broadcast_to(limit, ref.shape)[at]:.3g})")


def draw(rng, shape, dtype, scale=1.0, mean=0.0):
    """A seeded CPU tensor of the storage type; its values are what both
    sides read."""
    return torch.from_numpy((rng.standard_normal(shape) * scale + mean).astype(np.float32)).to(dtype)


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def strided(t, pad_value=float("nan")):
    """t's values on the GPU in a wider buffer (rows apart, NaN between): the
    last dimension stays contiguous."""
    wide = torch.full(t.shape[:-1] + (t.shape[-1] + 24,), pad_value, dtype=t.dtype)
    wide[..., 8:8 + t.shape[-1]] = t
    return wide.cuda()[..., 8:8 + t.shape[-1]]


def shifted(t):
    """t's values on the GPU one element off every vector alignment."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    out = flat[1:].view(t.shape)
    out.copy_(t)
    return out
