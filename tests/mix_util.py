"""Helpers shared by the tests of the sequence mixers: inputs, comparison."""
from __future__ import annotations

import torch

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def gen(seed):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    return g


def normal(g, *shape, dtype=torch.float32, scale=1.0, shift=0.0):
    """Seeded N(shift, scale^2) values on the GPU, rounded to dtype."""
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype).cuda()


def leaf(t):
    """A float64 copy on the CPU that collects a gradient."""
    return None if t is None else t.detach().cpu().double().requires_grad_(True)


def half_step(dtype):
    """Half a step of a type, relative: what one rounding is off by at most."""
    return torch.finfo(dtype).eps / 2


def check(got, ref, mag, what, steps=16.0, weights=0.0):
    """|got - ref| <= half_step(dtype) |ref| + (steps 2^-24 + weights) mag.

    ref: the exact value in 64 bits.  mag: what it is a sum of, in absolute
    values.  steps: float32 half steps the computation may lose relative to
    mag; weights: the relative error of weights that are rounded to fewer bits
    before they enter a sum of magnitude mag.
    """
    r = ref.detach().double().cpu()
    g = got.detach().double().cpu()
    assert g.shape == r.shape, f"{what}: {tuple(g.shape)} != {tuple(r.shape)}"
    assert torch.isfinite(g).all(), f"{what}: non-finite output"
    m = mag.detach().double().cpu() if isinstance(mag, torch.Tensor) else mag
    step = half_step(got.dtype)
    tol = step * r.abs() + (steps * 2.0 ** -24 + weights) * (1 + step) * m + 1e-37
    bad = ((g - r).abs() / tol)
    worst = float(bad.max()) if bad.numel() else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3g} times the bound"
    return worst
