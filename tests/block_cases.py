"""Inputs and comparison shared by the tests of the operators around the sequence layer."""
from __future__ import annotations

import math

import torch

KINDS = {"bf16": torch.bfloat16, "f32": torch.float32}


def half_step(dtype) -> float:
    return 0.0 if dtype == torch.float64 else torch.finfo(dtype).eps / 2


def close(name, got, want, bound):
    """|got - want| <= the float32 bound and half a step of got's type; not finite only where want is not."""
    assert got.shape == want.shape, f"{name}: {tuple(got.shape)} instead of {tuple(want.shape)}"
    step = half_step(got.dtype) if got.dtype != torch.float32 else 0.0  # fp32's last rounding is in the bound
    g = got.detach().to("cpu", torch.float64)
    if g.numel() == 0:
        return
    assert torch.isfinite(g).all(), f"{name}: not finite"
    excess = (g - want).abs() - bound * (1 + step) - step * want.abs() - 1e-37
    i = int(excess.argmax())
    assert excess.max() <= 0, (f"{name}: off by {float((g - want).abs().flatten()[i]):.3e} at {i} of {g.numel()}, "
                               f"value {float(want.flatten()[i]):.3e}, bound {float(bound.flatten()[i]):.3e}")


def normal(gen, *shape, std=1.0):
    return torch.randn(shape, generator=gen) * std


def lengths_for(B, T, gen):
    """One full sequence, one empty where there are more than two, the rest anywhere between."""
    n = torch.randint(0, T + 1, (B,), generator=gen, dtype=torch.int32)
    n[0] = T
    if B > 2:
        n[B // 2] = 0
    return n


def slice_of(t, before, after, fill=float("nan")):
    """t as a slice of wider rows whose other elements must not be read."""
    B, T, C = t.shape
    wide = torch.full((B, T, before + C + after), fill, dtype=t.dtype)
    wide[..., before:before + C] = t
    return wide, (Ellipsis, slice(before, before + C))


def ssm_inputs(B, T, C, N, kind, seed, softplus=True):
    """Inputs of the scan as a layer has them: steps between 1e-3 and 0.1, decays of -1 to -N."""
    g = torch.Generator().manual_seed(seed)
    ty = KINDS[kind]
    u = normal(g, B, T, C)
    step = torch.exp(torch.rand(C, generator=g) * (math.log(0.1) - math.log(1e-3)) + math.log(1e-3))
    dt = normal(g, B, T, C, std=0.5)
    bias = step + torch.log(-torch.expm1(-step))
    if not softplus:
        dt, bias = 0.1 * dt.abs(), step
    return dict(u=(u * torch.sigmoid(u)).to(ty), dt=dt.to(ty),
                A=-torch.arange(1, N + 1).float() * torch.exp(normal(g, C, N, std=0.1)),
                Bm=normal(g, B, T, N).to(ty), Cm=normal(g, B, T, N).to(ty), D=1 + normal(g, C, std=0.1),
                z=normal(g, B, T, C).to(ty), dt_bias=bias, h0=normal(g, B, C, N))


def cuda(d):
    return {k: None if v is None else v.cuda() for k, v in d.items()}
