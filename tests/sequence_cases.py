"""Inputs of the sequence and adapter tests, and how their results are compared."""
from __future__ import annotations

import torch

from parity import say

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(lens, D, *, dtype="f32", cpw=1, lam=True, u=True, h0=True, pad=0, seed=0, spread=2.0):
    """CPU tensors of packed sequences, rounded to dtype; gates from -spread to 6 + spread or so."""
    g = torch.Generator().manual_seed(seed)
    T, dt = sum(lens) + pad, DT[dtype]
    rn = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    ru = lambda *s: torch.rand(*s, generator=g)    # noqa: E731
    return dict(x=rn(T, D).to(dt), gate=(spread * rn(T, D // cpw) + 6 * ru(D // cpw)).to(dt),
                lam=ru(T, D).to(dt) if lam else None, u=ru(T, D).to(dt) if u else None,
                h0=rn(len(lens), D) if h0 else None, lens=list(lens), cpw=cpw, gy=rn(T, D).to(dt),
                gh=rn(len(lens), D), pad=pad)


def offsets_of(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32)


def up(t, dev="cuda"):
    return None if t is None else t.to(dev)


def close(name, got, want, bound):
    got = got.detach().double().cpu()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{name} is not finite"
    over = (got - want).abs() - bound
    worst = float(over.max()) if over.numel() else 0.0
    ratio = float(((got - want).abs() / bound.clamp_min(1e-300)).max()) if over.numel() else 0.0
    say(f"  {name}: largest error is {ratio:.3f} of its bound")
    assert worst <= 0, f"{name}: off by {worst:.3e} more than its bound (at most {float(bound.max()):.3e})"


def strided(t, extra=5):
    """The same rows, further apart: a column range of a wider tensor."""
    if t is None:
        return None
    wide = torch.full(t.shape[:-1] + (t.shape[-1] + 2 * extra,), float("nan"), dtype=t.dtype, device=t.device)
    wide[..., extra:extra + t.shape[-1]] = t
    return wide[..., extra:extra + t.shape[-1]]
