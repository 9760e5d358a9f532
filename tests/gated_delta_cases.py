"""Inputs and error metric shared by the gated delta rule tests."""
from __future__ import annotations

import torch

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NAMES = ("Q", "K", "V", "g", "beta", "C0")


def make(B=1, NHK=2, NH=2, T=200, DK=64, DV=64, dtype="bf16", init=True, gates="mild", keys="unit",
         seed=0):
    """CPU inputs.  gates: "mild" decays between almost none and a few tokens;
    "strong" e^g mostly below 0.1; "hold" g = 0; "zero_beta" a third of the
    tokens write nothing (and do not decay); "reset" some g = -inf.  keys:
    "unit" random unit vectors, "alike" nearly the same key every time."""
    gen = torch.Generator().manual_seed(seed)

    def randn(*s):
        return torch.randn(*s, generator=gen)

    q, k = randn(B, NHK, T, DK), randn(B, NHK, T, DK)
    if keys == "alike":
        k = k + 6.0 * randn(B, NHK, 1, DK)
    g = -torch.exp(randn(B, NH, T) - 3.0)
    beta = torch.sigmoid(randn(B, NH, T))
    if gates == "strong":
        g = -torch.exp(randn(B, NH, T) + 1.5)
    elif gates == "hold":
        g = torch.zeros(B, NH, T)
    elif gates == "zero_beta":
        off = torch.rand(B, NH, T, generator=gen) < 0.33
        g, beta = g.masked_fill(off, 0.0), beta.masked_fill(off, 0.0)
    elif gates == "reset":
        g = g.masked_fill(torch.rand(B, NH, T, generator=gen) < 0.03, float("-inf"))
    dt = DT[dtype]
    return {"Q": (q / q.norm(dim=-1, keepdim=True)).to(dt),
            "K": (k / k.norm(dim=-1, keepdim=True)).to(dt), "V": randn(B, NH, T, DV).to(dt),
            "g": g, "beta": beta, "C0": 0.3 * randn(B, NH, DK, DV) if init else None}


def cuda(x):
    return {n: None if v is None else v.cuda() for n, v in x.items()}


def fp64(x):
    return {n: None if v is None else v.double() for n, v in x.items()}


def worst(got, want):
    """max|x - y| / max|y| per (b, head), the worst of them."""
    got, want = got.detach().double().cpu().flatten(2), want.detach().double().flatten(2)
    assert got.shape == want.shape and torch.isfinite(got).all()
    if got.numel() == 0:
        return 0.0
    d, m = (got - want).abs().amax(-1), want.abs().amax(-1)
    return float((d / torch.where(m > 0, m, torch.ones_like(m))).max())
