"""fp64 reference of the gated delta rule (test infrastructure, CPU torch).

The recurrence is written token by token exactly as defined,

    y_t = v_t - e^{g_t} C_{t-1}^T k_t
    C_t = e^{g_t} C_{t-1} + k_t (beta_t y_t)^T
    h_t = scale C_t^T q_t

and the gradients come from torch.autograd on that restatement.  g below -1000
(-inf among it) acts as -1000, as the library documents.
"""
from __future__ import annotations

import torch


def forward(Q, K, V, g, beta, C0=None, scale=None):
    """fp64 tensors in, (H, C_T) out; value head n reads key head n // (NH // NHK)."""
    B, NH, T, DV = V.shape
    NHK, DK = Q.shape[1], Q.shape[3]
    scale = DK ** -0.5 if scale is None else scale
    head = torch.arange(NH) // (NH // NHK)
    Q, K = Q[:, head], K[:, head]
    a = torch.exp(torch.clamp(g, min=-1000.0))
    C = torch.zeros(B, NH, DK, DV, dtype=Q.dtype) if C0 is None else C0
    H = []
    for t in range(T):
        C = a[:, :, t, None, None] * C
        y = V[:, :, t] - torch.einsum("bhkv,bhk->bhv", C, K[:, :, t])
        C = C + torch.einsum("bhk,bhv->bhkv", K[:, :, t], beta[:, :, t, None] * y)
        H.append(scale * torch.einsum("bhkv,bhk->bhv", C, Q[:, :, t]))
    return (torch.stack(H, 2) if H else torch.zeros_like(V)), C


def gradients(x: dict, dH=None, dC_T=None, scale=None) -> dict:
    """Gradients of sum(H * dH) + sum(C_T * dC_T) with respect to every input."""
    x = {n: None if v is None else v.detach().double().cpu().requires_grad_()
         for n, v in x.items()}
    H, C = forward(x["Q"], x["K"], x["V"], x["g"], x["beta"], x["C0"], scale)
    loss = H.sum() * 0 + C.sum() * 0
    if dH is not None:
        loss = loss + (H * dH.double().cpu()).sum()
    if dC_T is not None:
        loss = loss + (C * dC_T.double().cpu()).sum()
    names = [n for n in ("Q", "K", "V", "g", "beta", "C0") if x[n] is not None]
    grads = torch.autograd.grad(loss, [x[n] for n in names])
    return {"d" + n: d for n, d in zip(names, grads)}
