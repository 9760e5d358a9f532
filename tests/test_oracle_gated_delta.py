"""The gated delta rule's fp64 reference against its definition's corner cases,
an independent chunkwise restatement and finite differences (CPU)."""
import torch

import gated_delta_cases as gd
from oracle import gated_delta as ref


def test_first_token_and_no_write():
    x = gd.fp64(gd.make(T=3, dtype="f32", init=False))
    H, C = ref.forward(**x)
    k, v, q, b = (x[n][:, :, 0] for n in ("K", "V", "Q", "beta"))
    want = (k * q).sum(-1, keepdim=True) * b[..., None] * v * 64 ** -0.5
    assert torch.allclose(H[:, :, 0], want, atol=1e-14)
    x = gd.fp64(gd.make(T=5, dtype="f32"))
    x["g"].zero_(), x["beta"].zero_()
    assert torch.equal(ref.forward(**x)[1], x["C0"])


def test_beta_one_stores_the_value_at_a_unit_key():
    """With beta = 1 and a unit key the write replaces what the key held:
    C_T^T k = v of the last token exactly."""
    x = gd.fp64(gd.make(T=40, dtype="f32"))
    x["K"] = x["K"] / x["K"].norm(dim=-1, keepdim=True)
    x["beta"].fill_(1.0)
    _, C = ref.forward(**x)
    got = torch.einsum("bhkv,bhk->bhv", C, x["K"][:, :, -1])
    assert torch.allclose(got, x["V"][:, :, -1], atol=1e-12)


def test_chunkwise_restatement():
    """The chunk formulas of csrc/gdn.h, written with dense matrices."""
    x = gd.fp64(gd.make(B=1, NHK=1, NH=1, T=48, DK=16, DV=8, dtype="f32", gates="strong"))
    H, C_T = ref.forward(**x)
    C, out, L = x["C0"][0, 0], [], 16
    for t0 in range(0, 48, L):
        Q, K, V = (x[n][0, 0, t0:t0 + L] for n in ("Q", "K", "V"))
        gc, b = x["g"][0, 0, t0:t0 + L].cumsum(0), x["beta"][0, 0, t0:t0 + L]
        gam = torch.exp(gc[:, None] - gc[None, :]).tril()
        A = (gam * (K @ K.T) * b).tril(-1)
        y = torch.linalg.solve(torch.eye(L, dtype=A.dtype) + A, V - gc.exp()[:, None] * (K @ C))
        out.append(0.25 * (gc.exp()[:, None] * (Q @ C) + (gam * (Q @ K.T) * b) @ y))
        C = gc[-1].exp() * C + K.T @ ((gc[-1] - gc).exp()[:, None] * b[:, None] * y)
    assert torch.allclose(torch.cat(out), H[0, 0], atol=1e-12)
    assert torch.allclose(C, C_T[0, 0], atol=1e-12)


def test_gradients_against_differences():
    x = gd.make(B=1, NHK=1, NH=2, T=7, DK=4, DV=3, dtype="f32", seed=3)
    gen = torch.Generator().manual_seed(5)
    dH = torch.randn(1, 2, 7, 3, generator=gen).double()
    dC = torch.randn(1, 2, 4, 3, generator=gen).double()
    grads = ref.gradients(x, dH, dC)
    x = gd.fp64(x)

    def loss():
        H, C = ref.forward(**x)
        return float((H * dH).sum() + (C * dC).sum())

    for n in gd.NAMES:
        flat = x[n].view(-1)
        for i in range(0, flat.numel(), 5):
            keep, e = float(flat[i]), 1e-5
            flat[i] = keep + e
            up = loss()
            flat[i] = keep - e
            down = loss()
            flat[i] = keep
            want = (up - down) / (2 * e)  # error O(e^2) + 1e-16 / e
            assert abs(float(grads["d" + n].view(-1)[i]) - want) < 1e-7 * max(1.0, abs(want))
