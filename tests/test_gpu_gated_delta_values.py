"""Gated delta rule on the GPU: values that are not finite, and how exact the
decays and the fp32 outputs are."""
import pytest
import torch

import gated_delta_cases as gd
from mlstm_chunkwise_b200 import _lib, api

pytestmark = pytest.mark.gpu

# (algorithm, batch, heads, tokens, the token's chunk length): the fp32 path, the
# staged tensor-core forward, and the fused one (many heads; one chunk)
PATHS = [("simt", 1, 2, 300, 64), ("tc", 1, 2, 700, 128), ("tc", 40, 4, 300, 128),
         ("tc", 2, 2, 100, 128)]


@pytest.mark.parametrize("algo,B,NH,T,L", PATHS, ids=str)
def test_nan_gate_is_no_reset(algo, B, NH, T, L):
    """A NaN in one head's g: that head's outputs from the token on and its final
    state are NaN, gradients too; chunks before and other heads keep their bits."""
    x = gd.cuda(gd.make(B=B, NHK=NH, NH=NH, T=T, DK=64, DV=72))
    dH = torch.randn_like(x["V"])

    def both():
        H, C = api.gated_delta_fw(*(x[n] for n in gd.NAMES), algo=algo)
        return H, C, api.gated_delta_bw(*(x[n] for n in gd.NAMES[:5]), dH, x["C0"], algo=algo)

    H, C, d = both()
    t = T - T // 4
    x["g"][0, 1, t] = float("nan")
    H2, C2, d2 = both()
    torch.cuda.synchronize()
    assert api.last_device_error() == _lib.OK
    assert H2[0, 1, t:].isnan().all() and C2[0, 1].isnan().all()
    assert torch.equal(H2[0, 1, :t // L * L], H[0, 1, :t // L * L])
    for n in ("dg", "dbeta", "dQ", "dK"):
        assert d2[n][0, 1, t].isnan().all(), n
    others = torch.ones(B, NH, dtype=torch.bool)
    others[0, 1] = False
    for a, b in ((H, H2), (C, C2), *((d[n], d2[n]) for n in d)):
        assert torch.equal(a[others], b[others])


@pytest.mark.parametrize("DV", [64, 7])
def test_nan_gate_in_a_step(DV):
    x = gd.cuda(gd.make(NHK=2, NH=2, T=1, DK=64, DV=DV))
    tok = [x[n][:, :, 0].contiguous() for n in gd.NAMES[:5]]
    C, C2 = x["C0"].clone(), x["C0"].clone()
    h = api.gated_delta_step(*tok, C)
    tok[3][0, 1] = float("nan")
    h2 = api.gated_delta_step(*tok, C2)
    assert C2[0, 1].isnan().all() and h2[0, 1].isnan().all()
    assert torch.equal(C[0, 0], C2[0, 0]) and torch.equal(h[0, 0], h2[0, 0])


def kept(**kw):
    """Leaves, the output of a call that keeps its inputs, and its initial state
    as a tensor of the caller's own."""
    d = {n: v.requires_grad_() for n, v in gd.cuda(gd.make(T=80, **kw)).items()}
    state = d["C0"].detach()
    H, _ = api.gated_delta_chunkwise(*(d[n] for n in gd.NAMES), recompute=True)
    return d, state, H


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_autograd_sees_writes_in_place(dtype):
    """A state that a later call overwrites is not used for gradients."""
    modified = pytest.raises(RuntimeError, match="modified by an inplace operation")
    d, state, H = kept(dtype=dtype)
    tok = [d[n].detach()[:, :, 0].contiguous() for n in gd.NAMES[:5]]
    api.gated_delta_step(*tok, state)
    with modified:
        H.float().sum().backward()
    d, state, H = kept(dtype=dtype)
    api.gated_delta_fw(*(d[n].detach() for n in gd.NAMES), out={"C_T": state})
    with modified:
        H.float().sum().backward()
    d, state, H = kept(dtype=dtype)
    api.gated_delta_fw(*(d[n].detach() for n in gd.NAMES), out={"H": d["V"].detach().clone()})
    H.float().sum().backward()  # nothing that was kept


def test_outputs_given_by_the_caller_are_marked():
    x = gd.cuda(gd.make(T=80))
    H, h = torch.empty_like(x["V"]), torch.empty_like(x["V"][:, :, 0])
    Y = torch.empty(1, 80, 2 * 64, dtype=torch.bfloat16, device="cuda")
    api.gated_delta_fw(*(x[n] for n in gd.NAMES), out={"H": H}, return_last_state=False)
    api.gated_delta_step(*(x[n][:, :, 0].contiguous() for n in gd.NAMES[:5]), x["C0"], h=h)
    api.head_norm_fw(H, torch.ones(2, 64, device="cuda"), out=Y)
    assert [t._version for t in (H, h, x["C0"], Y)] == [1, 1, 1, 1]
    with torch.inference_mode():
        C = x["C0"].clone()  # tensors without a version
        api.gated_delta_step(*(x[n][:, :, 0].contiguous() for n in gd.NAMES[:5]), C)


def test_no_training_forward_where_nothing_is_differentiated():
    """Under no_grad, with a state that requires a gradient (and with no such
    input), the call is gated_delta_fw: its bits and its launches."""
    x = gd.cuda(gd.make(B=40, NHK=4, NH=4, T=300))
    launches = _lib.lib().mlstm_kernel_launches

    def count(call):
        n = launches()
        return call(), launches() - n

    want, n = count(lambda: api.gated_delta_fw(*(x[m] for m in gd.NAMES)))
    plain = count(lambda: api.gated_delta_chunkwise(*(x[m] for m in gd.NAMES)))
    x["C0"].requires_grad_()
    with torch.no_grad():
        off = count(lambda: api.gated_delta_chunkwise(*(x[m] for m in gd.NAMES)))
    for got, k in (plain, off):
        assert k == n and all(torch.equal(a, b) for a, b in zip(got, want))
        assert not any(t.requires_grad for t in got)
    got, k = count(lambda: api.gated_delta_chunkwise(*(x[m] for m in gd.NAMES)))
    assert k > n and all(t.requires_grad for t in got)


@pytest.mark.parametrize("decay", [2.0, 15.0, 31.0, 44.0, 56.0, 75.0])
def test_decays_of_neighbours(decay):
    """e^{g_{s+1}} as dbeta_s alone shows it: keys are the unit vectors, so that y
    is V, and each query is the key before, so that
        dbeta_s = e^{g_{s+1}} dH_{s+1}.v_s
    with an exact integer behind the decay.  `decay` is that of 32 tokens: up to 60
    Gam is the product of two factors, of which the larger is e^decay.  Two
    exponentials and a quotient, each off by 2^-22, and eight roundings of 2^-24:
    3 x 2^-22 + 8 x 2^-24 = 1.2e-6."""
    T = DK = 128
    gen = torch.Generator().manual_seed(int(decay))
    g = -decay / 32 * (0.5 + torch.rand(1, 1, T, generator=gen))
    g = g * (decay / 32) / -g.mean()
    eye = torch.eye(T).view(1, 1, T, DK)
    V, dH = (torch.randint(-4, 5, (1, 1, T, 64), generator=gen).float() for _ in range(2))
    x = {"Q": eye.roll(1, 2), "K": eye, "V": V, "g": g, "beta": torch.rand(1, 1, T, generator=gen)}
    d = {n: (v if n in ("g", "beta") else v.bfloat16()).contiguous().cuda() for n, v in x.items()}
    got = api.gated_delta_bw(*d.values(), dH.bfloat16().cuda(), scale=1.0, algo="tc")["dbeta"]
    dots = (dH[:, :, 1:] * V[:, :, :-1]).sum(-1).double()
    want = torch.exp(g[:, :, 1:].double()) * dots
    err = (got[0, 0, :-1].double().cpu() - want[0, 0]).abs() / want[0, 0].abs().clamp(min=1e-300)
    # token 0's query is the last token's key, which it does not see
    assert float(err[dots[0, 0] != 0].max()) < 1.2e-6
    assert not got[0, 0, :-1].cpu()[dots[0, 0] == 0].any() and got[0, 0, -1] == 0


@pytest.mark.parametrize("B,T", [(1, 128), (60, 300), (1, 640)], ids=str)
def test_the_final_state_keeps_24_bits_of_what_is_written(B, T):
    """With unit vectors as keys y is V, and row t of the final state is
    D_t beta_t v_t: the decay (2^-22), the last operand of the state's product in
    three terms (2^-24), and the products and sums around it (twelve of 2^-24):
    2^-22 + 13 x 2^-24 < 2^-19.  On the fused forward (one chunk; many heads) and the
    staged one (640 tokens of one head); a reset in front of the last 128 tokens
    makes them a sequence of their own."""
    L = DK = 128
    gen = torch.Generator().manual_seed(3)
    g = -0.02 * torch.rand(B, 1, T, generator=gen)
    beta = torch.rand(B, 1, T, generator=gen)
    t0 = (T - 1) // L * L
    if t0:
        g[:, :, t0] = float("-inf")
    V = torch.randint(-9, 10, (B, 1, T, 72), generator=gen).float()
    K = torch.eye(L)[torch.arange(T) % L].expand(B, 1, T, DK)
    x = [t.contiguous().bfloat16().cuda() for t in (K, K, V)]
    _, C = api.gated_delta_fw(*x, g.cuda(), beta.cuda(), algo="tc")
    G, n = g[:, :, t0:].double(), T - t0
    if t0:
        G[:, :, 0] = 0.0
    D = torch.exp(G.flip(-1).cumsum(-1).flip(-1) - G)  # the decays behind each token
    want = (D * beta[:, :, t0:].double())[..., None] * V[:, :, t0:].double()
    C = C.double().cpu()
    assert not C[:, :, n:].any()
    err = (C[:, :, :n] - want).abs() / want.abs().clamp(min=1e-300)
    assert float(err[want != 0].max()) < 2.0 ** -19
    assert not C[:, :, :n][want == 0].any()


@pytest.mark.parametrize("algo,B,NH,T,L", PATHS, ids=str)
@pytest.mark.parametrize("stale", [float("nan"), float("inf")])
def test_reset_at_the_first_token_forgets_any_state(algo, B, NH, T, L, stale):
    """A slot whose last sequence left infinities or NaN: a new sequence that starts
    with a reset has the bits of one that starts from zeros."""
    x = gd.cuda(gd.make(B=B, NHK=NH, NH=NH, T=T, DK=64, DV=72))
    x["g"][0, 1, 0] = float("-inf")
    dH, dC = torch.randn_like(x["V"]), torch.randn_like(x["C0"])

    def both():
        d = api.gated_delta_bw(*(x[n] for n in gd.NAMES[:5]), dH, x["C0"], dC, algo=algo)
        return (*api.gated_delta_fw(*(x[n] for n in gd.NAMES), algo=algo), *d.values())

    x["C0"][0, 1] = 0.0
    want = both()
    x["C0"][0, 1] = stale
    got = both()
    assert torch.isfinite(got[0]).all() and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("DK,DV", [(64, 64), (33, 7), (256, 40), (1024, 6)])
def test_reset_in_a_step_forgets_any_state(DK, DV):
    x = gd.cuda(gd.make(NHK=2, NH=2, T=1, DK=DK, DV=DV))
    tok = [x[n][:, :, 0].contiguous() for n in gd.NAMES[:5]]
    tok[3][0, 1] = float("-inf")
    C = [x["C0"].clone(), x["C0"].clone()]
    C[0][0, 1], C[1][0, 1] = 0.0, float("nan")
    C[1][0, 1, ::2] = float("inf")
    h = [api.gated_delta_step(*tok, c) for c in C]
    assert torch.isfinite(h[1]).all() and torch.equal(*h) and torch.equal(*C)
