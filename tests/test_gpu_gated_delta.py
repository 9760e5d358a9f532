"""Gated delta rule on the GPU against the fp64 token-by-token reference.

Error metric: per (b, head), max|x - y| / max|y|.  Tolerances, derived:
  fp32 CUDA-core path ("simt"): fp32 sums of at most a few hundred rounded
    terms per output on every path from input to output, 300 x 2^-24 = 1.8e-5;
  tensor-core path ("tc"): the fp32 operands of the products are carried as two
    bf16 terms, each off by at most 2^-16 of its value; up to eight such
    operands lie on the way to an output (state, z, inverse, y of a chunk and
    the same of the reverse recurrence): 8 x 2^-16 = 1.2e-4;
  16-bit outputs add half a step of their type: 2^-8.
"""
import pytest
import torch

import gated_delta_cases as gd
from mlstm_chunkwise_b200 import _lib, api
from oracle import gated_delta as ref

pytestmark = pytest.mark.gpu

F32_TOL = {"simt": 1.8e-5, "tc": 1.2e-4}
ALGOS = ["simt", "tc"]


def tol(algo, out_dtype):
    return F32_TOL[algo] + (2.0 ** -8 if out_dtype == torch.bfloat16 else 0.0)


def check(algo, got, want):
    torch.cuda.synchronize()
    assert api.last_device_error() == _lib.OK
    bad = {}
    for n, w in want.items():
        e = gd.worst(got[n], w)
        if e > tol(algo, got[n].dtype):
            bad[n] = (e, tol(algo, got[n].dtype))
    assert not bad, bad


def run_case(algo, kw, backward=True, scale=None):
    x = gd.make(**kw)
    d = gd.cuda(x)
    H, C_T = api.gated_delta_fw(*(d[n] for n in gd.NAMES), scale=scale, algo=algo)
    H64, C64 = ref.forward(**gd.fp64(x), scale=scale)
    check(algo, {"H": H, "C_T": C_T}, {"H": H64, "C_T": C64})
    if not backward:
        return
    gen = torch.Generator().manual_seed(kw.get("seed", 0) + 1)
    dH = torch.randn(x["V"].shape, generator=gen).to(x["V"].dtype)
    dC = torch.randn(C64.shape, generator=gen)
    want = ref.gradients(x, dH, dC, scale)
    got = api.gated_delta_bw(*(d[n] for n in gd.NAMES[:5]), dH.cuda(), d["C0"], dC.cuda(),
                             scale=scale, algo=algo)
    check(algo, got, want)


def supported(algo, dtype, DK, DV):
    return algo == "simt" or (dtype == "bf16" and DK <= 128 and DK % 8 == 0 and DV % 8 == 0)


SIZES = [
    # B, NHK, NH, T, DK, DV
    (1, 1, 1, 1, 64, 64),
    (2, 1, 2, 2, 128, 128),
    (1, 2, 2, 63, 64, 64),
    (1, 1, 2, 64, 64, 128),
    (1, 2, 2, 65, 96, 64),
    (1, 1, 3, 127, 128, 64),
    (2, 2, 2, 128, 128, 128),
    (1, 1, 2, 129, 128, 256),
    (1, 2, 4, 300, 128, 96),
    (2, 1, 1, 513, 64, 72),
    (1, 1, 1, 700, 8, 8),
    (1, 1, 2, 130, 100, 52),     # no multiples of 8
    (1, 2, 2, 70, 33, 7),
    (1, 1, 1, 100, 256, 512),    # the 7B head
    (1, 1, 1, 66, 1024, 40),     # the widest key
    (1, 1, 2, 200, 64, 512),     # several pairs of value tiles
    (1, 1, 1, 130, 128, 1000),
    (1, 2, 2, 40, 16, 8),
]


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
def test_sizes(algo, dtype, size):
    B, NHK, NH, T, DK, DV = size
    if not supported(algo, dtype, DK, DV):
        pytest.skip("not a shape of this algorithm")
    run_case(algo, dict(B=B, NHK=NHK, NH=NH, T=T, DK=DK, DV=DV, dtype=dtype))


# enough heads for the fused forward at any length (with few heads it runs up to
# 256 tokens)
MANY_HEADS = [(12, 2, 4, 77, 64, 72), (10, 4, 8, 300, 128, 128), (40, 1, 2, 129, 96, 64),
              (7, 1, 4, 260, 8, 200), (16, 1, 3, 1, 128, 128), (1, 16, 64, 385, 128, 64)]


@pytest.mark.parametrize("size", MANY_HEADS, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("init", [True, False])
def test_many_heads(size, init):
    B, NHK, NH, T, DK, DV = size
    run_case("tc", dict(B=B, NHK=NHK, NH=NH, T=T, DK=DK, DV=DV, init=init), backward=T < 100)


@pytest.mark.parametrize("size,backward", [((4, 2, 4, 2437, 64, 64), True),
                                           ((15, 2, 4, 700, 128, 72), False)], ids=str)
def test_more_chunks_than_blocks(size, backward):
    """Every persistent stage takes several items a block (320 and 360 chunks)."""
    B, NHK, NH, T, DK, DV = size
    run_case("tc", dict(B=B, NHK=NHK, NH=NH, T=T, DK=DK, DV=DV, gates="reset", seed=4),
             backward=backward)


@pytest.mark.parametrize("gates", ["strong", "hold", "zero_beta", "reset"])
@pytest.mark.parametrize("keys", ["unit", "alike"])
def test_many_heads_gates_and_keys(gates, keys):
    run_case("tc", dict(B=20, NHK=2, NH=4, T=333, DK=128, DV=128, gates=gates, keys=keys, seed=3),
             backward=False)


@pytest.mark.parametrize("algo", ALGOS)
@pytest.mark.parametrize("gates", ["strong", "hold", "zero_beta", "reset"])
@pytest.mark.parametrize("keys", ["unit", "alike"])
def test_gates_and_keys(algo, gates, keys):
    run_case(algo, dict(NHK=1, NH=2, T=333, DK=128, DV=128, gates=gates, keys=keys, seed=7))


@pytest.mark.parametrize("size", [(1, 1, 1, 64, 64, 64), (2, 2, 4, 131, 96, 72),
                                  (1, 1, 2, 300, 128, 256), (1, 2, 2, 513, 128, 128)],
                         ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("init", [True, False])
def test_training_pair(size, init):
    """The pair against fp64, and its gradients the recomputing call's."""
    B, NHK, NH, T, DK, DV = size
    x = gd.make(B=B, NHK=NHK, NH=NH, T=T, DK=DK, DV=DV, init=init)
    d = gd.cuda(x)
    H, C_T, saved = api.gated_delta_fw_train(*(d[n] for n in gd.NAMES), scale=0.2)
    H64, C64 = ref.forward(**gd.fp64(x), scale=0.2)
    check("tc", {"H": H, "C_T": C_T}, {"H": H64, "C_T": C64})
    gen = torch.Generator().manual_seed(1)
    dH = torch.randn(x["V"].shape, generator=gen).to(x["V"].dtype)
    dC = torch.randn(C_T.shape, generator=gen)
    got = api.gated_delta_bw_saved(*(d[n] for n in gd.NAMES[:5]), saved, dH.cuda(), d["C0"],
                                   dC.cuda(), scale=0.2)
    want = ref.gradients(x, dH, dC, 0.2)
    check("tc", got, {n: w for n, w in want.items() if n in got})
    # and the recomputing call's
    again = api.gated_delta_bw(*(d[n] for n in gd.NAMES[:5]), dH.cuda(), d["C0"], dC.cuda(),
                               scale=0.2)
    assert all(torch.equal(got[n], again[n]) for n in got)


@pytest.mark.parametrize("algo", ALGOS)
def test_no_initial_state_and_scale(algo):
    run_case(algo, dict(T=150, init=False, DK=128, DV=64), scale=0.37)


@pytest.mark.parametrize("algo", ALGOS)
def test_reset_starts_a_new_sequence(algo):
    """g = -inf at a token: what follows equals a fresh sequence, bit for bit
    where the chunks line up (token 128)."""
    x = gd.cuda(gd.make(T=256, DK=128, DV=64))
    x["g"][:, :, 128] = float("-inf")
    H, C = api.gated_delta_fw(*(x[n] for n in gd.NAMES), algo=algo)
    y = {n: x[n][:, :, 128:].contiguous() for n in gd.NAMES[:5]}
    H2, C2 = api.gated_delta_fw(*(y[n] for n in gd.NAMES[:5]), algo=algo)
    assert torch.equal(H[:, :, 128:], H2) and torch.equal(C, C2)


@pytest.mark.parametrize("algo", ALGOS)
def test_padding_leaves_the_state(algo):
    """g = beta = 0 behind a row's end: state and gradients of the shorter row."""
    x = gd.make(T=200, DK=128, DV=128)
    for n in ("g", "beta"):
        x[n][:, :, 137:] = 0.0
    d = gd.cuda(x)
    _, C = api.gated_delta_fw(*(d[n] for n in gd.NAMES), algo=algo)
    cut = {n: v if n == "C0" else v[:, :, :137].contiguous() for n, v in x.items()}
    check(algo, {"C": C}, {"C": ref.forward(**gd.fp64(cut))[1]})


@pytest.mark.parametrize("kw", [dict(T=300), dict(T=100), dict(T=300, dtype="f32")], ids=str)
def test_without_the_final_state(kw):
    """H is the same bits whether or not the final state is asked for."""
    x = gd.cuda(gd.make(DK=64, DV=96, **kw))
    a = [x[n] for n in gd.NAMES]
    H, _ = api.gated_delta_fw(*a)
    assert torch.equal(H, api.gated_delta_fw(*a, return_last_state=False))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_longest_sequence(dtype):
    """2^22 tokens: behind a reset near the end, a sequence of its own."""
    T, n = 1 << 22, 300
    gen = torch.Generator(device="cuda").manual_seed(3)
    mk = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    q, k = (torch.nn.functional.normalize(mk(1, 1, T, 8), dim=-1).to(gd.DT[dtype])
            for _ in range(2))
    v = mk(1, 1, T, 8).to(gd.DT[dtype])
    g, beta = -0.1 * mk(1, 1, T).abs(), torch.sigmoid(mk(1, 1, T))
    g[:, :, T - n] = float("-inf")
    x = dict(zip(gd.NAMES, (q, k, v, g, beta, None)))
    H, C = api.gated_delta_fw(q, k, v, g, beta)
    tail = {m: None if t is None else t[:, :, T - n:].cpu() for m, t in x.items()}
    H64, C64 = ref.forward(**gd.fp64(tail))
    check("simt" if dtype == "f32" else "tc", {"H": H[:, :, T - n:], "C": C},
          {"H": H64, "C": C64})
    assert torch.isfinite(H).all()


def test_zero_length():
    x = gd.cuda(gd.make(T=0))
    H, C = api.gated_delta_fw(*(x[n] for n in gd.NAMES))
    assert H.shape[2] == 0 and torch.equal(C, x["C0"])
    _, C = api.gated_delta_fw(*(x[n] for n in gd.NAMES[:5]))
    assert not C.any()
    dC = torch.randn_like(x["C0"])
    d = api.gated_delta_bw(*(x[n] for n in gd.NAMES[:5]), x["V"], x["C0"], dC)
    assert torch.equal(d["dC0"], dC)
    d = api.gated_delta_bw(*(x[n] for n in gd.NAMES[:5]), x["V"], x["C0"])
    assert not d["dC0"].any()


def test_no_value_outside_the_outputs():
    """H, C_T and the gradients inside larger buffers: the rest stays."""
    x = gd.cuda(gd.make(B=1, NHK=2, NH=2, T=77, DK=64, DV=72))
    n = x["V"].numel()
    buf = torch.full((n + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    H = buf[32:32 + n].view(x["V"].shape)
    want, _ = api.gated_delta_fw(*(x[k] for k in gd.NAMES))
    got, _ = api.gated_delta_fw(*(x[k] for k in gd.NAMES), out={"H": H})
    assert torch.equal(got, want)
    assert (buf[:32] == 7).all() and (buf[32 + n:] == 7).all()


def test_state_in_place_and_segments():
    """A sequence in two calls, the state handed on in one buffer."""
    x = gd.make(T=300, DK=128, DV=128)
    d = gd.cuda(x)
    H64, C64 = ref.forward(**gd.fp64(x))
    C, parts = d["C0"].clone(), []
    for a, b in ((0, 111), (111, 300)):
        y = [d[n][:, :, a:b].contiguous() for n in gd.NAMES[:5]]
        H, _ = api.gated_delta_fw(*y, C, out={"C_T": C})
        parts.append(H)
    check("tc", {"H": torch.cat(parts, 2), "C": C}, {"H": H64, "C": C64})


STEP_SIZES = [(1, 1, 1, 128, 128), (3, 2, 4, 64, 96), (2, 1, 2, 100, 52), (1, 2, 2, 33, 7),
              (1, 1, 1, 256, 512), (1, 1, 2, 1024, 1024), (2, 1, 1, 1, 1), (1, 1, 1, 130, 66),
              (40, 4, 8, 128, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", STEP_SIZES, ids=lambda s: "x".join(map(str, s)))
def test_step(dtype, size):
    B, NHK, NH, DK, DV = size
    T = 4
    x = gd.make(B=B, NHK=NHK, NH=NH, T=T, DK=DK, DV=DV, dtype=dtype)
    x["g"][:, :, 2] = float("-inf")
    d = gd.cuda(x)
    H64, C64 = ref.forward(**gd.fp64(x))
    C, hs = d["C0"].clone(), []
    for t in range(T):
        y = [d[n][:, :, t].contiguous() for n in gd.NAMES[:5]]
        hs.append(api.gated_delta_step(*y, C))
    check("simt", {"H": torch.stack(hs, 2), "C": C}, {"H": H64, "C": C64})


def test_prefill_then_steps():
    """The forward's final state continued by the step: one sequence."""
    x = gd.make(NHK=1, NH=2, T=203, DK=128, DV=128)
    d = gd.cuda(x)
    H64, C64 = ref.forward(**gd.fp64(x))
    y = [d[n][:, :, :200].contiguous() for n in gd.NAMES[:5]]
    H, C = api.gated_delta_fw(*y, d["C0"])
    hs = [api.gated_delta_step(*(d[n][:, :, t].contiguous() for n in gd.NAMES[:5]), C)
          for t in range(200, 203)]
    check("tc", {"H": torch.cat([H, torch.stack(hs, 2)], 2), "C": C}, {"H": H64, "C": C64})


@pytest.mark.parametrize("dtype,recompute", [("bf16", False), ("bf16", True), ("f32", False)])
def test_autograd(dtype, recompute):
    """Gradients of losses on H, on C_T and on both, through the public call."""
    x = gd.make(NHK=1, NH=2, T=140, DK=64, DV=64, dtype=dtype)
    gen = torch.Generator().manual_seed(9)
    wH = torch.randn(x["V"].shape, generator=gen).to(x["V"].dtype)
    wC = torch.randn(x["C0"].shape, generator=gen)
    for use_h, use_c in ((True, False), (False, True), (True, True)):
        d = {n: v.detach().requires_grad_() for n, v in gd.cuda(x).items()}
        H, C = api.gated_delta_chunkwise(*(d[n] for n in gd.NAMES), recompute=recompute)
        # wH carries a stride that the upstream gradient hands on
        up = wH.cuda().transpose(1, 2).contiguous().transpose(1, 2)
        outs, ws = ([H] if use_h else []) + ([C] if use_c else []), \
            ([up] if use_h else []) + ([wC.cuda()] if use_c else [])
        grads = torch.autograd.grad(outs, [d[n] for n in gd.NAMES], ws)
        want = ref.gradients(x, wH if use_h else None, wC if use_c else None)
        check("tc", {"d" + n: g for n, g in zip(gd.NAMES, grads)}, want)


def test_repeat_calls_agree_bit_for_bit():
    x = gd.cuda(gd.make(B=2, NHK=2, NH=4, T=400, DK=128, DV=128))
    dH = torch.randn_like(x["V"])
    first = None
    for _ in range(3):
        H, C = api.gated_delta_fw(*(x[n] for n in gd.NAMES))
        g = api.gated_delta_bw(*(x[n] for n in gd.NAMES[:5]), dH, x["C0"])
        now = [H, C, *g.values()]
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_inputs_are_checked(dtype):
    """What the binding refuses with tensors on the GPU: shapes, types, strides."""
    x = gd.cuda(gd.make(NHK=1, NH=2, T=64, DK=64, DV=64, dtype=dtype))
    a = [x[n] for n in gd.NAMES]

    def refuse(match, i, bad, call=api.gated_delta_fw):
        with pytest.raises(ValueError, match=match):
            call(*(bad if j == i else t for j, t in enumerate(a)))

    refuse("contiguous", 0, x["Q"].transpose(2, 3).contiguous().transpose(2, 3))
    refuse("shape", 1, x["K"][:, :, :-1].contiguous())
    refuse("shape", 3, x["g"][:, :1].contiguous())
    refuse("float32", 4, x["beta"].double())
    refuse("shape", 5, x["C0"][..., :-1].contiguous())
    refuse("CUDA tensor", 2, x["V"].cpu())
    out = torch.empty_like(x["V"])[:, :, :-1]
    with pytest.raises(ValueError, match="shape"):
        api.gated_delta_fw(*a, out={"H": out})
    with pytest.raises(ValueError, match="workspace"):
        api.gated_delta_fw(*a, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    if dtype == "bf16":
        _, _, saved = api.gated_delta_fw_train(*a)
        with pytest.raises(ValueError, match="shape"):
            api.gated_delta_bw_saved(*a[:5], saved[:-16].contiguous(), x["V"], a[5])
    torch.cuda.synchronize()
    assert api.last_device_error() == _lib.OK


def test_a_workspace_of_the_callers_holds_other_data():
    """Nothing is read from the workspace before it is written."""
    for kw in (dict(T=200), dict(B=12, NHK=4, NH=4, T=200), dict(T=200, dtype="f32")):
        x = gd.cuda(gd.make(DK=64, DV=64, **kw))
        a = [x[n] for n in gd.NAMES]
        want = api.gated_delta_fw(*a)
        B, NHK, T, DK = x["Q"].shape
        n = api.gated_delta_workspace_size(B, NHK, x["V"].shape[1], T, DK, 64, x["Q"].dtype)
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN in every type
        got = api.gated_delta_fw(*a, workspace=ws)
        assert all(torch.equal(p, q) for p, q in zip(want, got))


def test_two_streams_at_once():
    xs = [gd.cuda(gd.make(T=500, DK=128, DV=128, seed=s)) for s in (1, 2)]
    want = [api.gated_delta_fw(*(x[n] for n in gd.NAMES)) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for x, s in zip(xs, streams):
        with torch.cuda.stream(s):
            got.append(api.gated_delta_fw(*(x[n] for n in gd.NAMES)))
    torch.cuda.synchronize()
    for (a, b), (c, d) in zip(want, got):
        assert torch.equal(a, c) and torch.equal(b, d)


def test_captured_and_replayed():
    """Forward, backward and step in one CUDA graph, replayed on new inputs,
    while an eager autograd graph of the same tensors is alive.  (The captured
    pass differentiates leaves of its own: autograd ties a leaf that a live
    eager graph holds to that graph's stream, which a capture may not touch.)"""
    x = gd.cuda(gd.make(T=260, DK=128, DV=64))
    dH = torch.randn_like(x["V"])
    eager, _ = api.gated_delta_chunkwise(*(v.detach().requires_grad_() for v in x.values()))
    tok = [x[n][:, :, -1].contiguous() for n in gd.NAMES[:5]]
    C = x["C0"].clone()

    def work():
        leaves = [x[n].detach().requires_grad_() for n in gd.NAMES]
        H, C_T = api.gated_delta_chunkwise(*leaves)
        grads = torch.autograd.grad(H, leaves, dH)
        C.copy_(C_T.detach())
        return [H.detach(), *grads, api.gated_delta_step(*tok, C), C]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = work()
    fresh = gd.cuda(gd.make(T=260, DK=128, DV=64, seed=5))
    for n in gd.NAMES:
        x[n].copy_(fresh[n])
    graph.replay()
    torch.cuda.synchronize()
    got = [o.clone() for o in outs]
    assert all(torch.equal(a, b) for a, b in zip(got, work()))
    del eager


def test_cell_then_norm():
    """The cell and its output norm as a block uses them, against fp64."""
    x = gd.make(B=2, NHK=2, NH=4, T=150, DK=64, DV=64)
    d = {n: v.requires_grad_() for n, v in gd.cuda(x).items()}
    gen = torch.Generator().manual_seed(2)
    w, b = 1 + 0.1 * torch.randn(4, 64, generator=gen), 0.1 * torch.randn(4, 64, generator=gen)
    wd, bd = w.cuda().requires_grad_(), b.cuda().requires_grad_()
    H, _ = api.gated_delta_chunkwise(*(d[n] for n in gd.NAMES))
    Y = api.head_norm(H, wd, bd)
    dY = torch.randn(Y.shape, generator=gen).to(torch.bfloat16)
    grads = torch.autograd.grad(Y, [*(d[n] for n in gd.NAMES), wd, bd], dY.cuda())

    r = {n: v.detach().double().requires_grad_() for n, v in x.items()}
    w64, b64 = w.double().requires_grad_(), b.double().requires_grad_()
    H64, _ = ref.forward(**r)
    mu = H64.mean(-1, keepdim=True)
    xh = (H64 - mu) / (((H64 - mu) ** 2).mean(-1, keepdim=True) + 1e-5).sqrt()
    Y64 = (xh * w64[None, :, None] + b64[None, :, None]).transpose(1, 2).reshape(Y.shape)
    want = torch.autograd.grad(Y64, [*(r[n] for n in gd.NAMES), w64, b64], dY.double())
    # H is rounded to bf16 between the two (2^-8 of each value) and dH again on
    # the way back; relative norms, where those roundings average out
    for n, a, e in zip((*gd.NAMES, "weight", "bias"), grads, want):
        a = a.double().cpu()
        assert float((a - e).norm() / e.norm()) < 2 * 2.0 ** -8, n
    Y64 = Y64.detach()
    assert float((Y.detach().double().cpu() - Y64).norm() / Y64.norm()) < 2 * 2.0 ** -8
