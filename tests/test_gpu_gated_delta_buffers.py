"""Gated delta rule and cell-output layer norm through the C ABI: every output
between guard bytes, every workspace and saved buffer of exactly the size asked
for, between guard bytes and full of NaN; the bits are those of the binding's
calls.  And gradients of padded rows, and the norm behind the mLSTM."""
import pytest
import torch

import gated_delta_cases as gd
from mlstm_chunkwise_b200 import _lib, api
from oracle import gated_delta as ref

pytestmark = pytest.mark.gpu

GUARD, MARK = 256, 0xA5
_DT = {torch.float32: _lib.DT_F32, torch.bfloat16: _lib.DT_BF16}
_ALGO = {"simt": _lib.ALGO_SIMT, "tc": _lib.ALGO_TC, "auto": _lib.ALGO_AUTO}


class Guarded:
    """Tensors inside larger buffers; 0xFF, a NaN in every type, is what they hold."""

    def __init__(self):
        self.all = {}

    def __call__(self, name, shape, dtype):
        n = torch.empty(shape, dtype=dtype, device="meta").numel() * dtype.itemsize
        buf = torch.full((n + 2 * GUARD,), MARK, dtype=torch.uint8, device="cuda")
        buf[GUARD:GUARD + n] = 255
        t = buf[GUARD:GUARD + n].view(dtype).view(shape)
        self.all[name] = (buf, n)
        return t

    def check(self):
        torch.cuda.synchronize()
        assert api.last_device_error() == _lib.OK
        for name, (buf, n) in self.all.items():
            assert (buf[:GUARD] == MARK).all() and (buf[GUARD + n:] == MARK).all(), name


def p(t):
    return None if t is None else t.data_ptr()


def same(got, want):
    for n, w in want.items():
        assert torch.equal(got[n], w), n


SHAPES = [(1, 2, 4, 77, 64, 72), (2, 1, 3, 300, 96, 128), (1, 2, 2, 129, 128, 200),
          (1, 1, 2, 65, 72, 64), (2, 2, 2, 40, 8, 8), (1, 1, 1, 257, 128, 392),
          (40, 1, 2, 130, 64, 64)]
ODD = [(1, 1, 2, 130, 100, 52), (2, 1, 2, 70, 33, 7), (1, 2, 2, 65, 256, 96)]
CASES = [("tc", "bf16", s) for s in SHAPES] + [("simt", "bf16", s) for s in SHAPES[:3] + ODD] + \
    [("simt", "f32", s) for s in SHAPES[:2] + ODD]


def inputs(dtype, size, init, seed=0):
    B, NHK, NH, T, DK, DV = size
    x = gd.cuda(gd.make(B=B, NHK=NHK, NH=NH, T=T, DK=DK, DV=DV, dtype=dtype, init=init, seed=seed))
    return x, [x[n] for n in gd.NAMES], torch.randn_like(x["V"]), \
        torch.randn(B, NH, DK, DV, device="cuda")


def grads(x, init, new):
    return {"d" + n: new("d" + n, x[n].shape, x[n].dtype) for n in gd.NAMES[:5]} | \
        ({"dC0": new("dC0", x["C0"].shape, torch.float32)} if init else {})


@pytest.mark.parametrize("init", [True, False])
@pytest.mark.parametrize("algo,dtype,size", CASES, ids=str)
def test_forward_and_gradients(algo, dtype, size, init):
    x, a, dH, dC = inputs(dtype, size, init)
    B, NHK, NH, T, DK, DV = size
    dt, tail, L = x["V"].dtype, (1.0, _DT[x["V"].dtype], _ALGO[algo]), _lib.lib()
    new = Guarded()
    H, C = new("H", x["V"].shape, dt), new("C_T", dC.shape, torch.float32)
    ws = [new("ws", (api.gated_delta_workspace_size(*size, dt, algo, backward=b),), torch.uint8)
          for b in (False, True)]
    assert L.mlstm_gated_delta_fw(*map(p, a), p(H), p(C), *size, *tail, p(ws[0]), ws[0].numel(),
                                  None) == _lib.OK
    new.check()
    want = api.gated_delta_fw(*a, scale=1.0, algo=algo)
    assert torch.equal(H, want[0]) and torch.equal(C, want[1])
    d = grads(x, init, new)
    assert L.mlstm_gated_delta_bw(*map(p, a), p(dH), p(dC), *(p(d["d" + n]) for n in gd.NAMES[:5]),
                                  p(d.get("dC0")), *size, *tail, p(ws[1]), ws[1].numel(),
                                  None) == _lib.OK
    new.check()
    same(d, api.gated_delta_bw(*a[:5], dH, x["C0"], dC, scale=1.0, algo=algo))


@pytest.mark.parametrize("init", [True, False])
@pytest.mark.parametrize("size", [s for s in SHAPES if s[0] * s[2] * s[3] >= 64], ids=str)
def test_training_pair(size, init):
    x, a, dH, dC = inputs("bf16", size, init)
    tail, L = (1.0, _lib.DT_BF16), _lib.lib()
    sizes = api.gated_delta_train_sizes(*size)
    new = Guarded()
    H, C = new("H", x["V"].shape, torch.bfloat16), new("C_T", dC.shape, torch.float32)
    saved, ws, ws2 = (new(n, (k,), torch.uint8) for n, k in zip(("saved", "ws", "ws2"), sizes))
    assert L.mlstm_gated_delta_fw_train(*map(p, a), p(H), p(C), p(saved), sizes[0], *size, *tail,
                                        p(ws), sizes[1], None) == _lib.OK
    new.check()
    want = api.gated_delta_fw_train(*a, scale=1.0)
    assert torch.equal(H, want[0]) and torch.equal(C, want[1])
    d = grads(x, init, new)
    assert L.mlstm_gated_delta_bw_saved(*map(p, a[:5]), p(saved), sizes[0], p(dH), p(dC),
                                        *(p(d["d" + n]) for n in gd.NAMES[:5]), p(d.get("dC0")),
                                        *size, *tail, p(ws2), sizes[2], None) == _lib.OK
    new.check()
    same(d, api.gated_delta_bw_saved(*a[:5], want[2], dH, x["C0"], dC, scale=1.0))
    same(d, api.gated_delta_bw(*a[:5], dH, x["C0"], dC, scale=1.0))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("size", [(3, 2, 4, 64, 96), (1, 2, 2, 33, 7), (1, 1, 1, 130, 66),
                                  (1, 1, 1, 1, 1)], ids=str)
def test_step(dtype, size):
    B, NHK, NH, DK, DV = size
    x, _, _, _ = inputs(dtype, (B, NHK, NH, 1, DK, DV), True)
    tok = [x[n][:, :, 0].contiguous() for n in gd.NAMES[:5]]
    new = Guarded()
    C, h = new("C", x["C0"].shape, torch.float32), new("h", tok[2].shape, tok[2].dtype)
    C.copy_(x["C0"])
    assert _lib.lib().mlstm_gated_delta_step(*map(p, tok), p(C), p(h), *size, 1.0,
                                             _DT[h.dtype], None) == _lib.OK
    new.check()
    assert torch.equal(h, api.gated_delta_step(*tok, x["C0"], scale=1.0))
    assert torch.equal(C, x["C0"])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", [(1, 1, 1, 1), (2, 3, 5, 64), (3, 1, 17, 100), (1, 2, 33, 72),
                                  (1, 1, 9, 511), (2, 1, 21, 1032), (1, 2, 5, 1500),
                                  (1, 1, 3, 8191), (1, 1, 5, 8192)], ids=str)
def test_norm(dtype, size):
    B, NH, T, D = size
    X, dY = torch.randn(size, device="cuda").to(dtype), \
        torch.randn(B, T, NH * D, device="cuda").to(dtype)
    w, b = torch.randn(NH, D, device="cuda"), torch.randn(NH, D, device="cuda")
    new, L = Guarded(), _lib.lib()
    f32 = torch.float32
    Y = new("Y", dY.shape, dtype)
    mean, rstd = new("mean", size[:3], f32), new("rstd", size[:3], f32)
    assert L.mlstm_head_norm_fw(p(X), p(w), p(b), p(Y), p(mean), p(rstd), *size, 1e-5, _DT[dtype],
                                None) == _lib.OK
    new.check()
    want = api.head_norm_fw(X, w, b)
    assert all(torch.equal(u, v) for u, v in zip((Y, mean, rstd), want))
    d = {"dX": new("dX", size, dtype), "dweight": new("dweight", (NH, D), f32),
         "dbias": new("dbias", (NH, D), f32)}
    ws = new("ws", (api._head_norm_workspace(*size, dtype),), torch.uint8)
    assert L.mlstm_head_norm_bw(p(X), p(dY), p(w), p(mean), p(rstd), *map(p, d.values()), *size,
                                _DT[dtype], p(ws), ws.numel(), None) == _lib.OK
    new.check()
    same(d, api.head_norm_bw(X, dY, w, mean, rstd))


@pytest.mark.parametrize("algo", ["simt", "tc"])
@pytest.mark.parametrize("NHK,NH", [(2, 2), (1, 2)])
def test_gradients_of_padded_rows(algo, NHK, NH):
    """g = beta = 0 and no upstream gradient behind a row's end: the tokens' own q, k
    and v get exactly none, and the rest are the shorter row's, to the tolerance of
    the gradients' tests (8 x 2^-16 on the tensor cores, 300 x 2^-24 in fp32, and
    half a step of a 16-bit output)."""
    T, n = 200, 137
    x = gd.make(NHK=NHK, NH=NH, T=T, DK=128, DV=128)
    gen = torch.Generator().manual_seed(4)
    dH = torch.randn(x["V"].shape, generator=gen).bfloat16()
    dC = torch.randn(x["C0"].shape, generator=gen)
    for t in (x["g"], x["beta"], dH):
        t[:, :, n:] = 0.0
    d = gd.cuda(x)
    got = api.gated_delta_bw(*(d[m] for m in gd.NAMES[:5]), dH.cuda(), d["C0"], dC.cuda(),
                             algo=algo)
    assert not any(got[m][:, :, n:].any() for m in ("dQ", "dK", "dV"))
    cut = {m: v if m == "C0" else v[:, :, :n].contiguous() for m, v in x.items()}
    want = ref.gradients(cut, dH[:, :, :n], dC)
    for m, w in want.items():
        g = got[m] if m == "dC0" else got[m][:, :, :n]
        tol = (1.2e-4 if algo == "tc" else 1.8e-5) + \
            (2.0 ** -8 if g.dtype == torch.bfloat16 else 0.0)
        assert gd.worst(g, w) < tol, m


def test_norm_behind_the_mlstm():
    """head_norm on mlstm_chunkwise's output: Y against fp64 of the same H, and the
    gradients those of the two calls one after the other."""
    B, NH, T, DK, DV = 2, 4, 256, 128, 256
    gen = torch.Generator().manual_seed(6)
    mk = lambda *s: torch.randn(*s, generator=gen).cuda()
    leaves = [mk(B, NH, T, DK).bfloat16(), mk(B, NH, T, DK).bfloat16(), mk(B, NH, T, DV).bfloat16(),
              mk(B, NH, T), mk(B, NH, T) + 3]
    w, b, dY = 1 + 0.1 * mk(NH, DV), 0.1 * mk(NH, DV), mk(B, T, NH * DV).bfloat16()
    for t in (*leaves, w, b):
        t.requires_grad_()
    H, _ = api.mlstm_chunkwise(*leaves)
    Y = api.head_norm(H, w, b)
    got = torch.autograd.grad(Y, (*leaves, w, b), dY)
    X = H.detach().double()
    c = X - X.mean(-1, keepdim=True)
    Y64 = c / (c.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w.detach().double()[:, None] + \
        b.detach().double()[:, None]
    Y64 = Y64.transpose(1, 2).reshape(B, T, NH * DV)
    # half a step of bf16, and the row sums in fp32 (6e-6, four times where they cancel)
    assert float(((Y.detach().double() - Y64).abs() - Y64.abs() * 2.0 ** -8).max()) < 2.4e-5 * \
        float(Y64.abs().max())
    with torch.no_grad():
        _, mean, rstd = api.head_norm_fw(H, w, b)
        d = api.head_norm_bw(H, dY, w, mean, rstd)
    H2, _ = api.mlstm_chunkwise(*leaves)
    want = (*torch.autograd.grad(H2, leaves, d["dX"]), d["dweight"], d["dbias"])
    assert all(torch.equal(u, v) for u, v in zip(got, want))


@pytest.fixture(scope="module")
def dbg():
    from mlstm_chunkwise_b200 import build
    return _lib.open_library(build.build(debug_bounds=True))


@pytest.mark.parametrize("algo,dtype,size", CASES, ids=str)
def test_bounds_checked_build(dbg, monkeypatch, algo, dtype, size):
    """Its checks of workspace copies and stores find nothing and change no bit."""
    B, NHK, NH, T, DK, DV = size
    x, a, dH, dC = inputs(dtype, size, True)
    w = torch.ones(NH, DV, device="cuda")
    pair = algo == "tc" and B * NH * T >= 64

    def work():
        H, C = api.gated_delta_fw(*a, algo=algo)
        out = [H, C, *api.gated_delta_bw(*a[:5], dH, x["C0"], dC, algo=algo).values()]
        if pair:
            H, C, saved = api.gated_delta_fw_train(*a)
            out += [H, C, *api.gated_delta_bw_saved(*a[:5], saved, dH, x["C0"], dC).values()]
        C = C.clone()
        out += [api.gated_delta_step(*(t[:, :, -1].contiguous() for t in a[:5]), C), C]
        Y, mean, rstd = api.head_norm_fw(H, w, w)
        return out + [Y, mean, rstd, *api.head_norm_bw(H, Y, w, mean, rstd).values()]

    want = work()
    torch.cuda.synchronize()
    dbg.mlstm_set_watchdog(1 << 22)
    monkeypatch.setattr(_lib, "_lib", dbg)
    got = work()
    torch.cuda.synchronize()
    assert dbg.mlstm_last_device_error(None) == _lib.OK
    assert dbg.mlstm_last_device_error_word() == 0
    assert all(torch.equal(u, v) for u, v in zip(got, want))
