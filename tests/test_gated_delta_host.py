"""Argument checks of the gated delta rule and the cell-output layer norm that
need no GPU: every call here is refused before any CUDA call."""
import ctypes

import pytest
import torch

from mlstm_chunkwise_b200 import _lib, api, build

P = ctypes.c_void_p(0x10000)
U = ctypes.c_void_p(0x10004)  # not 16-byte aligned
O = ctypes.c_void_p(0x10001)  # not aligned by any element
GATES = ("g", "beta", "dg", "dbeta")  # read element by element


@pytest.fixture(scope="module")
def L():
    build.build()
    return _lib.lib()


def size(B=1, NHK=2, NH=4, T=100, DK=64, DV=64, dt=_lib.DT_BF16, algo=_lib.ALGO_SIMT, bw=0):
    n = ctypes.c_size_t(0)
    st = _lib.lib().mlstm_gated_delta_workspace_size(B, NHK, NH, T, DK, DV, dt, algo, bw,
                                                     ctypes.byref(n))
    return st, n.value


BAD = [
    (dict(B=0), _lib.ERR_INVALID_ARG), (dict(NHK=0), _lib.ERR_INVALID_ARG),
    (dict(NHK=3), _lib.ERR_INVALID_ARG),  # 4 value heads over 3 key heads
    (dict(NHK=8), _lib.ERR_INVALID_ARG), (dict(T=-1), _lib.ERR_INVALID_ARG),
    (dict(DK=0), _lib.ERR_INVALID_ARG), (dict(DV=0), _lib.ERR_INVALID_ARG),
    (dict(dt=5), _lib.ERR_INVALID_ARG), (dict(algo=9), _lib.ERR_INVALID_ARG),
    (dict(DK=1025), _lib.ERR_UNSUPPORTED), (dict(DV=2048), _lib.ERR_UNSUPPORTED),
    (dict(T=(1 << 22) + 1), _lib.ERR_UNSUPPORTED),
    (dict(B=1 << 15), _lib.ERR_UNSUPPORTED),
    (dict(algo=_lib.ALGO_TC_FUSED), _lib.ERR_UNSUPPORTED),
    (dict(algo=_lib.ALGO_TC, dt=_lib.DT_F32), _lib.ERR_UNSUPPORTED),
    (dict(algo=_lib.ALGO_TC, DK=256), _lib.ERR_UNSUPPORTED),
    (dict(algo=_lib.ALGO_TC, DK=60), _lib.ERR_UNSUPPORTED),
    (dict(algo=_lib.ALGO_TC, DV=12), _lib.ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,expect", BAD, ids=lambda v: str(v))
def test_sizes_refused(L, kw, expect):
    for bw in (0, 1):
        assert size(bw=bw, **kw)[0] == expect


def test_workspace_grows_with_the_call(L):
    for algo in (_lib.ALGO_SIMT, _lib.ALGO_AUTO):
        st, fw = size(algo=algo)
        st2, bw = size(algo=algo, bw=1)
        assert st == st2 == _lib.OK and 0 < fw < bw
        assert size(algo=algo, T=0) == (_lib.OK, 0)


def fw(**over):
    a = dict(Q=P, K=P, V=P, g=P, beta=P, C0=None, H=P, C_T=None, B=1, NHK=1, NH=2, T=64, DK=64,
             DV=64, scale=1.0, dt=_lib.DT_BF16, algo=_lib.ALGO_SIMT, ws=P, wsb=1 << 40)
    a.update(over)
    return _lib.lib().mlstm_gated_delta_fw(*a.values(), None)


def bw(**over):
    a = dict(Q=P, K=P, V=P, g=P, beta=P, C0=None, dH=P, dC_T=None, dQ=P, dK=P, dV=P, dg=P,
             dbeta=P, dC0=None, B=1, NHK=1, NH=2, T=64, DK=64, DV=64, scale=1.0,
             dt=_lib.DT_BF16, algo=_lib.ALGO_SIMT, ws=P, wsb=1 << 40)
    a.update(over)
    return _lib.lib().mlstm_gated_delta_bw(*a.values(), None)


def step(**over):
    a = dict(q=P, k=P, v=P, g=P, beta=P, C=P, h=P, B=1, NHK=1, NH=2, DK=64, DV=64, scale=1.0,
             dt=_lib.DT_BF16)
    a.update(over)
    return _lib.lib().mlstm_gated_delta_step(*a.values(), None)


@pytest.mark.parametrize("name", ["Q", "K", "V", "g", "beta", "H", "ws"])
def test_fw_pointers(L, name):
    assert fw(**{name: None}) == _lib.ERR_INVALID_ARG
    assert fw(**{name: O if name in GATES else U}) == _lib.ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["Q", "K", "V", "g", "beta", "dH", "dQ", "dK", "dV", "dg",
                                  "dbeta", "ws"])
def test_bw_pointers(L, name):
    assert bw(**{name: None}) == _lib.ERR_INVALID_ARG
    assert bw(**{name: O if name in GATES else U}) == _lib.ERR_INVALID_ARG


def train_sizes(B=1, NHK=2, NH=4, T=100, DK=64, DV=64, dt=_lib.DT_BF16):
    z = [ctypes.c_size_t(0) for _ in range(3)]
    st = _lib.lib().mlstm_gated_delta_train_sizes(B, NHK, NH, T, DK, DV, dt,
                                                  *(ctypes.byref(n) for n in z))
    return st, [n.value for n in z]


def test_train_sizes(L):
    st, (saved, fw_ws, bw_ws) = train_sizes()
    assert st == _lib.OK and min(saved, fw_ws, bw_ws) > 0
    # the three together hold what the recomputing backward needs
    assert saved + fw_ws + bw_ws >= size(algo=_lib.ALGO_TC, bw=1)[1]
    for kw in (dict(dt=_lib.DT_F32), dict(DK=136), dict(DK=60), dict(DV=12), dict(T=0),
               dict(T=15)):  # 4 x 15 tokens: AUTO's gradients take the fp32 path
        assert train_sizes(**kw)[0] == _lib.ERR_UNSUPPORTED, kw
    for kw in (dict(B=0), dict(NHK=3), dict(T=-1), dict(dt=7)):
        assert train_sizes(**kw)[0] == _lib.ERR_INVALID_ARG, kw
    n = ctypes.c_size_t(0)
    assert L.mlstm_gated_delta_train_sizes(1, 1, 1, 100, 64, 64, _lib.DT_BF16, None,
                                           ctypes.byref(n), ctypes.byref(n)) == \
        _lib.ERR_INVALID_ARG
    assert api.gated_delta_train_sizes(1, 2, 4, 100, 64, 64) == (saved, fw_ws, bw_ws)
    assert api.gated_delta_train_sizes(1, 2, 4, 100, 64, 64, torch.float32) is None


def fw_train(**over):
    a = dict(Q=P, K=P, V=P, g=P, beta=P, C0=None, H=P, C_T=None, saved=P, sb=1 << 40, B=1, NHK=1,
             NH=2, T=64, DK=64, DV=64, scale=1.0, dt=_lib.DT_BF16, ws=P, wsb=1 << 40)
    a.update(over)
    return _lib.lib().mlstm_gated_delta_fw_train(*a.values(), None)


def bw_saved(**over):
    a = dict(Q=P, K=P, V=P, g=P, beta=P, saved=P, sb=1 << 40, dH=P, dC_T=None, dQ=P, dK=P, dV=P,
             dg=P, dbeta=P, dC0=None, B=1, NHK=1, NH=2, T=64, DK=64, DV=64, scale=1.0,
             dt=_lib.DT_BF16, ws=P, wsb=1 << 40)
    a.update(over)
    return _lib.lib().mlstm_gated_delta_bw_saved(*a.values(), None)


@pytest.mark.parametrize("call", [fw_train, bw_saved])
def test_training_pair_refusals(L, call):
    names = ["Q", "K", "V", "g", "beta", "saved", "ws"] + \
        (["H"] if call is fw_train else ["dH", "dQ", "dK", "dV", "dg", "dbeta"])
    for n in names:
        assert call(**{n: None}) == _lib.ERR_INVALID_ARG, n
        assert call(**{n: O if n in GATES else U}) == _lib.ERR_INVALID_ARG, n
    assert call(sb=64) == _lib.ERR_INVALID_ARG
    assert call(wsb=64) == _lib.ERR_INVALID_ARG
    assert call(scale=float("inf")) == _lib.ERR_INVALID_ARG
    assert call(NHK=3) == _lib.ERR_INVALID_ARG
    assert call(dt=_lib.DT_F32) == _lib.ERR_UNSUPPORTED
    assert call(DK=256) == _lib.ERR_UNSUPPORTED
    assert call(T=0) == _lib.ERR_UNSUPPORTED


@pytest.mark.parametrize("name", ["q", "k", "v", "g", "beta", "C", "h"])
def test_step_pointers(L, name):
    assert step(**{name: None}) == _lib.ERR_INVALID_ARG
    assert step(**{name: U if name == "C" else O}) == _lib.ERR_INVALID_ARG


def test_other_refusals(L):
    for call in (fw, bw):
        assert call(wsb=16) == _lib.ERR_INVALID_ARG
        assert call(C0=U) == _lib.ERR_INVALID_ARG
        assert call(scale=float("nan")) == _lib.ERR_INVALID_ARG
        assert call(NHK=3) == _lib.ERR_INVALID_ARG
        assert call(dt=-1) == _lib.ERR_INVALID_ARG
    assert step(dt=4) == _lib.ERR_INVALID_ARG
    assert step(NHK=3) == _lib.ERR_INVALID_ARG
    assert step(DK=2000) == _lib.ERR_UNSUPPORTED


def test_head_norm_refusals(L):
    def nfw(X=P, w=P, b=None, Y=P, mean=P, rstd=P, B=1, NH=2, T=4, D=64, eps=1e-5,
            dt=_lib.DT_BF16):
        return L.mlstm_head_norm_fw(X, w, b, Y, mean, rstd, B, NH, T, D, eps, dt, None)

    def nbw(X=P, dY=P, w=P, mean=P, rstd=P, dX=P, dw=P, db=None, B=1, NH=2, T=4, D=64,
            dt=_lib.DT_BF16, ws=P, wsb=1 << 40):
        return L.mlstm_head_norm_bw(X, dY, w, mean, rstd, dX, dw, db, B, NH, T, D, dt, ws, wsb,
                                    None)

    for call, names in ((nfw, ("X", "w", "Y")), (nbw, ("X", "dY", "w", "mean", "rstd", "dX", "dw",
                                                       "ws"))):
        for n in names:
            assert call(**{n: None}) == _lib.ERR_INVALID_ARG
            assert call(**{n: U}) == _lib.ERR_INVALID_ARG
        for kw in (dict(B=0), dict(NH=0), dict(T=-1), dict(D=0), dict(dt=3)):
            assert call(**kw) == _lib.ERR_INVALID_ARG
        assert call(D=8193) == _lib.ERR_UNSUPPORTED
        assert call(B=70000) == _lib.ERR_UNSUPPORTED
    assert nfw(b=U) == _lib.ERR_INVALID_ARG
    assert nfw(eps=-1.0) == _lib.ERR_INVALID_ARG
    assert nfw(eps=float("nan")) == _lib.ERR_INVALID_ARG
    assert nbw(wsb=8) == _lib.ERR_INVALID_ARG


def test_binding_refuses(L):
    q = torch.zeros(1, 2, 4, 8)
    g = torch.zeros(1, 2, 4)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.gated_delta_fw(q, q, q, g, g)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.gated_delta_bw(q, q, q, g, g, q)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.gated_delta_fw_train(q, q, q, g, g)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.gated_delta_bw_saved(q, q, q, g, g, torch.zeros(8, dtype=torch.uint8), q)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.gated_delta_chunkwise(q, q, q, g, g)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.gated_delta_step(q[:, :, 0], q[:, :, 0], q[:, :, 0], g[:, :, 0], g[:, :, 0],
                             torch.zeros(1, 2, 8, 8))
    with pytest.raises(ValueError, match="multiple"):
        api.gated_delta_fw(torch.zeros(1, 3, 4, 8), torch.zeros(1, 3, 4, 8), q, g, g)
    with pytest.raises(ValueError, match="dtype"):
        api.gated_delta_fw(q.half(), q.half(), q.half(), g, g)
    with pytest.raises(ValueError, match=r"\[B, NHK, T, DK\]"):
        api.gated_delta_fw(q[0], q[0], q[0], g, g)
    with pytest.raises(ValueError, match="CUDA tensor"):
        api.head_norm_fw(q, torch.ones(2, 8))
    with pytest.raises(ValueError, match=r"\[B, NH, T, D\]"):
        api.head_norm(q[0], torch.ones(2, 8))
