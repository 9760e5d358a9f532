"""Cell-output layer norm on the GPU against fp64.

Tolerances, derived: statistics and sums are fp32 (a row's sum of D <= 8192
terms in at most 64 sequential additions per lane plus the tree: 100 x 2^-24 =
6e-6 of the sum of absolute values); a 16-bit output adds half a step, 2^-8.
Errors are relative to the largest value of the row's head; the input rows have
means of the order of their spread, so differences lose at most a factor of 4.
"""
import pytest
import torch

from mlstm_chunkwise_b200 import api

pytestmark = pytest.mark.gpu

TOL = {torch.float32: 2.4e-5, torch.bfloat16: 2.0 ** -8 + 2.4e-5}
SHAPES = [
    # B, NH, T, D
    (1, 1, 1, 1), (1, 1, 3, 7), (2, 3, 5, 64), (1, 2, 33, 72), (3, 1, 17, 100), (2, 8, 65, 128),
    (1, 4, 200, 512), (1, 1, 9, 511), (1, 1, 40, 1024), (2, 1, 21, 1032), (1, 1, 37, 2048),
    (1, 2, 5, 1500), (1, 1, 6, 4095), (1, 1, 5, 8192), (1, 1, 3, 8191), (5, 160, 2, 64),
]


def make(B, NH, T, D, dtype, bias, seed=0):
    gen = torch.Generator().manual_seed(seed)
    X = (torch.randn(B, NH, T, D, generator=gen) +
         torch.randn(B, NH, T, 1, generator=gen)).to(dtype)
    w = 1 + 0.3 * torch.randn(NH, D, generator=gen)
    b = torch.randn(NH, D, generator=gen) if bias else None
    return X, w, b, torch.randn(B, T, NH * D, generator=gen).to(dtype)


def reference(X, w, b, dY, eps):
    B, NH, T, D = X.shape
    X = X.double().requires_grad_()
    w = w.double().requires_grad_()
    b = None if b is None else b.double().requires_grad_()
    mean = X.mean(-1)
    rstd = ((X - mean[..., None]).square().mean(-1) + eps).rsqrt()
    Y = (X - mean[..., None]) * rstd[..., None] * w[None, :, None]
    if b is not None:
        Y = Y + b[None, :, None]
    Y = Y.transpose(1, 2).reshape(B, T, NH * D)
    grads = torch.autograd.grad(Y, [X, w] + ([] if b is None else [b]), dY.double())
    return Y.detach(), mean.detach(), rstd.detach(), grads


def err(got, want, scale=None):
    got = got.detach().double().cpu()
    assert got.shape == want.shape and torch.isfinite(got).all()
    s = float(want.abs().max()) if scale is None else scale
    return float((got - want).abs().max()) / max(s, 1e-30)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("bias", [True, False])
def test_against_fp64(dtype, shape, bias):
    X, w, b, dY = make(*shape, dtype, bias)
    eps = 1e-5
    Y64, m64, r64, g64 = reference(X, w, b, dY, eps)
    Xd, wd, dYd = X.cuda(), w.cuda(), dY.cuda()
    bd = None if b is None else b.cuda()
    Y, mean, rstd = api.head_norm_fw(Xd, wd, bd, eps=eps)
    if shape[3] > 1:  # a single column has variance 0: y = b, dx = 0
        assert err(Y, Y64) < TOL[dtype]
        assert err(rstd, r64) < TOL[torch.float32]
    else:
        assert torch.equal(Y.cpu(), Y64.to(dtype))
    assert err(mean, m64, max(1.0, float(m64.abs().max()))) < TOL[torch.float32]
    d = api.head_norm_bw(Xd, dYd, wd, mean, rstd, bias=bias)
    if shape[3] > 1:
        assert err(d["dX"], g64[0]) < TOL[dtype]
    else:  # a - mean(a) cancels exactly; xh is exactly 0
        assert not d["dX"].any()
    n = shape[0] * shape[2]
    # sums over n rows: n terms of rms |dy xh| ~ 1, rounded at most n / 64 + 64 times each
    s = max(float(g64[1].abs().max()), n ** 0.5)
    assert err(d["dweight"], g64[1], s) < TOL[torch.float32]
    if bias:
        assert err(d["dbias"], g64[2], max(float(g64[2].abs().max()), n ** 0.5)) < \
            TOL[torch.float32]
    else:
        assert "dbias" not in d


def test_autograd_and_repeat():
    X, w, b, dY = make(2, 4, 130, 128, torch.bfloat16, True)
    Y64, _, _, g64 = reference(X, w, b, dY, 1e-3)
    leaves = [t.cuda().requires_grad_() for t in (X, w, b)]
    runs = []
    for _ in range(2):
        Y = api.head_norm(*leaves, eps=1e-3)
        runs.append([Y, *torch.autograd.grad(Y, leaves, dY.cuda())])
    assert all(torch.equal(p, q) for p, q in zip(*runs))
    assert err(runs[0][0], Y64) < TOL[torch.bfloat16]
    for got, want in zip(runs[0][1:], g64):
        assert err(got, want) < TOL[got.dtype]


def test_large_offset_and_constant_rows():
    """A mean far above the spread (the variance comes from differences), and
    rows without any spread: y = bias, and dx finite."""
    X = torch.randn(1, 2, 50, 256, generator=torch.Generator().manual_seed(1)) + 1000.0
    w, b = torch.ones(2, 256), torch.zeros(2, 256)
    Y64, _, _, _ = reference(X, w, b, torch.zeros(1, 50, 512), 1e-5)
    Y, _, _ = api.head_norm_fw(X.cuda(), w.cuda(), b.cuda())
    # the mean is off by at most 100 x 2^-24 x 1000 = 6e-3 of the unit spread
    assert err(Y, Y64, 1.0) < 1.2e-2
    X = torch.full((1, 2, 5, 96), 3.0, device="cuda", dtype=torch.bfloat16)
    w, b = torch.ones(2, 96, device="cuda"), torch.full((2, 96), 0.5, device="cuda")
    Y, mean, rstd = api.head_norm_fw(X, w, b)
    assert (Y == 0.5).all()
    d = api.head_norm_bw(X, torch.randn(1, 5, 192, device="cuda").bfloat16(), w, mean, rstd)
    assert torch.isfinite(d["dX"]).all() and not d["dweight"].any()


def test_no_rows():
    X = torch.zeros(2, 3, 0, 64, device="cuda")
    w = torch.ones(3, 64, device="cuda")
    Y, mean, rstd = api.head_norm_fw(X, w)
    assert Y.shape == (2, 0, 192)
    d = api.head_norm_bw(X, Y, w, mean, rstd)
    assert not d["dweight"].any() and not d["dbias"].any()


def test_captured():
    X, w, b, dY = (t.cuda() for t in make(1, 4, 64, 128, torch.bfloat16, True))
    leaves = [t.requires_grad_() for t in (X, w, b)]
    Y = api.head_norm(*leaves)
    want = [Y.detach(), *torch.autograd.grad(Y, leaves, dY)]
    del Y  # an eager graph that holds the leaves ties them to its stream
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.autograd.grad(api.head_norm(*leaves), leaves, dY)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y = api.head_norm(*leaves)
        got = [Y, *torch.autograd.grad(Y, leaves, dY)]
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(want, got))
