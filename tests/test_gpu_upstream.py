"""Upstream gradients as autograd hands them on: slices that start off a 16-byte
boundary (two calls' outputs joined), expanded ones, and a backward run twice."""
import pytest
import torch

import gated_delta_cases as gd
from mlstm_chunkwise_b200 import api

pytestmark = pytest.mark.gpu


def both(calls, leaves):
    """Gradients through torch.cat of the calls' outputs, and of each call alone
    from gradients of its own."""
    outs = [c() for c in calls]
    up = [torch.randn_like(o) for o in outs]
    assert up[0].numel() * up[0].element_size() % 16  # the second slice starts there
    got = torch.autograd.grad(torch.cat(outs), leaves, torch.cat(up))
    want = [torch.autograd.grad(c(), x, u) for c, x, u in
            zip(calls, (leaves[:len(leaves) // 2], leaves[len(leaves) // 2:]), up)]
    assert all(torch.equal(a, b) for a, b in zip(got, (*want[0], *want[1])))


def cells():
    xs = [gd.cuda(gd.make(NHK=1, NH=1, T=33, DK=9, DV=7, dtype="f32", seed=s)) for s in (1, 2)]
    return [{n: v.requires_grad_() for n, v in x.items()} for x in xs]


@pytest.mark.parametrize("part", [0, 1])
def test_gated_delta(part):
    xs = cells()
    both([lambda x=x: api.gated_delta_chunkwise(*(x[n] for n in gd.NAMES))[part] for x in xs],
         [x[n] for x in xs for n in gd.NAMES])


def test_norm():
    Xs = [torch.randn(1, 1, 33, 7, device="cuda", requires_grad=True) for _ in range(2)]
    w = torch.ones(1, 7, device="cuda")
    both([lambda X=X: api.head_norm(X, w) for X in Xs], Xs)


def test_mlstm():
    xs = [[torch.randn(1, 1, 33, d, device="cuda", requires_grad=True) for d in (9, 9, 7)] +
          [torch.randn(1, 1, 33, device="cuda", requires_grad=True) for _ in range(2)]
          for _ in range(2)]
    both([lambda x=x: api.mlstm_chunkwise(*x)[0] for x in xs], [t for x in xs for t in x])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_expanded_and_twice(dtype):
    x = {n: v.requires_grad_() for n, v in gd.cuda(gd.make(T=150, dtype=dtype)).items()}
    H, C = api.gated_delta_chunkwise(*(x[n] for n in gd.NAMES))
    loss = H.float().sum() + 0.5 * C.sum()
    first = torch.autograd.grad(loss, list(x.values()), retain_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(first, torch.autograd.grad(loss, list(x.values()))))
    d = {n: v.detach() for n, v in x.items()}
    want = api.gated_delta_bw(*(d[n] for n in gd.NAMES[:5]), torch.ones_like(d["V"]), d["C0"],
                              torch.full_like(d["C0"], 0.5))
    assert all(torch.equal(a, want["d" + n]) for n, a in zip(x, first))
