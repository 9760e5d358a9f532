"""The mLSTM's in-place writes raise the tensors' versions, so that autograd
refuses a backward that kept an overwritten state."""
import pytest
import torch

from mlstm_chunkwise_b200 import api

pytestmark = pytest.mark.gpu

B, NH, T, D = 1, 2, 96, 64
INPUTS = ("Q", "K", "V", "i_pre", "f_pre")


def make():
    gen = torch.Generator().manual_seed(1)
    x = {n: torch.randn(B, NH, T, D, generator=gen).cuda() for n in "QKV"}
    x.update({n: torch.randn(B, NH, T, generator=gen).cuda() for n in ("i_pre", "f_pre")})
    x.update(C0=torch.zeros(B, NH, D, D).cuda(), n0=torch.zeros(B, NH, D).cuda(),
             m0=torch.zeros(B, NH).cuda())
    return x


def test_step_and_forward_on_a_kept_state():
    x = make()
    tok = [x[n][:, :, 0].contiguous() for n in INPUTS]
    for write in (lambda: api.mlstm_step(*tok, x["C0"], x["n0"], x["m0"]),
                  lambda: api.mlstm_fw(*(x[n] for n in INPUTS), out={"C_T": x["C0"]})):
        x["V"] = x["V"].detach().requires_grad_()
        H, _ = api.mlstm_chunkwise(*x.values())
        write()
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            H.sum().backward()


def test_versions():
    x = make()
    h = torch.empty(B, NH, D, device="cuda")
    H = torch.empty(B, NH, T, D, device="cuda")
    api.mlstm_step(*(x[n][:, :, 0].contiguous() for n in INPUTS),
                   x["C0"], x["n0"], x["m0"], h=h)
    assert [t._version for t in (x["C0"], x["n0"], x["m0"], h)] == [1, 1, 1, 1]
    api.mlstm_fw(*x.values(), out={"H": H})
    assert H._version == 1 and x["C0"]._version == 1
