"""Calls of the same kernels with small and large shared memory from two host
threads at once (the binding lets go of the interpreter lock during a call):
each launch is accepted whatever the other thread asks for."""
import threading

import pytest
import torch

import gated_delta_cases as gd
from mlstm_chunkwise_b200 import _lib, api

pytestmark = pytest.mark.gpu

ROUNDS = 1000


def together(works):
    """Runs each of `works` ROUNDS times on a thread and a stream of its own and
    compares every result's bits with those of a call made alone."""
    want = [w() for w in works]
    torch.cuda.synchronize()
    errors, start = [], threading.Barrier(len(works))

    def loop(work, ref):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                start.wait()
                for i in range(ROUNDS):
                    got = work()
                    if i % 250 == 0:
                        assert all(torch.equal(a, b) for a, b in zip(got, ref))
                stream.synchronize()
        except Exception as e:  # noqa: BLE001 (handed to the main thread)
            errors.append(e)

    threads = [threading.Thread(target=loop, args=x) for x in zip(works, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    assert api.last_device_error() == _lib.OK


def test_gated_delta_key_widths():
    def work(DK):
        x = gd.cuda(gd.make(B=1, NHK=1, NH=1, T=64, DK=DK, DV=16, dtype="f32"))
        a = [x[n] for n in gd.NAMES]
        return lambda: api.gated_delta_fw(*a)

    together([work(64), work(1024)])


@pytest.mark.parametrize("backward", [False, True])
def test_norm_widths(backward):
    def work(D):
        X = torch.randn(1, 1, 3, D, device="cuda")
        w = torch.ones(1, D, device="cuda")
        Y, mean, rstd = api.head_norm_fw(X, w)
        if not backward:
            return lambda: api.head_norm_fw(X, w)
        return lambda: tuple(api.head_norm_bw(X, Y, w, mean, rstd).values())

    together([work(4096), work(8192)])
