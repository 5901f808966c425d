"""Calls of several host threads, each with its own handle, tensors and stream: the same kernels
at sizes that need different amounts of shared memory.  No call may be refused because another
thread's came between, and the results are those of calls made alone, bit for bit."""
import threading

import pytest
import torch

from mixture_experts_layer_16_gb300 import MoEBalanceLoss, MoELayerNorm
from tests import gpu_util as G

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def together(makers, rounds):
    """makers: functions (stream) -> (call, outputs).  Each call is made once alone, then `rounds`
    times beside the other threads' calls."""
    jobs, errors = [], []
    for make in makers:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        call, outs = make(s)
        call()
        torch.cuda.synchronize()
        jobs.append((call, outs, [t.clone() for t in outs]))
    torch.cuda.synchronize()
    start = threading.Barrier(len(jobs))

    def work(call):
        start.wait()
        try:
            for _ in range(rounds):
                call()
        except Exception as e:
            errors.append(e)

    threads = [threading.Thread(target=work, args=(call,)) for call, _, _ in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for _, outs, want in jobs:
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def norm_job(T, H, back):
    def make(s):
        gen = torch.Generator(device="cuda").manual_seed(T)
        x, dy, y, dx = (torch.randn((T, H), generator=gen, device="cuda").to(BF) for _ in range(4))
        w, b, dw, db = (torch.randn(H, generator=gen, device="cuda").to(BF) for _ in range(4))
        n = MoELayerNorm(T, H)
        n.forward(x, w, b, y=y)
        if back:
            return lambda: n.backward(dy, x, w, out=(dx, dw, db), stream=s), (dx, dw, db)
        return lambda: n.forward(x, w, b, y=y, stream=s), (y, n.mean, n.rstd)
    return make


@pytest.mark.parametrize("back,sizes", [(False, (700, 4096)), (True, (300, 4096))])
def test_norm_in_two_threads(back, sizes):
    together([norm_job(T, 2048, back) for T in sizes], 5000)


def balance_job(T, E, n_seq, back):
    def make(s):
        gen = torch.Generator(device="cuda").manual_seed(E + n_seq)
        lg = torch.randn((T, E), generator=gen, device="cuda")
        idx = torch.topk(lg, 4, dim=1).indices.to(torch.int32).contiguous()
        off = (torch.arange(n_seq + 1, device="cuda") * T // n_seq).to(torch.int32)
        h = MoEBalanceLoss(T, E, 4, n_seq)
        h.forward(lg, idx, off)
        dl, d = torch.ones(2, device="cuda"), torch.empty_like(lg)
        if back:
            return lambda: h.backward(lg, dl, off, dlogits=d, stream=s), (d,)
        return lambda: h.forward(lg, idx, off, stream=s), (h.losses, h.counts, h.lse)
    return make


@pytest.mark.parametrize("back,a,b", [(False, (3000, 132, 1), (3000, 256, 1)),
                                      (True, (2000, 1024, 1), (2000, 1024, 200))])
def test_balance_in_two_threads(back, a, b):
    together([balance_job(*a, back), balance_job(*b, back)], 5000)
