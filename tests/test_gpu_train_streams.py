"""The training-step operators on a stream that is not the current one: memory that they took
from the current stream's pool is not handed out again before that stream is done with it."""
import pytest
import torch

from mixture_experts_layer_16_gb300 import MoEBalanceLoss, MoEGradClip, MoELayerNorm
from tests import gpu_util as G

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
SLEEP = 1_000_000_000          # cycles: some 0.5 s


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def handed_out(ptr, size):
    """Whether new tensors of this size in bytes, 4 MB of them or four, overlap [ptr, ptr + size)."""
    new = [torch.empty(size, dtype=torch.uint8, device="cuda")
           for _ in range(max(4, (4 << 20) // max(size, 1024)))]
    return any(t.data_ptr() < ptr + size and ptr < t.data_ptr() + size for t in new)


def check(call):
    """call(stream): tensors of the operator's own making, which nothing else holds."""
    # (held and freed once, so that the pool has blocks to spare and asks the driver for none below)
    spare = [call(None) for _ in range(4)]
    for t in spare[0]:
        handed_out(t.data_ptr(), t.numel() * t.element_size())
    del spare, t
    torch.cuda.synchronize()
    for raw in (False, True):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(SLEEP)
        mine = call(s.cuda_stream if raw else s)
        places = [(t.data_ptr(), t.numel() * t.element_size()) for t in mine]
        del mine
        again = [handed_out(*p) for p in places]
        assert not s.query()        # it was busy all the while
        s.synchronize()
        assert not any(again), again


def test_norm_on_another_stream():
    T, H = 4096, 2048
    x, dy = (torch.randn((T, H), device="cuda").to(BF) for _ in range(2))
    w, b = (torch.randn(H, device="cuda").to(BF) for _ in range(2))

    def fwd(s):
        n = MoELayerNorm(T, H)
        return [n.forward(x, w, b, stream=s), n.mean, n.rstd]

    def bwd(s):
        n = MoELayerNorm(T, H)
        n.forward(x, w, b, stream=s)
        return [*n.backward(dy, x, w, stream=s), n.mean, n.rstd, n.workspace]
    check(fwd)
    check(bwd)


def test_balance_on_another_stream():
    T, E, k = 4096, 128, 4
    lg = torch.randn((T, E), device="cuda")
    idx = torch.topk(lg, k, dim=1).indices.to(torch.int32).contiguous()
    dl = torch.ones(2, device="cuda")

    def fwd(s):
        h = MoEBalanceLoss(T, E, k)
        h.forward(lg, idx, stream=s)
        return [h.losses, h.seq_loss, h.counts, h.tokens, h.lse, h.workspace]

    def bwd(s):
        h = MoEBalanceLoss(T, E, k)
        h.forward(lg, idx, stream=s)
        return [h.backward(lg, dl, stream=s), h.counts, h.tokens, h.workspace]
    check(fwd)
    check(bwd)


def test_clip_on_another_stream():
    g = [torch.randn(100000, device="cuda") for _ in range(3)]
    o = [torch.empty_like(t) for t in g]

    def norm(s):
        c = MoEGradClip(4)
        return [c.norm(g, stream=s), c.workspace]

    def clip(s):
        c = MoEGradClip(4)
        return [c.clip(g, 1.0, out=o, stream=s), c.workspace]
    check(norm)
    check(clip)


def test_capture_with_the_stream_named():
    """A graph captured on a stream that the calls name themselves, with tensors made inside."""
    T, H, E, k = 300, 256, 16, 2
    x, dy = (torch.randn((T, H), device="cuda").to(BF) for _ in range(2))
    w, b = (torch.randn(H, device="cuda").to(BF) for _ in range(2))
    lg = torch.randn((T, E), device="cuda")
    idx = torch.topk(lg, k, dim=1).indices.to(torch.int32).contiguous()
    dl = torch.ones(2, device="cuda")
    n, h, c = MoELayerNorm(T, H), MoEBalanceLoss(T, E, k), MoEGradClip(4)
    g = [torch.randn(5000, device="cuda") for _ in range(3)]
    o = [torch.empty_like(t) for t in g]

    def go(s):
        y = n.forward(x, w, b, stream=s)
        grads = n.backward(dy, x, w, stream=s)
        losses, counts = h.forward(lg, idx, stream=s)
        d = h.backward(lg, dl, stream=s)
        return [y, *grads, losses, counts, d, c.clip(g, 1.0, out=o, stream=s), *o]
    want = [t.clone() for t in go(None)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = go(s)
    for t in (*got, n.mean, n.rstd, h.workspace):
        t.zero_()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, v) for a, v in zip(got, want))
