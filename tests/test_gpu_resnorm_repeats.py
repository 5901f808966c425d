"""The residual norm's forward over long loops of rows, with every set of norms: the same bits at each call,
and the oracle's values.  (A group of threads adds up a row with one barrier a sum, so that neighbouring
sums need different buffers, whichever sums a row has.)"""
import pytest
import torch

from mixture_experts_layer_16_gb300 import MoEResidualNorm
from tests import gpu_util as G
from tests.test_gpu_resnorm import EPS, TYPES, check_forward, data

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


# 152 CTAs of up to 512 threads: some tens of rows to every group
@pytest.mark.parametrize("T,H", [(20000, 520), (20000, 1024), (9000, 2048), (6000, 2056), (6000, 4096),
                                 (3001, 5120), (9000, 1023), (40000, 256)])
@pytest.mark.parametrize("types", [TYPES[1], TYPES[3], TYPES[0]])
@pytest.mark.parametrize("post,pre", [(True, False), (True, True), (False, True)])
def test_repeats(T, H, types, post, pre):
    few = 40
    d = data(few, H, *types, post, "channel", pre)
    # rows of very different sizes next to one another, so that a sum of another row shows
    at = torch.arange(T, device="cuda") % few
    size = torch.exp2((torch.arange(T, device="cuda") * 7 % 13 - 6).float())[:, None]
    x, f = d["x"][at].contiguous(), (d["f"][at].float() * size).to(d["f"].dtype)
    h = MoEResidualNorm(T, H, *types, post=post, gate="channel", pre=pre, scale=0.7, eps=EPS)
    p = dict(post_weight=d["post_weight"], gate=d["gate"], pre_weight=d["pre_weight"])
    first = None
    for _ in range(10):
        out, n = h.forward(x, f, **p)
        got = [t.clone() for t in (out, n, h.rstd_f, h.rstd_out) if t is not None]
        if first is None:
            first = got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    # a few rows of every part of the loop against the oracle
    rows = torch.arange(0, T, T // 97, device="cuda")
    s = MoEResidualNorm(len(rows), H, *types, post=post, gate="channel", pre=pre, scale=0.7, eps=EPS)
    s.rstd_f, s.rstd_out = (None if t is None else t[rows] for t in (h.rstd_f, h.rstd_out))
    check_forward(s, {**d, "x": x[rows], "f": f[rows]}, types, out[rows], None if n is None else n[rows])
