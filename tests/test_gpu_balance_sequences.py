"""MoEBalanceLoss of sequences of very different lengths: a single token in many, all but one of which
are empty; one of nearly all tokens among many short ones."""
import pytest
import torch

import oracle.train as ot
from mixture_experts_layer_16_gb300 import MoEBalanceLoss
from tests import gpu_util as G
from tests.test_gpu_balance import DL, E32, case, check, f64, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


# the last: 2^31 counts and tokens, where their number leaves 32 bits
@pytest.mark.parametrize("E,n_seq,at", [(24, 1, 0), (24, 2, 1), (24, 3, 0), (24, 3, 2), (24, 600, 599),
                                        (5, 70000, 1234), (127, 1 << 24, (1 << 24) - 7)])
def test_balance_one_token_in_many_sequences(E, n_seq, at):
    """Over old results: every empty sequence's are zero."""
    gen = torch.Generator(device="cuda").manual_seed(E)
    lg = torch.randn((1, E), generator=gen, device="cuda")
    idx = torch.topk(lg, 3, dim=1).indices.to(torch.int32).contiguous()
    off = (torch.arange(n_seq + 1, device="cuda") > at).to(torch.int32)
    h = MoEBalanceLoss(1, E, 3, n_seq)
    for t in (h.losses, h.seq_loss, h.counts, h.tokens, h.lse, h.workspace):
        t.view(torch.uint8).fill_(0xff)
    losses, counts = h.forward(lg, idx, off)
    d = h.backward(lg, torch.tensor(DL, device="cuda"), off)
    f = ot.balance_forward(f64(lg), idx.cpu().numpy())
    assert torch.equal(counts[at].cpu(), torch.from_numpy(f["counts"][0]).int())
    assert int(h.tokens[at]) == 1
    # (a row of E probabilities, one token: the bounds of the larger cases hold)
    assert abs(float(h.seq_loss[at]) - f["seq_loss"][0]) <= 1420 * E32 * f["seq_loss"][0]
    assert abs(float(losses[0]) - f["losses"][0]) <= 1420 * E32 * f["losses"][0]
    assert abs(float(losses[1]) - f["losses"][1]) <= 1420 * E32 * (f["losses"][1] + 1)
    assert abs(float(h.lse) - f["lse"][0]) <= (abs(f["lse"][0]) + 16) * 2 * E32
    want = ot.balance_backward(f64(lg), idx.cpu().numpy(), DL)
    assert abs(f64(d) - want).max() <= 200 * E32 * (E + abs(f["lse"][0]))
    counts[at], h.tokens[at], h.seq_loss[at] = 0, 0, 0.0
    assert not counts.any() and not h.tokens.any() and not h.seq_loss.any()


@pytest.mark.parametrize("E,k,n_seq", [(16, 2, 64), (130, 4, 60)])
def test_balance_one_long_sequence_among_short_ones(E, k, n_seq):
    """One sequence of nearly all tokens, in some hundred pieces, and many of a few tokens."""
    T, at = 20000, n_seq // 3
    c = case(T, E, k, mask=True)
    lengths = torch.arange(n_seq) * 5 % 4
    lengths[at] = 0
    lengths[at] = T - int(lengths.sum())
    off = torch.cat([torch.zeros(1, dtype=torch.int64), lengths.cumsum(0)])
    c.update(off=off.to(torch.int32).cuda(), G=n_seq)
    check(c, *run(c))
