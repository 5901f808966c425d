"""MoEBalanceLoss on the GPU against the fp64 oracle.

Bounds (e = 2^-24).  A probability's relative error is at most (R + 8) e, R the largest
distance of a logit from its row's maximum (the rounded difference moves the exponential by
that much) plus a few roundings and the row's sum; every further sum (a CTA's tokens, then
at most 152 * 8 pieces, then the sequences) adds positive terms in chains of at most 1300, so
the losses are off by at most (R + 1400) e of themselves.  lse: (|lse| + 16) 2 e.  A logit
gradient's terms: (|c| + <p, |c|> + |z|) (p (2 R + 64) e + 2^-148), the last for a probability
below fp32's normal range (held to 2^-149), plus its storage type's half ulp.
Counts and tokens are exact."""
import numpy as np
import pytest
import torch

import oracle.train as ot
from mixture_experts_layer_16_gb300 import MoEBalanceLoss
from tests import gpu_util as G

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U = {n: torch.finfo(t).eps / 2 for n, t in DT.items()}
SUB = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -149}
E32 = 2.0 ** -24
DL = (0.75, -0.5)


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


def case(T, E, k, n_seq=1, mask=False, dtype="fp32", seed=0, scale=2.0):
    r = np.random.default_rng(seed + T + 31 * E)
    logits = torch.from_numpy((scale * r.standard_normal((T, E))).astype(np.float32)).to(
        "cuda", DT[dtype])
    idx = torch.topk(logits.float(), k, dim=1).indices.to(torch.int32).contiguous()
    off = None
    if n_seq > 1:
        o = np.concatenate([[0], np.sort(r.integers(0, T + 1, n_seq - 1)), [T]])
        if n_seq > 2:
            o[n_seq // 2] = o[n_seq // 2 - 1]        # an empty sequence
        off = torch.from_numpy(o.astype(np.int32)).cuda()
    m = torch.from_numpy(r.random(T) < 0.8).cuda() if mask else None
    return dict(logits=logits, idx=idx, off=off, mask=m, G=n_seq, dtype=dtype)


def run(c, dl=DL):
    T, E = c["logits"].shape
    h = MoEBalanceLoss(T, E, c["idx"].shape[1], c["G"], c["dtype"])
    losses, counts = h.forward(c["logits"], c["idx"], c["off"], c["mask"])
    d = h.backward(c["logits"], torch.tensor(dl, device="cuda"), c["off"], c["mask"])
    torch.cuda.synchronize()
    return h, losses, counts, d


def f64(t):
    return t.double().cpu().numpy()


def check(c, h, losses, counts, d, dl=DL):
    lg = f64(c["logits"])
    idx = c["idx"].cpu().numpy()
    off = None if c["off"] is None else c["off"].cpu().numpy()
    mask = None if c["mask"] is None else c["mask"].cpu().numpy()
    f = ot.balance_forward(lg, idx, c["G"], off, mask)
    assert np.array_equal(counts.cpu().numpy(), f["counts"])
    assert np.array_equal(h.tokens.cpu().numpy(), f["tokens"])
    on = f["lse"] != 0
    fin = np.where(np.isfinite(lg), lg, np.nan)
    rng = 0.0
    if on.any():
        rng = float(np.nanmax(np.nanmax(fin[on], axis=1) - np.nanmin(fin[on], axis=1)))
    rel = (rng + 1400) * E32
    assert np.all(np.abs(f64(h.lse) - f["lse"]) <= (np.abs(f["lse"]) + 16) * 2 * E32)
    assert np.array_equal(f64(h.lse) == 0, f["lse"] == 0)
    assert np.all(np.abs(f64(h.seq_loss) - f["seq_loss"]) <= rel * f["seq_loss"])
    lse2 = (np.abs(f["lse"]) + 16) * 4 * E32 * np.abs(f["lse"])   # of the squares
    got = f64(losses)
    assert abs(got[0] - f["losses"][0]) <= rel * f["losses"][0]
    n = max(int(f["tokens"].sum()), 1)
    assert abs(got[1] - f["losses"][1]) <= rel * f["losses"][1] + lse2.sum() / n
    dl = [float(np.float32(v)) for v in dl]
    want = ot.balance_backward(lg, idx, dl, c["G"], off, mask)
    live = max(int((f["tokens"] > 0).sum()), 1)
    E, k = lg.shape[1], idx.shape[1]
    o = [0, len(lg)] if off is None else off
    bound = np.zeros_like(want)
    for s in range(c["G"]):
        ns = int(f["tokens"][s])
        for t in range(o[s], o[s + 1]):
            if f["lse"][t] == 0 and not want[t].any():
                continue
            p = ot.softmax(lg[t])
            cc = abs(dl[0]) * E / (k * ns * ns * live) * f["counts"][s]
            bound[t] = (cc + p @ cc + abs(dl[1] * 2 * f["lse"][t] / n)) * \
                (p * (2 * rng + 64) * E32 + 2.0 ** -148)
    bound += U[c["dtype"]] * np.abs(want) + (want != 0) * SUB[c["dtype"]]
    bad = np.abs(f64(d) - want) > bound
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3])
    return f


@pytest.mark.parametrize("T,E,k,n_seq,mask", [
    (1, 1, 1, 1, False), (1, 8, 2, 1, False), (3, 5, 5, 1, True), (64, 8, 2, 1, False),
    (100, 33, 4, 3, True), (257, 64, 8, 1, False), (500, 128, 8, 7, True), (300, 130, 6, 2, False),
    (200, 256, 8, 40, True), (90, 257, 3, 5, False), (70, 512, 8, 2, True), (40, 1001, 16, 3, True),
    (33, 1024, 32, 1, False), (1500, 16, 4, 200, True), (2100, 6, 2, 1, True)])
def test_balance(T, E, k, n_seq, mask):
    c = case(T, E, k, n_seq, mask)
    check(c, *run(c))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,E,k,n_seq", [(77, 8, 2, 1), (130, 60, 4, 4), (65, 63, 4, 4),
                                         (50, 300, 8, 2)])
def test_balance_16_bit_logits(dtype, T, E, k, n_seq):
    c = case(T, E, k, n_seq, True, dtype)
    check(c, *run(c))


@pytest.mark.parametrize("T,E,k,n_seq", [
    (768, 8, 2, 1), (769, 8, 2, 1), (384, 8, 2, 2), (385, 8, 2, 2), (192, 128, 8, 1),
    (193, 128, 8, 1), (96, 256, 8, 2), (48, 512, 8, 1), (49, 1000, 8, 1), (384, 16, 3, 1)])
def test_balance_around_one_cta(T, E, k, n_seq):
    """Sizes up to which one CTA takes every token, and above."""
    c = case(T, E, k, n_seq, True)
    check(c, *run(c))


@pytest.mark.parametrize("off", [[0, 0, 90], [0, 90, 90], [20, 20, 20], [7, 40, 83], [0, 90]])
@pytest.mark.parametrize("stale", [0x00, 0xff])
def test_balance_few_tokens_and_empty_sequences(off, stale):
    """One CTA: sequences without tokens and tokens in no sequence, over old results."""
    c = case(90, 24, 3, len(off) - 1, True)
    h = MoEBalanceLoss(90, 24, 3, len(off) - 1)
    for t in (h.losses, h.seq_loss, h.counts, h.tokens, h.lse, h.workspace):
        t.view(torch.uint8).fill_(stale)
    c["off"] = torch.tensor(off, dtype=torch.int32, device="cuda")
    losses, counts = h.forward(c["logits"], c["idx"], c["off"], c["mask"])
    d = h.backward(c["logits"], torch.tensor(DL, device="cuda"), c["off"], c["mask"])
    a, b = off[0], off[-1]
    idx, mask, o = c["idx"].cpu().numpy()[a:b], c["mask"].cpu().numpy()[a:b], np.array(off) - a
    if a == b:
        assert not losses.any() and not counts.any() and not h.tokens.any()
        assert not h.seq_loss.any() and not h.lse.any() and not d.any()
        return
    f = ot.balance_forward(f64(c["logits"])[a:b], idx, c["G"], o, mask)
    assert np.array_equal(counts.cpu().numpy(), f["counts"])
    assert np.array_equal(h.tokens.cpu().numpy(), f["tokens"])
    assert np.all(np.abs(f64(h.seq_loss) - f["seq_loss"]) <= 1420 * E32 * f["seq_loss"])
    assert np.all(np.abs(f64(losses) - f["losses"]) <= 1420 * E32 * f["losses"])
    assert not h.lse[:a].any() and not h.lse[b:].any() and not d[:a].any() and not d[b:].any()


def test_balance_many_tokens():
    c = case(20000, 16, 2, 9, True)
    check(c, *run(c))


def test_balance_large_and_masked_logits():
    """Logits in the hundreds; experts masked by -inf and by fp32's lowest value; a token
    with nothing left; a token with a single expert left."""
    c = case(60, 16, 2, 3, True, scale=150.0)
    lg = c["logits"]
    lg[:, 5] = -float("inf")
    lg[10:20, 3] = torch.finfo(torch.float32).min
    lg[7] = -float("inf")
    lg[30, 1:] = -float("inf")
    c["mask"][30] = True
    h, losses, counts, d = run(c)
    # (fp32's lowest value is a distance no exponential sees: take it out of the range)
    c2 = dict(c, logits=torch.where(lg < -1e30, torch.full_like(lg, -float("inf")), lg))
    check(c2, h, losses, counts, d)
    assert not d[7].any() and float(h.lse[7]) == 0.0 and not d[:, 5].any()


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_balance_rows_of_the_lowest_value(dtype):
    """A row masked throughout with its type's lowest value is an even distribution."""
    c = case(40, 24, 3, 2, dtype=dtype)
    c["logits"][5] = torch.finfo(DT[dtype]).min
    c["logits"][6, 2:] = torch.finfo(DT[dtype]).min
    h, losses, counts, d = run(c, dl=(1.0, 0.0))
    f = ot.balance_forward(f64(c["logits"]), c["idx"].cpu().numpy(), 2, c["off"].cpu().numpy())
    assert np.array_equal(counts.cpu().numpy(), f["counts"]) and int(h.tokens.sum()) == 40
    assert abs(float(losses[0]) - f["losses"][0]) <= 1420 * E32 * f["losses"][0]
    assert abs(float(h.lse[5]) - f["lse"][5]) <= 4 * E32 * abs(f["lse"][5])
    want = ot.balance_backward(f64(c["logits"]), c["idx"].cpu().numpy(), (1.0, 0.0), 2,
                               c["off"].cpu().numpy())
    # the terms' size: p (c + <p, c>) <= 2 max c = 2 E counts / (k n^2 S)
    cmax = 2 * 24 * f["counts"].max() / (3 * max(f["tokens"].min(), 1) ** 2)
    assert np.abs(f64(d) - want).max() <= 100 * E32 * cmax + U[dtype] * np.abs(want).max()


def test_balance_nothing_counts():
    for n_seq in (1, 4):
        c = case(50, 8, 2, n_seq)
        c["mask"] = torch.zeros(50, dtype=torch.bool, device="cuda")
        h, losses, counts, d = run(c)
        assert not losses.any() and not counts.any() and not d.any() and not h.lse.any()
        assert not h.seq_loss.any() and not h.tokens.any()


def test_balance_offsets_past_32_bits():
    """4.3e9 logits: the last sequence against a call on its tokens alone.  Probabilities and
    counts are the same, sums over tokens are added in another order."""
    E, k, last = 1024, 2, 101
    T = (1 << 22) + last
    lg = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    c = case(last, E, k, dtype="bf16")
    lg[-last:], idx[-last:] = c["logits"], c["idx"]
    off = torch.tensor([0, T - last, T], dtype=torch.int32, device="cuda")
    dl = torch.tensor([1.0, 0.0], device="cuda")
    one, two = MoEBalanceLoss(last, E, k, 1, "bf16"), MoEBalanceLoss(T, E, k, 2, "bf16")
    one.forward(c["logits"], c["idx"])
    two.forward(lg, idx, off)
    assert torch.equal(two.counts[1], one.counts[0]) and two.tokens.tolist() == [T - last, last]
    assert torch.equal(two.lse[-last:], one.lse)
    assert int(two.counts[0, 0]) == k * (T - last)
    assert abs(float(two.seq_loss[1] - one.seq_loss[0])) <= 400 * E32 * float(one.seq_loss[0])
    d1 = f64(one.backward(c["logits"], dl))
    d2 = f64(two.backward(lg, dl, off)[-last:])
    # (half of it: two sequences; each is rounded once)
    assert np.all(np.abs(2 * d2 - d1) <= 2.0 ** -7 * np.abs(d1))


def test_balance_masked_garbage_does_not_count():
    c = case(120, 24, 3, 5, True)
    want = [t.clone() for t in run(c)[1:]]
    off = ~c["mask"]
    c["logits"][off] = float("nan")
    c["idx"][off] = 2 ** 30
    got = run(c)[1:]
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_balance_nan_shows():
    c = case(40, 8, 2, 2)
    c["logits"][3, 1] = float("nan")
    h, losses, _, d = run(c)
    assert losses.isnan().all() and d[3].isnan().all()
    o = c["off"].cpu()
    s = 0 if o[0] <= 3 < o[1] else 1
    assert h.seq_loss[s].isnan() and not h.seq_loss[1 - s].isnan()


def test_balance_indices_out_of_range_are_dropped():
    c = case(90, 12, 4, 3)
    c["idx"][::3, 1] = -1
    c["idx"][::4, 2] = 12
    check(c, *run(c))


def test_balance_tokens_outside_every_sequence():
    T = 200
    c = case(T, 16, 2, 3)
    c["off"] = torch.tensor([10, 60, 60, 150], dtype=torch.int32, device="cuda")
    h, losses, counts, d = run(c)
    sub = dict(c, logits=c["logits"][10:150].contiguous(), idx=c["idx"][10:150].contiguous(),
               off=(c["off"] - 10).contiguous())
    f = ot.balance_forward(f64(sub["logits"]), sub["idx"].cpu().numpy(), 3,
                           sub["off"].cpu().numpy())
    assert np.array_equal(counts.cpu().numpy(), f["counts"])
    assert np.allclose(f64(losses), f["losses"], rtol=1400 * E32)
    out = torch.ones(T, dtype=torch.bool)
    out[10:150] = False
    assert not d[out.cuda()].any() and not h.lse[out.cuda()].any()
    assert d[~out.cuda()].any(dim=1).all()


def test_balance_unaligned_logits():
    c = case(70, 32, 4, 2, True)
    want = [t.clone() for t in run(c)[1:]]
    b = torch.empty(70 * 32 + 1, device="cuda")[1:].view(70, 32)
    c["logits"] = b.copy_(c["logits"])
    for a, w in zip(run(c)[1:], want):
        assert torch.equal(a, w)


def test_balance_gradient_against_differences():
    c = case(80, 20, 3, 4, True)
    _, _, _, d = run(c)
    lg, idx = f64(c["logits"]), c["idx"].cpu().numpy()
    off, mask = c["off"].cpu().numpy(), c["mask"].cpu().numpy()
    v = np.random.default_rng(2).standard_normal(lg.shape)
    h = 1e-5
    L = lambda z: np.dot(DL, ot.balance_forward(z, idx, 4, off, mask)["losses"])
    num = (L(lg + h * v) - L(lg - h * v)) / (2 * h)
    assert abs(num - (f64(d) * v).sum()) <= 1e-5 * np.abs(f64(d) * v).sum()


def test_balance_repeats_streams_and_graph():
    c = case(3000, 64, 6, 11, True)
    h, losses, counts, d = run(c)
    want = [t.clone() for t in (losses, counts, h.lse, h.seq_loss, d)]
    dl = torch.tensor(DL, device="cuda")
    d2 = torch.empty_like(d)

    def go(stream=None):
        h.forward(c["logits"], c["idx"], c["off"], c["mask"], stream=stream)
        h.backward(c["logits"], dl, c["off"], c["mask"], dlogits=d2, stream=stream)

    def same():
        return all(torch.equal(a, b) for a, b in
                   zip((h.losses, h.counts, h.lse, h.seq_loss, d2), want))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    go(s)
    s.synchronize()
    assert same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        go()
    for _ in range(2):
        for t in (h.losses, h.counts, h.lse, h.seq_loss, d2, h.workspace):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert same()
