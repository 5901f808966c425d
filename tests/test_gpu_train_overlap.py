"""What may lie over or between one another in the training-step operators, and what may not."""
import pytest
import torch

from mixture_experts_layer_16_gb300 import MoEBalanceLoss, MoELayerNorm
from mixture_experts_layer_16_gb300.binding import MoEError
from tests import gpu_util as G

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    G.ensure_built()


# rows in one read (whole units, cut anywhere, two a barrier) and looped ones
@pytest.mark.parametrize("T,H", [(40, 256), (40, 250), (700, 4096), (5, 20001), (5, 20000), (1, 64)])
def test_norm_operands_between_and_over_one_another(T, H):
    gen = torch.Generator(device="cuda").manual_seed(H)
    rows = [torch.randn((T, H), generator=gen, device="cuda").to(BF) for _ in range(3)]
    w, b = (torch.randn(H, generator=gen, device="cuda").to(BF) for _ in range(2))
    x, dy, add = rows
    n = MoELayerNorm(T, H)
    y = n.forward(x, w, b)
    dx, dw, db = n.backward(dy, x, w, dx_add=add)
    pad = -H % 8                     # (parts that are cut alike)
    wide = torch.zeros((T, 5 * (H + pad)), dtype=BF, device="cuda")
    p = [wide[:, i * (H + pad):i * (H + pad) + H] for i in range(5)]
    for t, v in zip(p, rows):
        t.copy_(v)
    assert torch.equal(n.forward(p[0], w, b, y=p[3]), y)
    out = n.backward(p[1], p[0], w, dx_add=p[2],
                     out=(p[4], torch.empty_like(w), torch.empty_like(b)))
    if pad == 0 or T == 1:           # (else the rows above were cut otherwise, summed in another order)
        assert all(torch.equal(a, v) for a, v in zip(out, (dx, dw, db)))
    assert all(torch.equal(t, v) for t, v in zip(p, rows))
    for over in (p[0], p[1]):        # x, dy
        with pytest.raises(MoEError):
            n.backward(p[1], p[0], w, out=(over, dw, db))
    with pytest.raises(MoEError):
        n.forward(p[0], w, b, y=wide[:, 1:1 + H])
    flat = torch.zeros(T * H + H, dtype=BF, device="cuda")
    x2, y2 = flat[:T * H].view(T, H), flat[H // 2:H // 2 + T * H].view(T, H)
    with pytest.raises(MoEError):
        n.forward(x2, w, b, y=y2)
    with pytest.raises(MoEError):
        n.backward(dy, x, w, dx_add=x2, out=(y2, dw, db))
    x2.copy_(x)
    assert torch.equal(n.forward(x2, w, b, y=x2), y)         # in place
    x2.copy_(add)
    n.forward(x, w, b)
    got = n.backward(dy, x, w, dx_add=x2, out=(x2, dw.clone(), db.clone()))
    assert torch.equal(got[0], dx) and torch.equal(got[1], dw)


@pytest.mark.parametrize("E", [8, 33])
def test_balance_gradient_beside_the_logits(E):
    T, k = 200, 2
    both = torch.zeros((2 * T + 1, E), device="cuda")
    lg, d = both[:T], both[T:2 * T]
    lg.normal_()
    idx = torch.topk(lg, k, dim=1).indices.to(torch.int32).contiguous()
    dl = torch.tensor([1.0, 0.5], device="cuda")
    h = MoEBalanceLoss(T, E, k)
    h.forward(lg, idx)
    want = h.backward(lg, dl)
    assert torch.equal(h.backward(lg, dl, dlogits=d), want) and not both[2 * T].any()
    for over in (lg, both[T - 1:2 * T - 1], both[1:T + 1]):
        with pytest.raises(MoEError):
            h.backward(lg, dl, dlogits=over)
