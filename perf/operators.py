"""Timed cases of the operators around the expert layer in a training step: layer
normalisation (forward, backward), the router's balance and z losses (forward,
backward), and the global gradient norm with clipping.

`listed()` gives the cases, `draw()` more of the same ranges, `prepare()` a case's
inputs, `run()` one pass through its operator (the library's when `own` is set, else a
plain form in 32-bit torch operations), `work()` the bytes and operations the pass cannot
do without, and `exact()` the same outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

_TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_EPS = 1e-5          # of the layer norm
_CLIP_EPS = 1e-6     # added to the gradient norm before the division


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one token in front of the layer, as in decoding: nothing but latency
        dict(name="norm_fwd_token", op="norm_fwd", T=1, H=2048, dtype="bf16", param="bf16",
             bias=True),
        # the benchmark layer's input, a training step's micro-batch
        dict(name="norm_fwd_layer", op="norm_fwd", T=16384, H=2048, dtype="bf16", param="bf16",
             bias=True),
        # an odd width and an odd number of rows in fp32, no bias
        dict(name="norm_fwd_odd", op="norm_fwd", T=5003, H=1111, dtype="fp32", param="fp32",
             bias=False),
        # the tiny layer's backward, residual gradient joined in
        dict(name="norm_bwd_tiny", op="norm_bwd", T=64, H=128, dtype="bf16", param="bf16",
             bias=True, add=True),
        # the benchmark layer's backward: dx with the residual's gradient, dweight, dbias
        dict(name="norm_bwd_layer", op="norm_bwd", T=16384, H=2048, dtype="bf16", param="bf16",
             bias=True, add=True),
        # the wide layer's width, fp16 activations under fp32 parameters, ragged rows
        dict(name="norm_bwd_wide", op="norm_bwd", T=8191, H=4096, dtype="fp16", param="fp32",
             bias=True, add=False),
        # the tiny layer's router: 8 experts, one sequence
        dict(name="balance_fwd_tiny", op="balance_fwd", T=64, E=8, k=2, G=1, mask=False,
             dtype="fp32"),
        # a long packed batch: 256 experts, 96 ragged sequences (some empty), padding masked
        dict(name="balance_fwd_packed", op="balance_fwd", T=131072, E=256, k=8, G=96, mask=True,
             dtype="fp32"),
        # the benchmark layer's router gradient, 16 ragged sequences
        dict(name="balance_bwd_layer", op="balance_bwd", T=16384, E=128, k=8, G=16, mask=True,
             dtype="fp32"),
        # the tiny layer's gradients, clipped into fp32 gradients for the optimiser
        dict(name="clip_tiny", op="clip", sizes=0, n=6, total=0, dtypes="bf16", out="fp32"),
        # many tensors of odd sizes and all three types, norm under the bound: in place
        dict(name="clip_many", op="clip", sizes=7, n=48, total=200_000_000, dtypes="mixed",
             out="inplace"),
        # the benchmark layer's gradients (three expert weights, router, norm), clipped
        dict(name="clip_layer", op="clip", sizes=1, n=6, total=0, dtypes="bf16", out="same"),
    ]


def _log_int(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "balance_fwd", "balance_bwd", "clip"])
    if op.startswith("norm"):
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        H = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:       # most widths are multiples of 64, the rest any
            H = max(64, H // 64 * 64)
        if H == 3072:
            H += 64
        T = _log_int(rng, 1, min(32768, 33_554_432 // H))
        case = dict(op=op, T=T, H=H, dtype=dtype, param=rng.choice([dtype, "fp32"]),
                    bias=rng.random() < 0.7)
        if op == "norm_bwd":
            case["add"] = rng.random() < 0.5
        return case
    if op.startswith("balance"):
        E = _log_int(rng, 4, 512)
        if rng.random() < 0.6:
            E = max(8, E // 8 * 8)
        T = _log_int(rng, 1, 131072)
        return dict(op=op, T=T, E=E, k=min(E, rng.choice([1, 2, 4, 6, 8])),
                    G=_log_int(rng, 1, min(T, 256)), mask=rng.random() < 0.5,
                    dtype=rng.choice(["fp32", "fp32", "bf16"]))
    n = _log_int(rng, 1, 60)
    return dict(op=op, sizes=rng.randrange(2, 1 << 30), n=n,
                total=_log_int(rng, 1000 + n, 300_000_000),
                dtypes=rng.choice(["bf16", "fp32", "mixed"]),
                out=rng.choice(["inplace", "same", "fp32"]))


def _clip_sizes(case):
    """(elements, type) of every tensor of a clip case."""
    if case["sizes"] in (0, 1):      # the tiny / the benchmark layer's parameters
        E, I, H = (8, 64, 128) if case["sizes"] == 0 else (128, 768, 2048)
        return [(n, "bf16") for n in (E * I * H, E * I * H, E * H * I, E * H, H, H)]
    r = np.random.default_rng(case["sizes"])
    share = np.exp(r.normal(0.0, 1.5, case["n"]))
    sizes = np.maximum(1, (share / share.sum() * case["total"]).astype(np.int64))
    names = ["bf16", "fp16", "fp32"] if case["dtypes"] == "mixed" else [case["dtypes"]]
    return [(int(s), names[int(i)]) for s, i in zip(sizes, r.integers(0, len(names), case["n"]))]


# -------------------------------------------------------------------------- inputs
def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _norm_inputs(case, gen):
    T, H = case["T"], case["H"]
    dt, pt = _TORCH[case["dtype"]], _TORCH[case["param"]]
    # a residual stream: unit noise, a per-channel offset, a few channels far larger
    scale = torch.ones(H, device="cuda")
    scale[:: max(1, H // 8)] = 12.0
    x = (_randn(gen, T, H) * scale + 0.3 * _randn(gen, H)).to(dt)
    s = dict(x=x, weight=(1.0 + 0.1 * _randn(gen, H)).to(pt),
             bias=(0.1 * _randn(gen, H)).to(pt) if case["bias"] else None)
    if case["op"] == "norm_bwd":
        s["dy"] = _randn(gen, T, H).to(dt)
        s["dx_add"] = _randn(gen, T, H).to(dt) if case["add"] else None
    return s


def _balance_inputs(case, gen, seed):
    T, E, k, G = case["T"], case["E"], case["k"], case["G"]
    # uneven experts: a popularity that falls off with the rank, over a random order
    rank = torch.randperm(E, generator=gen, device="cuda").float()
    logits = (_randn(gen, T, E) - 0.5 * torch.log1p(rank)).to(_TORCH[case["dtype"]])
    topk_idx = torch.topk(logits.float(), k, dim=1).indices.to(torch.int32).contiguous()
    r = np.random.default_rng(seed)
    off = np.concatenate([[0], np.sort(r.integers(0, T + 1, G - 1)), [T]]).astype(np.int64)
    if G > 2:
        off[G // 2] = off[G // 2 - 1]                # one sequence without a token
    mask = None
    if case["mask"]:                                 # the tail of each sequence is padding
        m = np.ones(T, dtype=np.uint8)
        for a, b in zip(off[:-1], off[1:]):
            m[int(a + math.ceil((b - a) * r.uniform(0.8, 1.0))):int(b)] = 0
        mask = torch.from_numpy(m).cuda()
    return dict(logits=logits, topk_idx=topk_idx, mask=mask,
                seq_offsets=torch.from_numpy(off.astype(np.int32)).cuda() if G > 1 else None)


def _clip_inputs(case, gen):
    grads, sq = [], 0.0
    for n, name in _clip_sizes(case):
        g = torch.empty(n, device="cuda", dtype=_TORCH[name])
        for a in range(0, n, 1 << 27):               # bounds the fp32 draw's memory
            b = min(n, a + (1 << 27))
            g[a:b] = 1e-3 * _randn(gen, b - a)
        grads.append(g)
        sq += 1e-6 * n
    if case["out"] == "inplace":                     # a calm step: the norm is under the bound
        return dict(grads=grads, out=None, max_norm=2.0 * math.sqrt(sq))
    dts = [torch.float32 if case["out"] == "fp32" else g.dtype for g in grads]
    return dict(grads=grads, out=[torch.empty(g.shape, device="cuda", dtype=d)
                                  for g, d in zip(grads, dts)],
                max_norm=0.3 * math.sqrt(sq))


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * (seed % (1 << 31)) + 17)
    if case["op"].startswith("norm"):
        return _norm_inputs(case, gen)
    if case["op"].startswith("balance"):
        return _balance_inputs(case, gen, seed)
    return _clip_inputs(case, gen)


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=case)
    op = case["op"]
    if op == "norm_bwd" and not own:                 # what the forward kept
        x = s["x"].float()
        s["mean"] = x.mean(1)
        s["rstd"] = torch.rsqrt((x - s["mean"][:, None]).square().mean(1) + _EPS)
    if op == "balance_bwd":
        s["dlosses"] = torch.tensor([1e-2, 1e-3], device="cuda")   # the losses' coefficients
        if not own:
            s["counts"], s["n"] = _counts(s)
    if own:
        import mixture_experts_layer_16_gb300 as M
        if op.startswith("norm"):
            s["norm"] = M.MoELayerNorm(case["T"], case["H"], case["dtype"], case["param"],
                                       eps=_EPS, bias=case["bias"])
            if op == "norm_bwd":
                s["norm"].forward(s["x"], s["weight"], s["bias"])
        elif op.startswith("balance"):
            s["loss"] = M.MoEBalanceLoss(case["T"], case["E"], case["k"], case["G"],
                                         case["dtype"])
            if op == "balance_bwd":
                s["loss"].forward(s["logits"], s["topk_idx"], s["seq_offsets"], s["mask"])
        else:
            s["clip"] = M.MoEGradClip(len(s["grads"]))
    return s


# --------------------------------------------------------------------- plain forms
def _token_groups(s):
    """The sequence of every token, and whether the token counts."""
    T = s["logits"].shape[0]
    tok = torch.arange(T, device="cuda")
    if s["seq_offsets"] is None:
        seq = torch.zeros(T, dtype=torch.int64, device="cuda")
    else:
        seq = (torch.searchsorted(s["seq_offsets"].long(), tok, right=True) - 1)
    keep = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"] != 0
    return seq, keep


def _counts(s):
    """Per sequence: routed pairs of each expert, and tokens that count."""
    case = s["case"]
    seq, keep = _token_groups(s)
    E, G = case["E"], case["G"]
    flat = (seq[:, None] * E + s["topk_idx"].long())[keep].reshape(-1)
    counts = torch.zeros(G * E, dtype=torch.int32, device="cuda")
    counts.index_add_(0, flat, torch.ones_like(flat, dtype=torch.int32))
    n = torch.zeros(G, dtype=torch.int32, device="cuda")
    n.index_add_(0, seq[keep], torch.ones_like(seq[keep], dtype=torch.int32))
    return counts.view(G, E), n


def _softmax(logits):
    l = logits.float()
    m = l.max(1, keepdim=True).values
    e = torch.exp(l - m)
    z = e.sum(1, keepdim=True)
    return e / z, (m + torch.log(z))[:, 0]


def _plain_norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1)
    xc = x - mean[:, None]
    rstd = torch.rsqrt(xc.square().mean(1) + _EPS)
    y = xc * rstd[:, None] * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return dict(y=y.to(s["x"].dtype), mean=mean, rstd=rstd)


def _plain_norm_bwd(s):
    dy = s["dy"].float()
    xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["weight"].float()
    dx = (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["dx_add"] is not None:
        dx = dx + s["dx_add"].float()
    out = dict(dx=dx.to(s["x"].dtype), dweight=(dy * xh).sum(0).to(s["weight"].dtype))
    if s["bias"] is not None:
        out["dbias"] = dy.sum(0).to(s["bias"].dtype)
    return out


def _plain_balance_fwd(s):
    case = s["case"]
    E, k, G = case["E"], case["k"], case["G"]
    seq, keep = _token_groups(s)
    counts, n = _counts(s)
    p, lse = _softmax(s["logits"])
    P = torch.zeros(G, E, device="cuda").index_add_(0, seq[keep], p[keep])
    nf = n.float().clamp(min=1.0)
    per_seq = (counts.float() * P).sum(1) * (E / k) / (nf * nf)
    balance = per_seq.sum() / (n > 0).sum().clamp(min=1)
    lse = torch.where(keep, lse, torch.zeros_like(lse))
    z = lse.square().sum() / n.sum().clamp(min=1)
    return dict(losses=torch.stack([balance, z]), seq_loss=per_seq, counts=counts, tokens=n,
                lse=lse)


def _plain_balance_bwd(s):
    case = s["case"]
    seq, keep = _token_groups(s)
    p, lse = _softmax(s["logits"])
    nf = s["n"].float().clamp(min=1.0)
    live = (s["n"] > 0).sum().clamp(min=1)
    c = s["counts"].float() * ((case["E"] / case["k"]) / (nf * nf * live))[:, None]
    c = (c * s["dlosses"][0])[seq]
    d = p * (c - (p * c).sum(1, keepdim=True))
    d = d + p * (s["dlosses"][1] * 2.0 / s["n"].sum().clamp(min=1) * lse)[:, None]
    return dict(dlogits=torch.where(keep[:, None], d, torch.zeros_like(d))
                .to(s["logits"].dtype))


def _plain_clip(s):
    total = torch.zeros((), device="cuda")
    for g in s["grads"]:
        f = g.float()
        total = total + (f * f).sum()
    norm = torch.sqrt(total)
    coef = (s["max_norm"] / (norm + _CLIP_EPS)).clamp(max=1.0)
    dst = s["grads"] if s["out"] is None else s["out"]
    return dict(norm=norm, grads=[(g.float() * coef).to(d.dtype)
                                  for g, d in zip(s["grads"], dst)])


# ------------------------------------------------------------------------ one pass
def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd,
                "balance_fwd": _plain_balance_fwd, "balance_bwd": _plain_balance_bwd,
                "clip": _plain_clip}[op](s)
    if op == "norm_fwd":
        y = s["norm"].forward(s["x"], s["weight"], s["bias"])
        return dict(y=y, mean=s["norm"].mean, rstd=s["norm"].rstd)
    if op == "norm_bwd":
        dx, dweight, dbias = s["norm"].backward(s["dy"], s["x"], s["weight"],
                                                dx_add=s["dx_add"])
        out = dict(dx=dx, dweight=dweight)
        if dbias is not None:
            out["dbias"] = dbias
        return out
    if op == "balance_fwd":
        losses, counts = s["loss"].forward(s["logits"], s["topk_idx"], s["seq_offsets"],
                                           s["mask"])
        return dict(losses=losses, seq_loss=s["loss"].seq_loss, counts=counts,
                    tokens=s["loss"].tokens, lse=s["loss"].lse)
    if op == "balance_bwd":
        return dict(dlogits=s["loss"].backward(s["logits"], s["dlosses"], s["seq_offsets"],
                                               s["mask"]))
    norm = s["clip"].clip(s["grads"], s["max_norm"], out=s["out"])
    return dict(norm=norm, grads=s["grads"] if s["out"] is None else s["out"])


# --------------------------------------------------------------- least work, exact
def work(case):
    op = case["op"]
    if op.startswith("norm"):
        T, H = case["T"], case["H"]
        a, p = _BYTES[case["dtype"]], _BYTES[case["param"]]
        params = 2 if case["bias"] else 1
        if op == "norm_fwd":
            return dict(bytes=2 * T * H * a + params * H * p + 8 * T, flops=8 * T * H)
        moved = (3 + (1 if case["add"] else 0)) * T * H * a
        return dict(bytes=moved + (1 + params) * H * p + 8 * T, flops=14 * T * H)
    if op.startswith("balance"):
        T, E, G = case["T"], case["E"], case["G"]
        side = (T if case["mask"] else 0) + (4 * (G + 1) if G > 1 else 0) + 4 * G * (E + 1)
        b = _BYTES[case["dtype"]]
        if op == "balance_fwd":
            return dict(bytes=T * E * b + 4 * T * (case["k"] + 1) + side + 4 * G + 8,
                        flops=6 * T * E)
        return dict(bytes=2 * T * E * b + side + 8, flops=10 * T * E)
    total = 0
    elements = 0
    for n, name in _clip_sizes(case):
        elements += n
        total += n * _BYTES[name]
        if case["out"] != "inplace":     # under the bound, in place: nothing to write
            total += n * (4 if case["out"] == "fp32" else _BYTES[name])
    return dict(bytes=total + 4, flops=(2 if case["out"] == "inplace" else 3) * elements)


def _exact_balance(case, s):
    """Per sequence, from the definition, in fp64."""
    E, k, G, T = case["E"], case["k"], case["G"], case["T"]
    off = [0, T] if s["seq_offsets"] is None else s["seq_offsets"].tolist()
    L = s["logits"].double()
    lse = torch.logsumexp(L, 1)
    prob = torch.softmax(L, 1)
    on = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"].bool()
    rows = [torch.nonzero(on[off[g]:off[g + 1]])[:, 0] + off[g] for g in range(G)]
    live = sum(1 for r in rows if len(r))
    n_all = sum(len(r) for r in rows)
    counts = torch.zeros(G, E, dtype=torch.int32, device="cuda")
    per_seq = torch.zeros(G, dtype=torch.float64, device="cuda")
    zsum = torch.zeros((), dtype=torch.float64, device="cuda")
    grad = torch.zeros(T, E, dtype=torch.float64, device="cuda")
    dl = torch.tensor([1e-2, 1e-3]).double().tolist()   # the values the fp32 coefficients hold
    for g, r in enumerate(rows):
        if len(r) == 0:
            continue
        cnt = torch.bincount(s["topk_idx"][r].reshape(-1).long(), minlength=E)
        counts[g] = cnt.to(torch.int32)
        f = cnt.double() * E / (k * len(r))
        pr = prob[r]
        per_seq[g] = (f * pr.mean(0)).sum()
        zsum = zsum + (lse[r] ** 2).sum() / n_all
        fb = f / (len(r) * live) * dl[0]
        grad[r] = pr * (fb - (pr @ fb)[:, None] + (2.0 * dl[1] / n_all) * lse[r][:, None])
    if case["op"] == "balance_fwd":
        keep = torch.zeros(T, dtype=torch.bool, device="cuda")
        keep[torch.cat(rows)] = True
        return dict(losses=torch.stack([per_seq.sum() / max(live, 1), zsum]), seq_loss=per_seq,
                    counts=counts,
                    tokens=torch.tensor([len(r) for r in rows], dtype=torch.int32, device="cuda"),
                    lse=torch.where(keep, lse, torch.zeros_like(lse)))
    return dict(dlogits=grad)


def exact(case, seed):
    s = dict(_inputs(case, seed), case=case)
    op = case["op"]
    if op.startswith("balance"):
        return _exact_balance(case, s)
    if op == "clip":
        norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(g, dtype=torch.float64)) ** 2
                                   for g in s["grads"]))
        coef = min(1.0, s["max_norm"] / (norm + _CLIP_EPS))
        return dict(norm=torch.tensor(norm, dtype=torch.float64),
                    grads=[g.double().mul_(coef) for g in s["grads"]])
    x, w = s["x"].double(), s["weight"].double()
    var, mean = torch.var_mean(x, 1, correction=0)
    rstd = (var + _EPS) ** -0.5
    xh = (x - mean[:, None]).mul_(rstd[:, None])
    if op == "norm_fwd":
        y = xh * w if s["bias"] is None else torch.addcmul(s["bias"].double(), xh, w)
        return dict(y=y, mean=mean, rstd=rstd)
    dy = s["dy"].double()
    # dx = J^T (w dy) with J = rstd (I - 1/H - xh xh^T / H)
    v = dy * w
    H = case["H"]
    dx = (v - v.sum(1, keepdim=True) / H
          - xh * (torch.einsum("th,th->t", v, xh) / H)[:, None]) * rstd[:, None]
    if s["dx_add"] is not None:
        dx += s["dx_add"].double()
    out = dict(dx=dx, dweight=torch.einsum("th,th->h", dy, xh))
    if s["bias"] is not None:
        out["dbias"] = dy.sum(0)
    return out
