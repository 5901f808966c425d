"""Timed cases of the further operators of a training step around the expert layer: the
selection of experts from the router's logits (scores, balance bias, groups, weights; and its
backward), the RMS norms before and after a block fused with its gate and residual scale
(forward, backward), and the AdamW step over many tensors with states in 32 or in 8 bits.

`listed()` gives the cases, `draw()` more of the same ranges, `prepare()` a case's
inputs, `run()` one pass through its operator (the library's when `own` is set, else a
plain form in elementary torch operations), `work()` the bytes and operations the pass cannot
do without, and `exact()` the same outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

_TORCH = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_RMS_EPS = 1e-6
_SUM_EPS = 1e-20     # added to the chosen scores' sum before the division
_CLIP_EPS = 1e-6     # added to the gradient norm before the division
_BETAS, _ADAM_EPS, _LR = (0.9, 0.99), 1e-8, 3e-4
_STEPS = 100         # steps that lie behind an AdamW case's states
_SEED = 7            # of the 8-bit states' rounding
_M32 = 0xffffffff


# --------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of the benchmark layer's router in decoding: softmax over all experts, top 8
        dict(name="select_fwd_token", op="select_fwd", T=1, E=128, k=8, score="softmax", groups=1,
             topk_groups=1, group_score="max", bias=False, renormalise=True, scale=1.0,
             dtype="fp32"),
        # a long packed batch: 256 experts, sigmoid scores with a balance bias, four of eight groups
        dict(name="select_fwd_groups", op="select_fwd", T=131072, E=256, k=8, score="sigmoid",
             groups=8, topk_groups=4, group_score="top2", bias=True, renormalise=True, scale=2.5,
             dtype="fp32"),
        # groups of 20 experts, an odd number of tokens, logits in bf16, weights as the softmax is
        dict(name="select_fwd_odd", op="select_fwd", T=5003, E=160, k=6, score="softmax", groups=8,
             topk_groups=3, group_score="max", bias=False, renormalise=False, scale=16.0,
             dtype="bf16"),
        # the benchmark layer's router gradient where the weights stay unnormalised: a dense one
        dict(name="select_bwd_layer", op="select_bwd", T=16384, E=128, k=8, score="softmax",
             groups=1, topk_groups=1, group_score="max", bias=False, renormalise=False, scale=1.0,
             dtype="fp32"),
        # the packed batch's router gradient: zero but for the chosen experts
        dict(name="select_bwd_groups", op="select_bwd", T=131072, E=256, k=8, score="sigmoid",
             groups=8, topk_groups=4, group_score="top2", bias=True, renormalise=True, scale=2.5,
             dtype="fp32"),
        # one token between two blocks in decoding
        dict(name="resnorm_fwd_token", op="resnorm_fwd", T=1, H=2048, dtype="bf16", res="bf16",
             param="bf16", post=True, gate="channel", pre=True, scale=1.0),
        # between two blocks of the benchmark layer's width, a training step's micro-batch
        dict(name="resnorm_fwd_layer", op="resnorm_fwd", T=16384, H=2048, dtype="bf16", res="bf16",
             param="bf16", post=True, gate="channel", pre=True, scale=0.5),
        # its backward
        dict(name="resnorm_bwd_layer", op="resnorm_bwd", T=16384, H=2048, dtype="bf16", res="bf16",
             param="bf16", post=True, gate="channel", pre=True, scale=0.5),
        # the wide layer's width: a residual stream and parameters in fp32, a gate for each token
        dict(name="resnorm_bwd_wide", op="resnorm_bwd", T=8191, H=4096, dtype="fp16", res="fp32",
             param="fp32", post=True, gate="token", pre=True, scale=1.0),
        # the tiny layer's parameters, fp32 states
        dict(name="adamw_tiny", op="adamw", sizes=0, n=6, total=0, dtype="bf16", grad="bf16",
             master=True, states="fp32", clip=True),
        # the benchmark layer's parameters: bf16 with fp32 masters and fp32 states, clipped
        dict(name="adamw_layer", op="adamw", sizes=1, n=6, total=0, dtype="bf16", grad="bf16",
             master=True, states="fp32", clip=True),
        # many tensors of odd sizes with states in 8 bits
        dict(name="adamw_many8", op="adamw", sizes=7, n=48, total=200_000_000, dtype="bf16",
             grad="bf16", master=True, states="8bit", clip=True),
    ]


def _log_int(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["select_fwd", "select_bwd", "resnorm_fwd", "resnorm_bwd", "adamw"])
    if op.startswith("select"):
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log_int(rng, 4, 512 // groups)
        topk_groups = rng.randint(1, groups)
        most = E // groups * topk_groups
        return dict(op=op, T=_log_int(rng, 1, 131072 if E <= 256 else 65536), E=E,
                    k=min(most, rng.choice([1, 2, 4, 6, 8])),
                    score=rng.choice(["softmax", "sigmoid"]), groups=groups,
                    topk_groups=topk_groups, group_score=rng.choice(["max", "top2"]),
                    bias=rng.random() < 0.5, renormalise=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["fp32", "fp32", "bf16"]))
    if op.startswith("resnorm"):
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        res = rng.choice([dtype, "fp32"])
        H = _log_int(rng, 64, 8192)
        if rng.random() < 0.7:           # most widths are multiples of 64, the rest any
            H = max(64, H // 64 * 64)
        return dict(op=op, T=_log_int(rng, 1, min(32768, 33_554_432 // H)), H=H, dtype=dtype,
                    res=res, param=rng.choice([dtype, "fp32"]), post=rng.random() < 0.7,
                    gate=rng.choice(["none", "channel", "token"]), pre=rng.random() < 0.7,
                    scale=rng.choice([1.0, 0.5]))
    n = _log_int(rng, 1, 60)
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    return dict(op=op, sizes=rng.randrange(2, 1 << 30), n=n,
                total=_log_int(rng, 1000 + n, 200_000_000), dtype=dtype,
                grad=rng.choice([dtype, "fp32"]), master=dtype != "fp32" and rng.random() < 0.7,
                states=rng.choice(["fp32", "8bit"]), clip=rng.random() < 0.6)


def _sizes(case):
    """Elements of every tensor of an AdamW case."""
    if case["sizes"] in (0, 1):      # the tiny / the benchmark layer's parameters
        E, I, H = (8, 64, 128) if case["sizes"] == 0 else (128, 768, 2048)
        return [E * I * H, E * I * H, E * H * I, E * H, H, H]
    r = np.random.default_rng(case["sizes"])
    share = np.exp(r.normal(0.0, 1.5, case["n"]))
    return [int(v) for v in np.maximum(1, (share / share.sum() * case["total"]).astype(np.int64))]


def _places(sizes):
    """First element of each tensor in a flat buffer, and its length: whole blocks of 32."""
    first = np.concatenate([[0], np.cumsum([-(-n // 32) * 32 for n in sizes])])
    return [int(v) for v in first[:-1]], int(first[-1])


# -------------------------------------------------------------------------- inputs
def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _select_inputs(case, gen):
    T, E = case["T"], case["E"]
    # uneven experts: a popularity that falls off with the rank, over a random order
    rank = torch.randperm(E, generator=gen, device="cuda").float()
    s = dict(logits=(_randn(gen, T, E) - 0.5 * torch.log1p(rank)).to(_TORCH[case["dtype"]]),
             # what balancing has added to the rarer experts' keys by then
             bias=None)
    if case["bias"]:
        size = 1.0 if case["score"] == "sigmoid" else 4.0 / E
        s["bias"] = size * (0.02 * torch.log1p(rank) + 0.005 * _randn(gen, E))
    if case["op"] == "select_bwd":
        s["topk_idx"] = torch.topk(s["logits"].float(), case["k"], dim=1).indices \
            .to(torch.int32).contiguous()
        s["dtopk_w"] = _randn(gen, T, case["k"])
    return s


def _resnorm_inputs(case, gen):
    T, H = case["T"], case["H"]
    dt, rt, pt = _TORCH[case["dtype"]], _TORCH[case["res"]], _TORCH[case["param"]]
    # a residual stream: unit noise, a few channels far larger
    big = torch.ones(H, device="cuda")
    big[:: max(1, H // 8)] = 12.0
    s = dict(f=(0.7 * _randn(gen, T, H)).to(dt), x=(_randn(gen, T, H) * big).to(rt),
             post_weight=(1.0 + 0.1 * _randn(gen, H)).to(pt) if case["post"] else None,
             pre_weight=(1.0 + 0.1 * _randn(gen, H)).to(pt) if case["pre"] else None, gate=None)
    if case["gate"] == "channel":
        s["gate"] = (0.3 + 0.1 * _randn(gen, H)).to(pt)
    elif case["gate"] == "token":
        s["gate"] = torch.sigmoid(_randn(gen, T)).to(pt)
    if case["op"] == "resnorm_bwd":
        s["out"] = s.pop("x")            # the forward's output, as it is stored
        s["dout"] = _randn(gen, T, H).to(rt)
        s["dn"] = _randn(gen, T, H).to(dt) if case["pre"] else None
    return s


def _adamw_inputs(case, gen):
    sizes = _sizes(case)
    first, total = _places(sizes)
    live = torch.zeros(total, dtype=torch.bool, device="cuda")
    for a, n in zip(first, sizes):
        live[a:a + n] = True

    def flat(scale, positive=False):
        t = torch.empty(total, device="cuda")
        for a in range(0, total, 1 << 27):           # bounds the draw's memory
            b = min(total, a + (1 << 27))
            t[a:b] = scale * _randn(gen, b - a)
        return (t.square_() if positive else t).mul_(live)
    p = flat(0.02)
    s = dict(sizes=sizes, first=first, master=p if case["master"] else None,
             param=p.to(_TORCH[case["dtype"]]),
             grad=flat(1e-3).to(_TORCH[case["grad"]]),
             m=flat(3e-4), v=flat(1e-3, positive=True))
    # matrices decay, what is as short as a norm's weight does not
    s["decay"] = [0.1 if n >= 4096 else 0.0 for n in sizes]
    if case["clip"]:
        s["norm"] = s["grad"].float().square().sum().sqrt()
        s["max_norm"] = 0.3e-3 * math.sqrt(sum(sizes))
    else:
        s["norm"], s["max_norm"] = None, None
    return s


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * (seed % (1 << 31)) + 29)
    if case["op"].startswith("select"):
        return _select_inputs(case, gen)
    if case["op"].startswith("resnorm"):
        return _resnorm_inputs(case, gen)
    return _adamw_inputs(case, gen)


def prepare(case, seed):
    s = dict(_inputs(case, seed), case=case)
    op = case["op"]
    if op == "resnorm_bwd":                          # what the forward kept
        s["rstd_f"] = torch.rsqrt(s["f"].float().square().mean(1) + _RMS_EPS)
        s["rstd_out"] = torch.rsqrt(s["out"].float().square().mean(1) + _RMS_EPS)
    if op == "adamw":
        s["steps"] = _STEPS
        if case["states"] == "8bit":
            for n, kind in (("m", _M8), ("v", _V8)):
                s[n], s[n + "_scale"] = _encode(s[n], kind, None)
    if own:
        import mixture_experts_layer_16_gb300 as M
        if op.startswith("select"):
            s["select"] = M.MoESelect(case["T"], case["E"], case["k"], case["score"],
                                      case["groups"], case["topk_groups"], case["group_score"],
                                      case["renormalise"], case["scale"], case["dtype"])
        elif op.startswith("resnorm"):
            s["norm"] = M.MoEResidualNorm(
                case["T"], case["H"], case["dtype"], case["res"], case["param"],
                post=case["post"], gate=None if case["gate"] == "none" else case["gate"],
                pre=case["pre"], scale=case["scale"], eps=_RMS_EPS)
            if op == "resnorm_bwd":
                s["norm"].load_stats(s["rstd_f"] if case["post"] else None,
                                     s["rstd_out"] if case["pre"] else None)
        else:
            s["params"], s["grads"], s["masters"] = (
                None if s[n] is None else
                [s[n][a:a + k] for a, k in zip(s["first"], s["sizes"])]
                for n in ("param", "grad", "master"))
            s["opt"] = M.MoEAdamW(s["params"], betas=_BETAS, eps=_ADAM_EPS,
                                  weight_decay=s["decay"], states=case["states"], seed=_SEED)
            s["opt"].m.copy_(s["m"])
            s["opt"].v.copy_(s["v"])
            if case["states"] == "8bit":
                s["opt"].m_scale.copy_(s["m_scale"])
                s["opt"].v_scale.copy_(s["v_scale"])
            s["opt"].set_step(_STEPS)
    return s


# ---------------------------------------------------------------- states in 8 bits
# Blocks of 32 elements share a power of two 2^(c - 127), the smallest under which the block's
# largest value fits the codes: sign, 4 exponent and 3 fraction bits up to 448 for the first moment
# (e4m3), 5 exponent and 3 fraction bits up to 1.875 * 2^16 for the second, which has no sign.
# (bits, exponent bias, largest value's fraction bits in fp32, fp32 exponent less c, signed)
_M8 = dict(bits=7, bias=7, top=0x600000, shift=8, signed=True)
_V8 = dict(bits=8, bias=15, top=0x700000, shift=16, signed=False)


def _pow2(e):
    """2^e in fp32, -149 <= e <= 127."""
    return torch.where(e < -126, torch.ldexp(torch.ones_like(e, dtype=torch.float32),
                                             e.clamp(min=-149).to(torch.int32)),
                       ((e.clamp(min=-126) + 127).to(torch.int32) << 23).view(torch.float32))


def _encode(t, kind, rand16):
    """Codes and scales (uint8) of a flat fp32 tensor; rand16: the random bits that a value's
    fraction between two codes is compared with (None: to nearest)."""
    b = t.view(-1, 32)
    amax = b.abs().amax(1).view(torch.int32)
    c = (((amax + (0x7fffff - kind["top"])) >> 23) - kind["shift"]).clamp(min=0)
    # in two exact steps: under the block's scale, then to where fp32's exponents are the codes'
    z = b.abs() * _pow2(127 - c)[:, None] * 2.0 ** (kind["bias"] - 127)
    bits = z.view(torch.int32)
    if rand16 is None:
        bits = bits + 0x7ffff + ((bits >> 20) & 1)
    else:
        bits = bits + (rand16.view(-1, 32) << 4)
    code = bits >> 20
    if kind["signed"]:
        code = code | ((b.view(torch.int32) >> 24) & 0x80)
    else:                                            # what is not zero stays above zero
        code = torch.where((code == 0) & (b > 0), torch.ones_like(code), code)
    return code.to(torch.uint8).view(-1), c.to(torch.uint8)


def _decode(codes, scales, kind):
    c = codes.to(torch.int32).view(-1, 32)
    mag = c & 0x7f if kind["signed"] else c
    x = (mag << 20).view(torch.float32) * 2.0 ** (127 - kind["bias"]) \
        * _pow2(scales.to(torch.int32) - 127)[:, None]
    if kind["signed"]:
        x = torch.where(c >= 128, -x, x)
    return x.view(-1)


def _mix(x):
    """A 32-bit hash (64-bit integers that hold 32)."""
    x = x ^ (x >> 16)
    x = x * 0x9E3779B1 & _M32
    x = x ^ (x >> 15)
    x = x * 0x6A09E667 & _M32
    return x ^ (x >> 16)


def _random(step, tensor, n):
    """Each element's 16 random bits for the first and for the second moment."""
    key = _mix(_mix((_SEED + 0x9E3779B1 * step) & _M32) ^ tensor)
    h = _mix(torch.arange(n, device="cuda", dtype=torch.int64) ^ key)
    return (h & 0xffff).to(torch.int32), (h >> 16).to(torch.int32)


# --------------------------------------------------------------------- plain forms
def _scores(logits, score):
    """The scores in 64 bits (keys lie next to one another)."""
    l = logits.double()
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.max(1, keepdim=True).values)
    return e / e.sum(1, keepdim=True)


def _best(keys, k):
    """The k largest of each row, descending, ties to the lowest index."""
    return torch.sort(keys, dim=1, descending=True, stable=True).indices[:, :k]


def _plain_select_fwd(s):
    case = s["case"]
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    p = _scores(s["logits"], case["score"])
    key = p if s["bias"] is None else p + s["bias"].double()
    if case["topk_groups"] < G:
        kg = key.view(T, G, E // G)
        two = torch.sort(kg, dim=2, descending=True).values[:, :, :2]
        gs = two.sum(2) if case["group_score"] == "top2" else two[:, :, 0]
        keep = torch.zeros(T, G, dtype=torch.bool, device="cuda")
        keep.scatter_(1, _best(gs, case["topk_groups"]), True)
        key = torch.where(keep[:, :, None], kg, torch.full_like(kg, -math.inf)).view(T, E)
    idx = _best(key, k)
    w = p.gather(1, idx)
    if case["renormalise"]:
        w = w / (w.sum(1, keepdim=True) + _SUM_EPS)
    return dict(topk_idx=idx.to(torch.int32), topk_w=(w * case["scale"]).float())


def _plain_select_bwd(s):
    case = s["case"]
    idx, g = s["topk_idx"].long(), s["dtopk_w"]
    l = s["logits"].float()
    if case["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-l))
    else:
        e = torch.exp(l - l.max(1, keepdim=True).values)
        p = e / e.sum(1, keepdim=True)
    sc = p.gather(1, idx)
    ds = g * case["scale"]
    if case["renormalise"]:
        N = sc.sum(1, keepdim=True) + _SUM_EPS
        ds = (ds - (ds * sc).sum(1, keepdim=True) / N) / N
    if case["score"] == "sigmoid":
        d = torch.zeros_like(l).scatter_add_(1, idx, ds * sc * (1.0 - sc))
    else:
        d = torch.zeros_like(l).scatter_add_(1, idx, ds)
        d = p * (d - (ds * sc).sum(1, keepdim=True))
    return dict(dlogits=d.to(s["logits"].dtype))


def _gate(s):
    if s["gate"] is None:
        return 1.0
    return s["gate"].float() if s["case"]["gate"] == "channel" else s["gate"].float()[:, None]


def _plain_resnorm_fwd(s):
    case = s["case"]
    u = s["f"].float()
    r = {}
    if case["post"]:
        r["rstd_f"] = torch.rsqrt(u.square().mean(1) + _RMS_EPS)
        u = u * r["rstd_f"][:, None] * s["post_weight"].float()
    out = s["x"].float() + u * _gate(s) * case["scale"]
    r["out"] = out.to(s["x"].dtype)
    if case["pre"]:
        r["rstd_out"] = torch.rsqrt(out.square().mean(1) + _RMS_EPS)
        r["n"] = (out * r["rstd_out"][:, None] * s["pre_weight"].float()).to(s["f"].dtype)
    return r


def _plain_resnorm_bwd(s):
    case = s["case"]
    D = s["dout"].float()
    f = s["f"].float()
    r = {}
    if case["pre"]:
        oh = s["out"].float() * s["rstd_out"][:, None]
        dn = s["dn"].float()
        g = dn * s["pre_weight"].float()
        D = D + (g - oh * (g * oh).mean(1, keepdim=True)) * s["rstd_out"][:, None]
        r["dpre_weight"] = (dn * oh).sum(0).to(s["pre_weight"].dtype)
    r["dx"] = D.to(s["out"].dtype)
    du = D * _gate(s) * case["scale"]
    u = f
    if case["post"]:
        fh = f * s["rstd_f"][:, None]
        u = fh * s["post_weight"].float()
        r["dpost_weight"] = (du * fh).sum(0).to(s["post_weight"].dtype)
        q = du * s["post_weight"].float()
        df = (q - fh * (q * fh).mean(1, keepdim=True)) * s["rstd_f"][:, None]
    else:
        df = du
    r["df"] = df.to(s["f"].dtype)
    if s["gate"] is not None:
        dim = 0 if case["gate"] == "channel" else 1
        r["dgate"] = ((u * D).sum(dim) * case["scale"]).to(s["gate"].dtype)
    return r


def _plain_adamw(s):
    case = s["case"]
    s["steps"] += 1
    t = s["steps"]
    b1, b2 = _BETAS
    c1, c2 = 1.0 / (1.0 - b1 ** t), 1.0 / math.sqrt(1.0 - b2 ** t)
    coef = 1.0
    if s["norm"] is not None:
        coef = (s["max_norm"] / (s["norm"] + _CLIP_EPS)).clamp(max=1.0)
    wide = s["param"] if s["master"] is None else s["master"]
    for i, (a, n) in enumerate(zip(s["first"], s["sizes"])):
        z = a + -(-n // 32) * 32                     # the states' blocks are whole
        g = s["grad"][a:z].float() * coef
        if case["states"] == "8bit":
            q = slice(a // 32, z // 32)
            m, v = (_decode(s[x][a:z], s[x + "_scale"][q], kind)
                    for x, kind in (("m", _M8), ("v", _V8)))
        else:
            m, v = s["m"][a:z], s["v"][a:z]
        m = m * b1 + g * (1.0 - b1)
        v = v * b2 + g * g * (1.0 - b2)
        p = wide[a:z].float()
        p = p * (1.0 - _LR * s["decay"][i]) - _LR * (m * c1) / (torch.sqrt(v) * c2 + _ADAM_EPS)
        wide[a:z] = p.to(wide.dtype)
        if s["master"] is not None:
            s["param"][a:z] = p.to(s["param"].dtype)
        if case["states"] == "8bit":
            for x, new, kind, bits in zip(("m", "v"), (m, v), (_M8, _V8), _random(t, i, z - a)):
                s[x][a:z], s[x + "_scale"][q] = _encode(new, kind, bits)
        else:
            s["m"][a:z], s["v"][a:z] = m, v
    r = dict(param=s["param"])
    if s["master"] is not None:
        r["master"] = s["master"]
    if case["states"] == "8bit":                     # the values that the codes stand for
        r["m"] = _decode(s["m"], s["m_scale"], _M8).to(torch.bfloat16)
        r["v"] = _decode(s["v"], s["v_scale"], _V8).to(torch.bfloat16)
    else:
        r["m"], r["v"] = s["m"], s["v"]
    return r


# ------------------------------------------------------------------------ one pass
def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"select_fwd": _plain_select_fwd, "select_bwd": _plain_select_bwd,
                "resnorm_fwd": _plain_resnorm_fwd, "resnorm_bwd": _plain_resnorm_bwd,
                "adamw": _plain_adamw}[op](s)
    if op == "select_fwd":
        idx, w = s["select"].forward(s["logits"], s["bias"])
        return dict(topk_idx=idx, topk_w=w)
    if op == "select_bwd":
        return dict(dlogits=s["select"].backward(s["logits"], s["topk_idx"], s["dtopk_w"]))
    if op == "resnorm_fwd":
        out, n = s["norm"].forward(s["x"], s["f"], post_weight=s["post_weight"], gate=s["gate"],
                                   pre_weight=s["pre_weight"])
        r = dict(out=out)
        if s["post_weight"] is not None:
            r["rstd_f"] = s["norm"].rstd_f
        if n is not None:
            r["n"], r["rstd_out"] = n, s["norm"].rstd_out
        return r
    if op == "resnorm_bwd":
        dx, df, grads = s["norm"].backward(s["dout"], s["dn"], s["out"], s["f"],
                                           post_weight=s["post_weight"], gate=s["gate"],
                                           pre_weight=s["pre_weight"])
        return dict(dx=dx, df=df, **{"d" + k: v for k, v in grads.items()})
    s["opt"].step(s["params"], s["grads"], _LR, masters=s["masters"], norm=s["norm"],
                  max_norm=s["max_norm"])
    r = dict(param=s["param"])
    if s["master"] is not None:
        r["master"] = s["master"]
    r["m"], r["v"] = s["opt"].moments()
    return r


# --------------------------------------------------------------- least work, exact
def work(case):
    op = case["op"]
    if op.startswith("select"):
        T, E, k = case["T"], case["E"], case["k"]
        b = _BYTES[case["dtype"]]
        if op == "select_fwd":
            return dict(bytes=T * E * b + 8 * T * k + (4 * E if case["bias"] else 0),
                        flops=8 * T * E)
        # (the weights' gradient stays with the chosen logits but for a softmax left as it is)
        dense = case["score"] == "softmax" and not case["renormalise"]
        return dict(bytes=T * E * b + (T * E * b if dense else T * k * b) + 8 * T * k,
                    flops=(8 * T * E if dense else 12 * T * k))
    if op.startswith("resnorm"):
        T, H = case["T"], case["H"]
        a, r, p = _BYTES[case["dtype"]], _BYTES[case["res"]], _BYTES[case["param"]]
        vec = H * p * (case["post"] + case["pre"]) \
            + (H * p if case["gate"] == "channel" else T * p if case["gate"] == "token" else 0)
        stats = 4 * T * (case["post"] + case["pre"])
        if op == "resnorm_fwd":
            return dict(bytes=T * H * (a + 2 * r + (a if case["pre"] else 0)) + vec + stats,
                        flops=(2 + 4 * case["post"] + 4 * case["pre"]) * T * H)
        # dout, f in, dx, df out; dn and out where there is a norm behind
        need_f = case["post"] or case["gate"] != "none"
        moved = 2 * r + a + (a if need_f else 0) + (a + r if case["pre"] else 0)
        return dict(bytes=T * H * moved + 2 * vec + stats,
                    flops=(3 + 10 * case["post"] + 10 * case["pre"]) * T * H)
    n = sum(_sizes(case))
    p, g = _BYTES[case["dtype"]], _BYTES[case["grad"]]
    state = 16 if case["states"] == "fp32" else 4 + 4 / 32
    weights = 8 + p if case["master"] else 2 * p
    return dict(bytes=n * (g + state + weights), flops=16 * n)


def _exact_select(case, s):
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    l = s["logits"].double()
    p = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    rows = torch.arange(T, device="cuda")
    place = torch.arange(E, device="cuda")
    if case["op"] == "select_fwd":
        key = p.clone() if s["bias"] is None else p + s["bias"].double()

        def take(v, n):
            """One after the other: the lowest index of the largest value left."""
            v, at, found = v.clone(), torch.arange(v.shape[1], device="cuda"), []
            for _ in range(n):
                i = torch.where(v == v.amax(1, keepdim=True), at, v.shape[1]).amin(1)
                found.append(i)
                v[rows, i] = -math.inf
            return torch.stack(found, 1)
        if case["topk_groups"] < G:
            kg = key.view(T, G, E // G)
            score = kg.amax(2)
            if case["group_score"] == "top2" and E > G:
                score = torch.kthvalue(kg, E // G - 1, dim=2).values + score
            chosen = take(score, case["topk_groups"])
            keep = (chosen[:, :, None] == (place // (E // G))[None, None, :]).any(1)
            key[~keep] = -math.inf
        idx = take(key, k)
        w = torch.stack([p[rows, i] for i in idx.unbind(1)], 1)
        if case["renormalise"]:
            w = w / (w.sum(1, keepdim=True) + _SUM_EPS)
        return dict(topk_idx=idx.to(torch.int32), topk_w=case["scale"] * w)
    # w_j = c s_j / N: by the chain rule, one chosen expert after the other
    cols = s["topk_idx"].long().unbind(1)
    sc = torch.stack([p[rows, i] for i in cols], 1)
    g = s["dtopk_w"].double() * case["scale"]
    if case["renormalise"]:
        N = sc.sum(1) + _SUM_EPS
        back = torch.stack([(g[:, j] * N - torch.einsum("tk,tk->t", g, sc)) / N ** 2
                            for j in range(k)], 1)
    else:
        back = g
    if case["score"] == "sigmoid":
        d = torch.zeros(T, E, dtype=torch.float64, device="cuda")
        for j, i in enumerate(cols):
            d[rows, i] += back[:, j] * sc[:, j] * torch.sigmoid(-l[rows, i])
        return dict(dlogits=d)
    d = p * -torch.einsum("tk,tk->t", back, sc)[:, None]
    for j, i in enumerate(cols):
        d[rows, i] += back[:, j] * sc[:, j]
    return dict(dlogits=d)


def _exact_resnorm(case, s):
    one = torch.ones((), dtype=torch.float64, device="cuda")
    alpha = case["scale"]
    gate = one if s["gate"] is None else s["gate"].double()
    if case["gate"] == "token":
        gate = gate[:, None]
    f = s["f"].double()
    H = case["H"]
    if case["op"] == "resnorm_fwd":
        r = {}
        coef = alpha * gate
        if case["post"]:
            r["rstd_f"] = (torch.einsum("th,th->t", f, f) / H + _RMS_EPS) ** -0.5
            coef = coef * s["post_weight"].double() * r["rstd_f"][:, None]
        r["out"] = torch.addcmul(s["x"].double(), f, coef)
        if case["pre"]:
            r["rstd_out"] = (torch.einsum("th,th->t", r["out"], r["out"]) / H + _RMS_EPS) ** -0.5
            r["n"] = torch.einsum("th,t,h->th", r["out"], r["rstd_out"], s["pre_weight"].double())
        return r
    # y = w x rho with rho = rstd(x) kept as given: dx = rho (w dy - xh <xh, w dy> / H)
    r = {}
    D = s["dout"].double()
    if case["pre"]:
        rho = s["rstd_out"].double()
        o = s["out"].double()
        wd = s["dn"].double() * s["pre_weight"].double()
        D = D + torch.einsum("t,th->th", rho, wd) \
            - torch.einsum("t,th,t->th", rho ** 3 / H, o, torch.einsum("th,th->t", o, wd))
        r["dpre_weight"] = torch.einsum("th,th,t->h", s["dn"].double(), o, rho)
    r["dx"] = D
    w = s["post_weight"].double() if case["post"] else one
    rho = s["rstd_f"].double() if case["post"] else one.expand(f.shape[0])
    if case["gate"] == "token":
        r["dgate"] = alpha * torch.einsum("th,th,t->t", f * w, D, rho)
    elif case["gate"] == "channel":
        r["dgate"] = alpha * w * torch.einsum("th,th,t->h", f, D, rho)
    du = alpha * gate * D
    if case["post"]:
        r["dpost_weight"] = torch.einsum("th,th,t->h", f, du, rho)
        wd = du * w
        r["df"] = torch.einsum("t,th->th", rho, wd) \
            - torch.einsum("t,th,t->th", rho ** 3 / H, f, torch.einsum("th,th->t", f, wd))
    else:
        r["df"] = du
    return r


def _held(values, kind, rand16):
    """What a state's codes stand for after the rounding, in 64 bits: each value lies between two
    neighbours of its block's grid, and goes to the upper one where its fraction and the
    random number add up to one."""
    b = values.view(-1, 32)
    a = b.abs()
    largest = (1.75 if kind["signed"] else 1.875) * 2.0 ** (kind["shift"])
    amax = a.amax(1)
    e = torch.ceil(torch.log2(amax / largest)).clamp(min=-127.0)
    e = torch.where(torch.ldexp(torch.full_like(e, largest), e) < amax, e + 1, e)
    lower = torch.ldexp(torch.full_like(e, largest), e - 1) >= amax
    e = torch.where(lower & (e > -127), e - 1, e)
    scale = torch.ldexp(torch.ones_like(e), e)[:, None]
    y = a / scale
    low = 1 - kind["bias"]                           # exponent of the smallest normal code
    ex = torch.floor(torch.log2(y.clamp(min=2.0 ** low))).clamp(min=low)
    ex = torch.where(torch.ldexp(torch.ones_like(y), ex) > y.clamp(min=2.0 ** low), ex - 1, ex)
    step = torch.ldexp(torch.ones_like(y), ex - 3)
    q = torch.floor(y / step + rand16.view(-1, 32).double() / 65536.0) * step
    if not kind["signed"]:
        q = torch.where((q == 0) & (a > 0), torch.full_like(q, 2.0 ** (low - 3)), q)
    return (torch.sign(b) * q * scale).view(-1)


def _exact_adamw(case, s):
    b1, b2 = _BETAS
    t = _STEPS + 1
    coef = 1.0
    if s["norm"] is not None:
        coef = min(1.0, s["max_norm"] / (float(s["norm"].double()) + _CLIP_EPS))
    wide = s["param"] if s["master"] is None else s["master"]
    got = {n: torch.zeros(wide.numel(), dtype=torch.float64, device="cuda")
           for n in ("param", "m", "v")}
    for i, (a, n) in enumerate(zip(s["first"], s["sizes"])):
        z = a + -(-n // 32) * 32
        g = s["grad"][a:z].double() * coef
        m, v = s["m"][a:z], s["v"][a:z]
        if case["states"] == "8bit":
            q = slice(a // 32, z // 32)
            m, v = _decode(m, s["m_scale"][q], _M8), _decode(v, s["v_scale"][q], _V8)
        m = torch.lerp(g, m.double(), b1)
        v = torch.lerp(g.square(), v.double(), b2)
        step = m / (1 - b1 ** t) / ((v / (1 - b2 ** t)).sqrt() + _ADAM_EPS)
        got["param"][a:z] = wide[a:z].double() - _LR * (step + s["decay"][i] * wide[a:z].double())
        if case["states"] == "8bit":
            rm, rv = _random(t, i, z - a)
            m, v = _held(m, _M8, rm), _held(v, _V8, rv)
        got["m"][a:z], got["v"][a:z] = m, v
    if s["master"] is not None:
        got["master"] = got["param"]
    return got


def exact(case, seed):
    s = dict(_inputs(case, seed), case=case)
    if case["op"].startswith("select"):
        return _exact_select(case, s)
    if case["op"].startswith("resnorm"):
        if case["op"] == "resnorm_bwd":              # the statistics that prepare() hands over
            s["rstd_f"] = torch.rsqrt(s["f"].float().square().mean(1) + _RMS_EPS)
            s["rstd_out"] = torch.rsqrt(s["out"].float().square().mean(1) + _RMS_EPS)
        return _exact_resnorm(case, s)
    if case["states"] == "8bit":
        for n, kind in (("m", _M8), ("v", _V8)):
            s[n], s[n + "_scale"] = _encode(s[n], kind, None)
    return _exact_adamw(case, s)
