"""Cases for the operators around an EP layer's dispatch and combine: the
residual norm that makes the 8-bit rows a dispatch sends, the router with its
balance loss, the experts' 8-bit products, and the sum of a receive row's
picks.  Each case has a plain form in elementary torch operations (32-bit
arithmetic, rounded once at the end) and a form that calls this package
(`own`); exact() gives the same outputs from the definitions in 64 bits.

8-bit rows are float8_e4m3fn values with one fp32 scale per 128 columns, kept
in one buffer per row (the values, then the scales, padded to 16 bytes) so
that a row travels through the dispatch as one piece.  8-bit expert weights
have one scale per block of 128 x 128."""
import math

import torch

own = False

BLOCK = 128
FP8_MAX = 448.0
FLOOR = 2.0 ** -100      # smallest block maximum a scale is made from
EPS = 1e-6
NEG = float("-inf")


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # serving: one rank's 128 tokens in the low-latency layer (hidden 7168), norm before the 8-bit dispatch
        dict(name="norm_decode", op="norm", tokens=128, hidden=7168, fp8=True, train=False),
        # serving a prompt: all 32 x 4096 tokens of the high-throughput layer
        dict(name="norm_prefill", op="norm", tokens=131072, hidden=7168, fp8=True, train=False),
        # training: a step's norm with its gradient at hidden 2048, a token count that divides by nothing
        dict(name="norm_train", op="norm", tokens=50021, hidden=2048, fp8=False, train=True),
        # serving: one rank's tokens through the router, top 8 of 256, no loss
        dict(name="route_decode", op="route", tokens=128, experts=256, topk=8, bf16=False, renorm=True, masked=False,
             train=False),
        # training the high-throughput layer: routing, balance loss and the logits' gradient
        dict(name="route_train", op="route", tokens=131072, experts=256, topk=8, bf16=False, renorm=True,
             masked=False, train=True),
        # training with padded tokens and experts switched off (rows left empty among them): bf16 logits, top 6 of 64
        dict(name="route_masked", op="route", tokens=65519, experts=64, topk=6, bf16=True, renorm=False,
             masked=True, train=True),
        # serving: one rank (8 experts) of the low-latency layer, about 128 rows an expert, gate and up products
        dict(name="up_decode", op="product", experts=8, picks=1024, width=7168, out=2048, gated=True),
        # serving a prompt: one rank of the high-throughput layer, about 4096 rows an expert
        dict(name="up_prefill", op="product", experts=8, picks=32768, width=7168, out=2048, gated=True),
        # serving single tokens: a handful of picks over 32 experts, some of them without any
        dict(name="down_decode", op="product", experts=32, picks=61, width=2048, out=7168, gated=False),
        # the prompt's second product, back to hidden 7168
        dict(name="down_prefill", op="product", experts=8, picks=32768, width=2048, out=7168, gated=False),
        # the picks of each receive row summed before the combine: the low-latency layer
        dict(name="sum_decode", op="sum", ranks=32, tokens_per_rank=128, hidden=7168, experts=256, topk=8, zipf=0.0),
        # the same with Zipf routing, hidden 2048, top 6 of 64 on 16 ranks
        dict(name="sum_skew", op="sum", ranks=16, tokens_per_rank=4096, hidden=2048, experts=64, topk=6, zipf=1.2),
    ]


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _sizes(case):
    """The drawn sizes, 3072 left out (3056 in its place)."""
    return {k: 3056 if type(v) is int and v == 3072 else v for k, v in case.items()}


def draw(rng):
    op = rng.choice(["norm", "route", "product", "sum"])
    if op == "norm":
        train = rng.random() < 0.4
        hidden = 8 * _between(rng, 8, 1024)
        most = 50021 * 2048 if train else 131072 * 7168
        case = dict(op=op, tokens=_between(rng, 1, min(131072, most // hidden)), hidden=hidden,
                    fp8=not train and rng.random() < 0.7, train=train)
    elif op == "route":
        experts = _between(rng, 2, 512)
        topk = rng.randint(1, min(8, experts))
        case = dict(op=op, tokens=_between(rng, 1, min(131072, 131072 * 256 // experts)), experts=experts, topk=topk,
                    bf16=rng.random() < 0.5, renorm=rng.random() < 0.5, masked=rng.random() < 0.5,
                    train=rng.random() < 0.6)
    elif op == "product":
        gated = rng.random() < 0.5
        width, out = 16 * _between(rng, 8, 448), 16 * _between(rng, 4, 256 if gated else 448)
        rows = 2 * out if gated else out
        experts = _between(rng, 1, min(64, max(1, 8 * 4096 * 7168 // (rows * width))))
        most = 8192 * 4096 * 7168 // (rows * width)
        case = dict(op=op, experts=experts, picks=_between(rng, 1, max(1, min(32768, most))), width=width, out=out,
                    gated=gated)
    else:
        ranks = rng.choice([1, 2, 4, 8, 16, 32])
        per = rng.choice([1, 2, 4, 8])
        experts = ranks * per
        topk = rng.randint(1, min(8, experts))
        hidden = 8 * _between(rng, 8, 1024)
        most = 65536 * 6 * 2048 // (topk * hidden)
        case = dict(op=op, ranks=ranks, tokens_per_rank=_between(rng, 1, max(1, min(4096, most // ranks))),
                    hidden=hidden, experts=experts, topk=topk, zipf=rng.choice([0.0, 1.2]))
    return _sizes(case)


def work(case):
    op = case["op"]
    if op == "norm":
        n, rows = case["tokens"] * case["hidden"], case["tokens"]
        per = 2 + 2 + 2 + (1 + 4 / BLOCK if case["fp8"] else 2) + (8 if case["train"] else 0)
        return {"bytes": n * per + rows * (8 if case["train"] else 0) + case["hidden"] * 4,
                "flops": n * (18 if case["train"] else 7)}
    if op == "route":
        n, s = case["tokens"] * case["experts"], 2 if case["bf16"] else 4
        picks = case["tokens"] * case["topk"]
        return {"bytes": n * s * (2 if case["train"] else 1) + picks * (12 if case["train"] else 8)
                + case["tokens"] * (1 if case["masked"] else 0),
                "flops": n * (14 if case["train"] else 5)}
    if op == "product":
        rows = case["out"] * (2 if case["gated"] else 1)
        weights = min(case["experts"], case["picks"]) * rows * case["width"]
        made = case["picks"] * case["out"] * (1 + 4 / BLOCK if case["gated"] else 2)
        return {"bytes": weights + case["picks"] * case["width"] * (1 + 4 / BLOCK) + made,
                "flops": 2 * case["picks"] * rows * case["width"]}
    tokens, per = case["ranks"] * case["tokens_per_rank"], case["experts"] // case["ranks"]
    rows = int(_there(_routing(case), case["ranks"], per).sum())
    return {"bytes": (tokens * case["topk"] + rows) * case["hidden"] * 2 + rows * case["topk"] * 8
            + tokens * case["topk"] * 4, "flops": 2 * tokens * case["topk"] * case["hidden"]}


# --------------------------------------------------------------------- inputs
def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed((int(seed) * 1000003 + salt) % (1 << 62))


def _randn(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _row_bytes(width):
    return -(-(width + 4 * -(-width // BLOCK)) // 16) * 16


def _packed(rows, width):
    """Room for 8-bit rows of `width` columns: the values and the scales, views of one buffer."""
    buf = torch.empty(rows, _row_bytes(width), dtype=torch.uint8, device="cuda")
    blocks = -(-width // BLOCK)
    at = -(-width // 4) * 4
    if at + 4 * blocks > buf.shape[1]:
        raise ValueError("width")
    return buf[:, :width].view(torch.float8_e4m3fn), buf[:, at:at + 4 * blocks].view(torch.float32)


def _columns(x):
    """x with its columns cut into blocks of 128 (the last one filled up with zeros)."""
    pad = -x.shape[-1] % BLOCK
    x = torch.nn.functional.pad(x, (0, pad)) if pad else x
    return x.reshape(*x.shape[:-1], -1, BLOCK)


def _quantize(y):
    """8-bit values and scales of fp32 rows."""
    blocks = _columns(y)
    most = blocks.abs().amax(-1).clamp_min(FLOOR)
    q = (blocks * (FP8_MAX / most)[..., None]).clamp(-FP8_MAX, FP8_MAX)
    q = q.reshape(*y.shape[:-1], -1)[..., :y.shape[-1]]
    return q.to(torch.float8_e4m3fn), most / FP8_MAX


def _spread(scales, width):
    """Block scales, one for each column."""
    return scales.repeat_interleave(BLOCK, -1)[..., :width]


def _weights(g, shape, fan):
    """Expert matrices [..., rows, columns] in 8 bits with a scale for each block of 128 x 128."""
    w = _randn(g, *shape) * fan ** -0.5
    rows, cols = shape[-2], shape[-1]
    rb, cb = -(-rows // BLOCK), -(-cols // BLOCK)
    full = torch.nn.functional.pad(w, (0, cb * BLOCK - cols, 0, rb * BLOCK - rows)) if rows % BLOCK or cols % BLOCK else w
    tiles = full.reshape(*shape[:-2], rb, BLOCK, cb, BLOCK)
    most = tiles.abs().amax((-3, -1)).clamp_min(FLOOR)
    q = (tiles * (FP8_MAX / most)[..., :, None, :, None]).clamp(-FP8_MAX, FP8_MAX)
    q = q.reshape(full.shape)[..., :rows, :cols].to(torch.float8_e4m3fn).contiguous()
    return q, (most / FP8_MAX).contiguous()


def prepare(case, seed):
    g = _gen(seed, 17)
    return dict(_INPUTS[case["op"]](case, g), case=case)


def _norm_inputs(case, g):
    t, h = case["tokens"], case["hidden"]
    # the stream grows over the layers and a few channels carry large values
    loud = 1 + 9 * (torch.rand(h, device="cuda", generator=g) < 0.01)
    s = dict(x=_randn(g, t, h).to(torch.bfloat16), residual=(_randn(g, t, h) * 3 * loud).to(torch.bfloat16),
             weight=(1 + 0.1 * _randn(g, h)).to(torch.bfloat16))
    if case["train"]:
        s["dout"] = (_randn(g, t, h) * 1e-2).to(torch.bfloat16)
        s["dresidual"] = (_randn(g, t, h) * 1e-2).to(torch.bfloat16)
    return s


def _route_inputs(case, g):
    t, e, k = case["tokens"], case["experts"], case["topk"]
    logits = _randn(g, t, e) * 1.5 + _randn(g, e) * 0.5     # some experts are liked more
    s = dict(mask=None)
    if case["masked"]:
        off = torch.rand(t, e, device="cuda", generator=g) < 0.1
        off |= torch.rand(t, 1, device="cuda", generator=g) < 0.02      # rows with no expert left
        logits = logits.masked_fill(off, NEG)
        s["mask"] = torch.rand(t, device="cuda", generator=g) < 0.9     # False: a padded token
    s["logits"] = logits.to(torch.bfloat16 if case["bf16"] else torch.float32)
    if case["train"]:
        s["coef"] = 1e-2
        s["dweights"] = _randn(g, t, k) * 1e-3
        s["dloss"] = 0.5 + torch.rand((), device="cuda", generator=g)
    return s


def _product_inputs(case, g):
    e, m, k, n = case["experts"], case["picks"], case["width"], case["out"]
    like = torch.rand(e, device="cuda", generator=g) + 0.25
    expert = torch.multinomial(like, m, replacement=True, generator=g) if m else torch.zeros(0, dtype=torch.long)
    count = torch.bincount(expert, minlength=e)
    s = dict(expert_count=count.to(torch.int32), expert_off=(count.cumsum(0) - count).to(torch.int32), rows=None)
    have = m
    if case["gated"]:     # the first product takes its rows out of the receive buffer
        have = max(1, m * 10 // 11)
        row = torch.randint(have, (m,), device="cuda", generator=g)
        s["rows"] = ((expert * have + row).sort().values % have).to(torch.int32)
    values, scales = _packed(have, k)
    q, sc = _quantize(_randn(g, have, k) * (0.5 + torch.rand(have, 1, device="cuda", generator=g)))
    values.copy_(q)
    scales.copy_(sc)
    s["values"], s["scales"] = values, scales
    s["w"], s["w_scales"] = _weights(g, (e, 2, n, k) if case["gated"] else (e, n, k), k)
    return s


def _routing(case):
    """The picks of a step's tokens: the case's own, so that its count of receive rows is; the seed orders the tokens."""
    e, k = case["experts"], case["topk"]
    t, g = case["ranks"] * case["tokens_per_rank"], _gen(1, 29)
    like = -case["zipf"] * torch.log(torch.randperm(e, device="cuda", generator=g).float() + 1)
    noise = -torch.log(-torch.log(torch.rand(t, e, device="cuda", generator=g).clamp(1e-7, 1 - 1e-7)))
    return (like + noise).topk(k, -1).indices


def _there(idx, ranks, per):
    """Which ranks each token reaches: [tokens, ranks]."""
    return torch.zeros(idx.shape[0], ranks, dtype=torch.bool, device="cuda").scatter_(1, idx // per, True)


def _sum_inputs(case, g):
    r, e, k, h = case["ranks"], case["experts"], case["topk"], case["hidden"]
    t, per = r * case["tokens_per_rank"], e // r
    idx = _routing(case)[torch.randperm(t, device="cuda", generator=g)]
    weights = torch.softmax(_randn(g, t, k), -1)
    there = _there(idx, r, per)
    count = there.sum(0)
    base = count.cumsum(0) - count
    rank, token = there.t().nonzero(as_tuple=True)          # receive rows: by rank, then by token
    local = (idx[token] // per) == rank[:, None]
    row = base + there.cumsum(0) - 1                        # [t, r]
    row = row.gather(1, idx // per)                         # the receive row of each pick
    n = rank.numel()
    key = (idx * n + row).reshape(-1).sort().values
    picks = torch.bincount(idx.reshape(-1), minlength=e)
    i32 = torch.int32
    return dict(recv_topk_idx=torch.where(local, idx[token] % per, -1).to(i32),
                recv_topk_weights=torch.where(local, weights[token], 0.0), recv_base=base.to(i32),
                expert_rows=(key % n).to(i32), expert_count=picks.to(i32),
                expert_off=(picks.cumsum(0) - picks).to(i32), y=_randn(g, t * k, h).to(torch.bfloat16))


_INPUTS = {"norm": _norm_inputs, "route": _route_inputs, "product": _product_inputs, "sum": _sum_inputs}


# ------------------------------------------------------------------ the calls
def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def _norm_own(s):
    import combine_ep_layout_04_gb300 as ep
    c = s["case"]
    n = ep.rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, fp8=c["fp8"], save_rstd=c["train"])
    if not c["train"]:
        if c["fp8"]:
            return {"values": n.out.values, "scales": n.out.scales, "residual": n.residual}
        return {"out": n.out, "residual": n.residual}
    dx, dw = ep.rms_norm_backward(s["dout"], n.residual, s["weight"], n.rstd, dresidual=s["dresidual"])
    return {"out": n.out, "residual": n.residual, "dx": dx, "dweight": dw}


def _norm_plain(s):
    c = s["case"]
    h = s["x"].float() + s["residual"].float()
    rstd = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
    y = h * rstd * s["weight"].float()
    h = h.to(torch.bfloat16)
    if not c["train"]:
        if c["fp8"]:
            q, sc = _quantize(y)
            return {"values": q, "scales": sc, "residual": h}
        return {"out": y.to(torch.bfloat16), "residual": h}
    unit = h.float() * rstd
    dout = s["dout"].float()
    dw = (dout * unit).sum(0)
    dunit = dout * s["weight"].float()
    dx = s["dresidual"].float() + rstd * (dunit - unit * (dunit * unit).mean(-1, keepdim=True))
    return {"out": y.to(torch.bfloat16), "residual": h, "dx": dx.to(torch.bfloat16), "dweight": dw}


def _route_own(s):
    import combine_ep_layout_04_gb300 as ep
    c = s["case"]
    r = ep.route(s["logits"], c["topk"], renormalize=c["renorm"], token_mask=s["mask"],
                 balance_coef=s["coef"] if c["train"] else None)
    if not c["train"]:
        return {"idx": r.topk_idx, "weights": r.topk_weights}
    return {"idx": r.topk_idx, "weights": r.topk_weights, "count": r.expert_count, "loss": r.balance_loss,
            "dlogits": ep.route_backward(s["logits"], r, s["dweights"], s["dloss"])}


def _route_plain(s):
    c, logits = s["case"], s["logits"].float()
    t, e, k = c["tokens"], c["experts"], c["topk"]
    live = torch.ones(t, 1, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"][:, None]
    logits = torch.where(live, logits, NEG)
    top, idx = (v[:, :k] for v in logits.sort(dim=-1, descending=True, stable=True))
    picked = top > NEG
    most = logits.amax(-1, keepdim=True)
    most = torch.where(most > NEG, most, 0.0)
    total = torch.exp(logits - most).sum(-1, keepdim=True)
    p = torch.exp(logits - most) / torch.where(total > 0, total, 1.0)
    w = p.gather(1, idx)
    if c["renorm"]:
        w = torch.exp(top - most)
        share = w.sum(-1, keepdim=True)
        w = w / torch.where(share > 0, share, 1.0)
    out_idx = torch.where(picked, idx, -1).to(torch.int32)
    if not c["train"]:
        return {"idx": out_idx, "weights": w}
    hot = torch.zeros(t, e, device="cuda").scatter_add_(1, idx, picked.float())
    count = hot.sum(0)
    tokens = live.sum().float().clamp_min(1.0)
    slope = s["coef"] * e / (k * tokens * tokens) * count            # d loss / d p[t, e]
    loss = (slope * p.sum(0)).sum()
    dw = torch.where(picked, s["dweights"], 0.0)
    dp = (slope * s["dloss"]).expand(t, e)
    if not c["renorm"]:
        dp = dp.scatter_add(1, idx, dw)
    dlogits = p * (dp - (p * dp).sum(-1, keepdim=True))
    if c["renorm"]:
        dlogits = dlogits.scatter_add(1, idx, w * (dw - (w * dw).sum(-1, keepdim=True)))
    return {"idx": out_idx, "weights": w, "count": count.to(torch.int32), "loss": loss,
            "dlogits": dlogits.to(s["logits"].dtype)}


def _product_own(s):
    import combine_ep_layout_04_gb300 as ep
    y = ep.expert_product(ep.Fp8Rows(s["values"], s["scales"]), s["w"], s["w_scales"], s["expert_off"],
                          s["expert_count"], rows=s["rows"])
    return {"values": y.values, "scales": y.scales} if s["case"]["gated"] else {"out": y}


def _product_plain(s):
    c = s["case"]
    a = s["values"].float() * _spread(s["scales"], c["width"])
    if s["rows"] is not None:
        a = a[s["rows"].long()]
    w = s["w"].float() * _spread(s["w_scales"], c["width"]).repeat_interleave(BLOCK, -2)[..., :c["out"], :]
    count = s["expert_count"].long()
    most = int(count.max())
    # each expert's rows, filled up to the longest expert's
    at = s["expert_off"].long()[:, None] + torch.arange(most, device="cuda")
    full = torch.arange(most, device="cuda") < count[:, None]
    y = torch.bmm(a[at.clamp_max(c["picks"] - 1)], w.reshape(c["experts"], -1, c["width"]).transpose(1, 2))[full]
    if not c["gated"]:
        return {"out": y.to(torch.bfloat16)}
    gate, up = y[:, :c["out"]], y[:, c["out"]:]
    q, sc = _quantize(gate / (1 + torch.exp(-gate)) * up)
    return {"values": q, "scales": sc}


def _sum_own(s):
    import combine_ep_layout_04_gb300 as ep
    return {"out": ep.pick_sum(s["y"], s["recv_topk_idx"], s["recv_topk_weights"], s["recv_base"], s["expert_off"],
                               s["expert_count"], s["expert_rows"])}


def _sum_plain(s):
    c = s["case"]
    n, per = s["recv_topk_idx"].shape[0], c["experts"] // c["ranks"]
    rank = (torch.arange(n, device="cuda")[:, None] >= s["recv_base"].long()).sum(-1) - 1
    local = s["recv_topk_idx"].long()
    there = local >= 0
    # a pick's place is found by its expert and row: the places are in that order
    of_place = torch.repeat_interleave(torch.arange(c["experts"], device="cuda"), s["expert_count"].long())
    place = torch.searchsorted(of_place * n + s["expert_rows"].long(),
                               (rank[:, None] * per + local) * n + torch.arange(n, device="cuda")[:, None])
    place = torch.where(there, place, 0)
    w = torch.where(there, s["recv_topk_weights"], 0.0)
    return {"out": (s["y"][place].float() * w[..., None]).sum(1).to(torch.bfloat16)}


_OWN = {"norm": _norm_own, "route": _route_own, "product": _product_own, "sum": _sum_own}
_PLAIN = {"norm": _norm_plain, "route": _route_plain, "product": _product_plain, "sum": _sum_plain}


# -------------------------------------------------------------- in 64 bits
def exact(case, seed):
    return _EXACT[case["op"]](prepare(case, seed))


def _scaled64(y):
    """What 8-bit values stand for before they are rounded (the row over its block's scale), and the scales."""
    rows, width = y.shape
    blocks = -(-width // BLOCK)
    values, scales = torch.empty_like(y), y.new_empty(rows, blocks)
    for b in range(blocks):
        part = y[:, b * BLOCK:(b + 1) * BLOCK]
        scales[:, b] = torch.clamp(part.abs().max(1).values, min=FLOOR) / 448
        values[:, b * BLOCK:(b + 1) * BLOCK] = part / scales[:, b:b + 1]
    return values, scales


def _norm_exact(s):
    c = s["case"]
    t, width = c["tokens"], c["hidden"]
    w = s["weight"].double()
    got = {}
    dw = torch.zeros(width, dtype=torch.float64, device="cuda")
    for i in range(0, t, 16384):      # a part of the tokens at a time
        part = slice(i, min(t, i + 16384))
        h = s["x"][part].double() + s["residual"][part].double()
        root = torch.sqrt(h.square().sum(1) / width + EPS)
        y = w * h / root[:, None]
        one = {"residual": h.float()}
        if c["fp8"]:
            v, sc = _scaled64(y)
            one.update(values=v.float(), scales=sc)
        else:
            one["out"] = y.float()
        if c["train"]:
            stored = h.to(torch.bfloat16).double()       # the backward pass has the stream as it is kept
            g = s["dout"][part].double()
            dw += torch.einsum("th,th,t->h", g, stored, 1 / root)
            inner = torch.einsum("th,th,h->t", g, stored, w)
            dx = s["dresidual"][part].double() + g * w / root[:, None]
            one["dx"] = (dx - stored * (inner / (width * root ** 3))[:, None]).float()
        for k, v in one.items():
            got.setdefault(k, []).append(v)
    got = {k: torch.cat(v) for k, v in got.items()}
    if c["train"]:
        got["dweight"] = dw
    return got


def _route_exact(s):
    c = s["case"]
    t, e, k = c["tokens"], c["experts"], c["topk"]
    x = s["logits"].double().clone()
    live = torch.ones(t, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"]
    x[~live] = NEG
    left, idx = x.clone(), torch.full((t, k), -1, dtype=torch.int32, device="cuda")
    some = x.max(1).values > NEG
    p = torch.zeros_like(x)
    p[some] = torch.softmax(x[some], 1)
    w = torch.zeros(t, k, dtype=torch.float64, device="cuda")
    rows = torch.arange(t, device="cuda")
    column = torch.arange(e, device="cuda")
    for j in range(k):                # one pick after another; the first of equals
        most = left.max(1).values
        at = torch.where(left == most[:, None], column, e).min(1).values
        ok = most > NEG
        idx[ok, j] = at[ok].to(torch.int32)
        w[ok, j] = p[rows, at][ok]
        left[rows[ok], at[ok]] = NEG
    if c["renorm"]:
        lift = torch.where(idx >= 0, x.gather(1, idx.clamp_min(0).long()), NEG)
        w = torch.where(some[:, None], torch.softmax(lift, 1), 0.0)
    if not c["train"]:
        return {"idx": idx, "weights": w}
    count = torch.bincount(idx[idx >= 0].long(), minlength=e)
    tokens = max(1, int(live.sum()))
    often = count.double() * e / (k * tokens)
    loss = s["coef"] * (often * p.sum(0) / tokens).sum()
    dp = (s["dloss"].double() * s["coef"] * often / tokens).repeat(t, 1)
    at = idx.clamp_min(0).long()
    dw = torch.where(idx >= 0, s["dweights"].double(), 0.0)
    if c["renorm"]:       # w = p / (sum of the picked p)
        share = torch.where(idx >= 0, p.gather(1, at), 0.0).sum(1, keepdim=True).clamp_min(1e-300)
        dp.scatter_add_(1, at, (dw - (dw * w).sum(1, keepdim=True)) / share * (idx >= 0))
    else:
        dp.scatter_add_(1, at, dw)
    return {"idx": idx, "weights": w, "count": count.to(torch.int32), "loss": loss,
            "dlogits": p * dp - p * (p * dp).sum(1, keepdim=True)}


def _product_exact(s):
    c = s["case"]
    width, out = c["width"], c["out"]
    parts = []
    off = 0
    block = torch.arange(width, device="cuda") // BLOCK
    for x, n in enumerate(s["expert_count"].tolist()):      # expert after expert
        at = torch.arange(off, off + n, device="cuda")
        off += n
        if not n:
            continue
        at = at if s["rows"] is None else s["rows"][at].long()
        a = s["values"][at].double() * s["scales"][at].double()[:, block]
        halves = [(s["w"][x, i], s["w_scales"][x, i]) for i in (0, 1)] if c["gated"] else [(s["w"][x], s["w_scales"][x])]
        line = torch.arange(out, device="cuda") // BLOCK
        y = [a @ (q.double() * sc.double()[line][:, block]).t() for q, sc in halves]
        parts.append(y[0] if not c["gated"] else y[0] * torch.sigmoid(y[0]) * y[1])
    y = torch.cat(parts)
    if not c["gated"]:
        return {"out": y}
    v, sc = _scaled64(y)
    return {"values": v, "scales": sc}


def _sum_exact(s):
    c = s["case"]
    n, per = s["recv_topk_idx"].shape[0], c["experts"] // c["ranks"]
    out = torch.zeros(n, c["hidden"], dtype=torch.float64, device="cuda")
    bases = s["recv_base"].tolist() + [n]
    off = s["expert_off"].tolist()
    count = s["expert_count"].tolist()
    for d in range(c["ranks"]):       # the rows of an expert are all on its rank, each once
        for e in range(d * per, (d + 1) * per):
            rows = s["expert_rows"][off[e]:off[e] + count[e]].long()
            w = s["recv_topk_weights"].double()[rows] * (s["recv_topk_idx"][rows] == e - d * per)
            assert bases[d] <= int(rows.min() if count[e] else bases[d])
            out[rows] += w.sum(1)[:, None] * s["y"][off[e]:off[e] + count[e]].double()
    return {"out": out}


_EXACT = {"norm": _norm_exact, "route": _route_exact, "product": _product_exact, "sum": _sum_exact}
