"""Measured cases of the MoE operators around the expert layer: the router's
top-k with its gradient, tokens sorted by expert and back with their weights
and gradients, matrix-vector products with NVFP4 weights, and the expert layer
for a few tokens on unquantized activations.

A case names an operator and its sizes.  prepare() makes what a program holds
before the call; run() makes one call, either of the package's entry points
(own) or in plain torch operations in binary32; exact() is the definition in
binary64.  Sizes follow the Qwen3-30B-A3B-shaped expert layer of workloads.py
(hidden 2048, 128 experts, top-8, intermediate 768) and its dense projections;
the odd ones are generic.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
# E2M1 values of the codes 0..15 (bit 3 is the sign)
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one new token's router logits: pure latency
        dict(name="router_t1", op="router", tokens=1, experts=128, topk=8, dtype="bf16", score=0,
             renorm=True, bias=False, masked=0),
        # a long prompt's or training batch's router
        dict(name="router_t32768", op="router", tokens=32768, experts=128, topk=8, dtype="fp32",
             score=0, renorm=True, bias=False, masked=0),
        # the router's gradient on a training batch, softmax over all of many
        # experts, some of them masked out
        dict(name="router_backward_t8191_e1000", op="router_backward", tokens=8191, experts=1000,
             topk=6, dtype="bf16", score=0, renorm=False, masked=10),
        # a training batch's rows brought into expert order
        dict(name="sort_t8192", op="sort", tokens=8192, hidden=2048, experts=128, topk=8, align=1,
             dropped=0.0, weighted=False, dtype="bf16"),
        # gradient of a weighted sort with padding, dropped entries, odd width
        dict(name="sort_backward_t1003_h1111", op="sort_backward", tokens=1003, hidden=1111,
             experts=60, topk=4, align=16, dropped=0.05, weighted=True, dtype="fp16"),
        # the rows of a serving batch back in token order, weighted
        dict(name="unsort_t256", op="unsort", tokens=256, hidden=2048, experts=128, topk=8, align=1,
             dropped=0.0, weighted=True, dtype="bf16"),
        # gradient of the weighted unsort on the long layer: rows and weights
        dict(name="unsort_backward_t32768", op="unsort_backward", tokens=32768, hidden=2048,
             experts=128, topk=8, align=1, dropped=0.0, weighted=True, dtype="bf16"),
        # the QKV projection of one new token
        dict(name="matvec_t1_qkv", op="matvec", tokens=1, n=5120, k=2048, tiled=True, dtype="bf16"),
        # a large projection of 64 sequences' new tokens
        dict(name="matvec_t64_n32768", op="matvec", tokens=64, n=32768, k=8192, tiled=False,
             dtype="fp16"),
        # one expert projection at sizes no tile divides, with dropped entries
        dict(name="expert_matvec_t37_odd", op="expert_matvec", tokens=37, n=1001, k=1040, experts=60,
             topk=4, dropped=0.05, tiled=False, dtype="fp32"),
        # the expert layer of one new token
        dict(name="decode_t1", op="decode", tokens=1, hidden=2048, inter=768, experts=128, topk=8,
             dropped=0.0, tiled=True, dtype="bf16"),
        # the expert layer of 256 sequences' new tokens: every expert is read
        dict(name="decode_t256", op="decode", tokens=256, hidden=2048, inter=768, experts=128,
             topk=8, dropped=0.0, tiled=True, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ones' ranges."""
    op = rng.choice(["router", "router_backward", "sort", "sort_backward", "unsort",
                     "unsort_backward", "matvec", "matvec", "expert_matvec", "decode", "decode"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("router", "router_backward"):
        experts = _log(rng, 4, 1024)
        tokens = min(_log(rng, 1, 32768), 8192000 // experts)
        c = dict(op=op, tokens=tokens, experts=experts, topk=rng.randint(1, min(experts, 10)),
                 dtype=dtype, score=rng.choice([0, 0, 1]), renorm=rng.random() < 0.6,
                 masked=rng.choice([0, 0, experts // 4]))
        if op == "router":
            c["bias"] = rng.random() < 0.3
        return c
    if op in ("sort", "sort_backward", "unsort", "unsort_backward"):
        experts = _log(rng, 4, 256)
        topk = rng.randint(1, min(experts, 10))
        hidden = _log(rng, 64, 8192)
        hidden = hidden if rng.random() < 0.4 else (hidden + 7) // 8 * 8
        tokens = max(1, min(_log(rng, 1, 32768), (1 << 28) // (hidden * topk)))
        return dict(op=op, tokens=tokens, hidden=hidden, experts=experts, topk=topk,
                    align=rng.choice([1, 1, 16, 128]), dropped=rng.choice([0.0, 0.0, 0.1]),
                    weighted=rng.random() < 0.6, dtype=dtype)
    tiled = rng.random() < 0.5
    if op == "matvec":
        n, k = _log(rng, 32, 32768), _log(rng, 64, 8192)
        n, k = ((n + 31) // 32 * 32, (k + 127) // 128 * 128) if tiled else (n, (k + 15) // 16 * 16)
        return dict(op=op, tokens=_log(rng, 1, 64), n=n, k=k, tiled=tiled, dtype=dtype)
    experts = _log(rng, 4, 128)
    topk = rng.randint(1, min(experts, 8))
    tokens = _log(rng, 1, 256)
    dropped = rng.choice([0.0, 0.0, 0.1])
    if op == "expert_matvec":
        n, k = _log(rng, 32, 2048), _log(rng, 64, 2048)
        n, k = ((n + 31) // 32 * 32, (k + 127) // 128 * 128) if tiled else (n, (k + 15) // 16 * 16)
        return dict(op=op, tokens=tokens, n=n, k=k, experts=experts, topk=topk, dropped=dropped,
                    tiled=tiled, dtype=dtype)
    m = 128 if tiled else 16
    hidden, inter = _log(rng, 128, 2048), _log(rng, 128, 768)
    return dict(op=op, tokens=tokens, hidden=(hidden + m - 1) // m * m,
                inter=(inter + m - 1) // m * m, experts=experts, topk=topk, dropped=dropped,
                tiled=tiled, dtype=dtype)


# ---- inputs ----------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std


def _logits(g, tokens, experts):
    """N(0, 1) logits with a falling bias, as workloads.py's stand-in."""
    e = torch.arange(1, experts + 1, device="cuda", dtype=torch.float32)
    return _normal(g, tokens, experts) - 0.5 * torch.log(e)


def _picks(g, tokens, experts, topk, dropped, even=False):
    """Distinct experts of each token and their weights; some entries dropped."""
    logits = _normal(g, tokens, experts) if even else _logits(g, tokens, experts)
    v, idx = torch.topk(logits, topk, dim=1)
    prob = torch.softmax(v, dim=1).contiguous()
    idx = idx.to(torch.int32)
    if dropped:
        gone = torch.rand((tokens, topk), generator=g, device="cuda") < dropped
        idx = torch.where(gone, torch.full_like(idx, -1), idx)
    return idx.contiguous(), prob


def _routing(idx, experts, align):
    """Rows of the routed entries in expert order, as moe_permute lays them."""
    tokens, topk = idx.shape
    cap = tokens * topk + experts * (align - 1)
    flat = idx.reshape(-1).long()
    key = torch.where(flat >= 0, flat, torch.full_like(flat, experts))
    order = torch.argsort(key, stable=True)
    count = torch.bincount(key, minlength=experts + 1)
    padded = (count[:experts] + align - 1) // align * align
    offsets = torch.zeros(experts + 1, dtype=torch.long, device="cuda")
    offsets[1:] = torch.cumsum(padded, 0)
    first = torch.zeros(experts + 1, dtype=torch.long, device="cuda")
    first[1:] = torch.cumsum(count, 0)[:experts]
    sorted_key = key[order]
    place = torch.arange(flat.numel(), device="cuda") - first[sorted_key]
    row = torch.where(sorted_key < experts, offsets[sorted_key.clamp(max=experts - 1)] + place,
                      torch.full_like(place, -1))
    dst = torch.empty_like(flat)
    dst[order] = row
    src = torch.full((cap + 1,), -1, dtype=torch.int32, device="cuda")
    src[torch.where(dst >= 0, dst, torch.full_like(dst, cap))] = (
        torch.arange(flat.numel(), device="cuda") // topk).to(torch.int32)
    src[cap] = -1
    return dict(dst_row=dst.to(torch.int32).view(tokens, topk), row_src=src[:cap].contiguous(),
                offsets=offsets.to(torch.int32))


def _weights(g, groups, n, k, tiled):
    """NVFP4 weights of N(0, 0.02) matrices: codes, E4M3 block scales and one
    outer scale per matrix, row-major and, if asked, in the tiled layout."""
    codes = torch.empty((groups, n, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((groups, n, k // 16), dtype=torch.uint8, device="cuda")
    outer = torch.empty(groups, dtype=torch.float32, device="cuda")
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    step = max(1, (1 << 27) // (n * k))
    for a in range(0, groups, step):
        w = _normal(g, min(step, groups - a), n, k // 16, 16, std=0.02)
        amax = w.abs().amax(dim=(1, 2, 3))
        sg = (amax / 2688.0).view(-1, 1, 1)
        s8 = (w.abs().amax(dim=3) / (6.0 * sg)).clamp(max=448.0).to(torch.float8_e4m3fn)
        d = (s8.float() * sg).unsqueeze(-1)
        q = torch.bucketize(w.abs() / d.clamp(min=1e-30), edges).to(torch.uint8)
        q = (q | ((w < 0).to(torch.uint8) << 3)).view(-1, n, k // 2, 2)
        codes[a:a + step] = q[..., 0] | (q[..., 1] << 4)
        scales[a:a + step] = s8.view(torch.uint8)
        outer[a:a + step] = amax / 2688.0
    w = dict(codes=codes, scales=scales, outer=outer, layout=0, as_held=(codes, scales))
    if tiled:
        t = codes.view(groups, n // 32, 32, k // 128, 2, 2, 16)
        s = scales.view(groups, n // 32, 32, k // 128, 2, 4)
        w["as_held"] = (t.permute(0, 1, 3, 5, 4, 2, 6).contiguous().view(codes.shape),
                        s.permute(0, 1, 3, 4, 2, 5).contiguous().view(scales.shape))
        w["layout"] = 1
    return w


def prepare(case, seed):
    g, c, op = _gen(seed), case, case["op"]
    t = DTYPES[c["dtype"]]
    s = dict(case=case)
    if op in ("router", "router_backward"):
        logits = _logits(g, c["tokens"], c["experts"])
        if c["masked"]:
            gone = torch.rand(logits.shape, generator=g, device="cuda").argsort(1) < c["masked"]
            logits = logits.masked_fill(gone, -math.inf)
            if c["tokens"] > 4:
                logits[c["tokens"] // 2] = -math.inf        # nothing left to pick
        s["logits"] = logits.to(t)
        if op == "router":
            s["bias"] = _normal(g, c["experts"], std=0.1) if c["bias"] else None
        else:
            v, i = torch.topk(s["logits"].float(), c["topk"], dim=1)
            s["idx"] = torch.where(v > -math.inf, i, torch.full_like(i, -1)).to(torch.int32)
            s["dprob"] = _normal(g, c["tokens"], c["topk"], std=0.1)
        return s
    if op in ("matvec", "expert_matvec", "decode"):
        if op == "matvec":
            s["x"] = _normal(g, c["tokens"], c["k"]).to(t)
            s["w"] = _weights(g, 1, c["n"], c["k"], c["tiled"])
            return s
        s["idx"], s["prob"] = _picks(g, c["tokens"], c["experts"], c["topk"], c["dropped"], True)
        if op == "expert_matvec":
            s["x"] = _normal(g, c["tokens"], c["k"]).to(t)
            s["w"] = _weights(g, c["experts"], c["n"], c["k"], c["tiled"])
            return s
        s["x"] = _normal(g, c["tokens"], c["hidden"]).to(t)
        s["w1"] = _weights(g, c["experts"], 2 * c["inter"], c["hidden"], c["tiled"])
        s["w2"] = _weights(g, c["experts"], c["hidden"], c["inter"], c["tiled"])
        return s
    idx, prob = _picks(g, c["tokens"], c["experts"], c["topk"], c["dropped"])
    s.update(_routing(idx, c["experts"], c["align"]))
    s["prob"] = prob if c["weighted"] else None
    cap = s["row_src"].numel()
    if op in ("sort", "unsort_backward"):
        # rows behind the last expert's are not written: the program's buffer
        s["out"] = torch.zeros((cap, c["hidden"]), dtype=t, device="cuda")
        s["tok"] = _normal(g, c["tokens"], c["hidden"]).to(t)
    if op in ("sort_backward", "unsort", "unsort_backward"):
        s["rows"] = _normal(g, cap, c["hidden"]).to(t)
    if op == "sort_backward":
        s["tok"] = _normal(g, c["tokens"], c["hidden"]).to(t)
    return s


# ---- one call ----------------------------------------------------------------

def run(state):
    return (_own if own else _plain)(state, state["case"])


def _own(s, c):
    from nvfp4_w4a4_quantized_amd import ops
    op = c["op"]

    def held(w):
        return ops.NvFp4Weights(*w["as_held"], w["outer"], layout=w["layout"])

    if op == "router":
        return ops.moe_router(s["logits"], c["topk"], bias=s["bias"], score=c["score"],
                              renormalize=c["renorm"])
    if op == "router_backward":
        return ops.moe_router_backward(s["dprob"], s["logits"], s["idx"], score=c["score"],
                                       renormalize=c["renorm"])
    if op == "sort":
        return ops.moe_sort_tokens(s["tok"], s["dst_row"], s["row_src"], s["offsets"],
                                   prob=s["prob"], out=s["out"])
    if op == "sort_backward":
        if c["weighted"]:
            return ops.moe_sort_tokens_backward(s["rows"], s["dst_row"], x=s["tok"],
                                                prob=s["prob"])
        return ops.moe_sort_tokens_backward(s["rows"], s["dst_row"])
    if op == "unsort":
        return ops.moe_unsort_tokens(s["rows"], s["dst_row"], prob=s["prob"])
    if op == "unsort_backward":
        return ops.moe_unsort_tokens_backward(s["tok"], s["dst_row"], s["row_src"], s["offsets"],
                                              rows=s["rows"] if c["weighted"] else None,
                                              prob=s["prob"], out=s["out"])
    if op == "matvec":
        return ops.nvfp4_matvec(s["x"], held(s["w"]))
    if op == "expert_matvec":
        return ops.nvfp4_expert_matvec(s["x"], s["idx"], held(s["w"]))
    return ops.moe_expert_decode(s["x"], s["idx"], s["prob"], c["experts"], c["inter"],
                                 held(s["w1"]), held(s["w2"]))


def _values(codes, scales, outer):
    """Weights in binary32: code value * block scale * outer scale."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    q = grid[torch.stack((codes & 15, codes >> 4), dim=-1).int()]
    q = q.view(*scales.shape, 16) * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)
    return (q * outer.view(-1, 1, 1, 1)).view(codes.shape[0], codes.shape[1], -1)


def _products(x, idx, w, by_entry):
    """x . W[e]^T for every entry: [T, k, n]; x [T, K] or (by_entry) [T, k, K]."""
    tokens, topk = idx.shape
    groups, n, _ = w["codes"].shape
    e = idx.clamp(min=0).long().view(-1)
    t = torch.arange(tokens * topk, device=x.device)
    t = t if by_entry else t // topk
    x = x.reshape(-1, x.shape[-1])
    if e.numel() <= groups:
        m = _values(w["codes"][e], w["scales"][e], w["outer"][e])
        y = torch.bmm(m, x[t].unsqueeze(-1)).squeeze(-1)
    else:
        m = _values(w["codes"], w["scales"], w["outer"])
        y = torch.mm(m.view(groups * n, -1), x.t().contiguous()).view(groups, n, -1)
        y = y[e, :, t]
    return y.view(tokens, topk, n) * (idx >= 0).unsqueeze(-1)


def _picked(rows, dst):
    """The rows of every entry in binary32, zeros for entries not routed."""
    return rows[dst.clamp(min=0).long()].float() * (dst >= 0).unsqueeze(-1)


def _plain(s, c):
    op, t = c["op"], DTYPES[c["dtype"]]
    if op == "router":
        z = s["logits"].float()
        key = z if s["bias"] is None else z + s["bias"]
        v, i = torch.sort(key, dim=1, descending=True, stable=True)
        v, i = v[:, :c["topk"]], i[:, :c["topk"]]
        ok = v > -math.inf
        zs = z.gather(1, i)
        if c["renorm"]:
            l = zs if c["score"] == 0 else torch.nn.functional.logsigmoid(zs)
            p = torch.softmax(l, dim=1)
        else:
            p = (torch.softmax(z, dim=1) if c["score"] == 0 else torch.sigmoid(z)).gather(1, i)
        return (torch.where(ok, i, torch.full_like(i, -1)).to(torch.int32),
                torch.where(ok, p, torch.zeros_like(p)))
    if op == "router_backward":
        z = s["logits"].float()
        i, ok = s["idx"].clamp(min=0).long(), s["idx"] >= 0
        dp = s["dprob"] * ok
        zs = torch.where(ok, z.gather(1, i), torch.full_like(dp, -math.inf))
        none = ~ok.any(dim=1, keepdim=True)
        if c["renorm"]:
            l = zs if c["score"] == 0 else torch.nn.functional.logsigmoid(zs)
            q = torch.softmax(l, dim=1)
            dl = q * (dp - (q * dp).sum(1, keepdim=True))
            if c["score"] == 1:
                dl = dl * torch.sigmoid(-zs)
            dz = torch.zeros_like(z).scatter_add_(1, i, torch.where(ok, dl, torch.zeros_like(dl)))
        elif c["score"] == 0:
            p = torch.softmax(z, dim=1)
            d = torch.zeros_like(z).scatter_add_(1, i, dp)
            dz = p * (d - (p * d).sum(1, keepdim=True))
        else:
            dl = dp * torch.sigmoid(zs) * torch.sigmoid(-zs)
            dz = torch.zeros_like(z).scatter_add_(1, i, torch.where(ok, dl, torch.zeros_like(dl)))
        return dz.masked_fill(none, 0.0).to(t)
    if op == "sort" or op == "unsort_backward":
        rows = s["tok"][s["row_src"].clamp(min=0).long()].float()
        rows = rows * (s["row_src"] >= 0).unsqueeze(-1)
        if s["prob"] is not None:
            at = torch.where(s["dst_row"] >= 0, s["dst_row"],
                             torch.full_like(s["dst_row"], rows.shape[0])).long().view(-1)
            w = torch.zeros(rows.shape[0] + 1, device=rows.device)
            w[at] = s["prob"].view(-1)
            rows = rows * w[:-1].unsqueeze(-1)
        if op == "sort":
            return rows.to(t)
        if not c["weighted"]:
            return rows.to(t), None
        dprob = (_picked(s["rows"], s["dst_row"]) * s["tok"].float().unsqueeze(1)).sum(-1)
        return rows.to(t), dprob
    if op == "unsort" or op == "sort_backward":
        r = _picked(s["rows"], s["dst_row"])
        y = r if s["prob"] is None else r * s["prob"].unsqueeze(-1)
        y = y.sum(1).to(t)
        if op == "unsort":
            return y
        if not c["weighted"]:
            return y, None
        return y, (r * s["tok"].float().unsqueeze(1)).sum(-1)
    if op == "matvec":
        w = _values(s["w"]["codes"], s["w"]["scales"], s["w"]["outer"])[0]
        return torch.mm(w, s["x"].float().t().contiguous()).t().to(t).contiguous()
    if op == "expert_matvec":
        return _products(s["x"].float(), s["idx"], s["w"], False).to(t)
    h = _products(s["x"].float(), s["idx"], s["w1"], False)
    g, u = h[..., :c["inter"]], h[..., c["inter"]:]
    d = g * torch.sigmoid(g) * u * s["prob"].unsqueeze(-1)
    return _products(d, s["idx"], s["w2"], True).sum(1).to(t)


def work(case):
    """Bytes that have to move and operations that have to be done."""
    c, op, b = case, case["op"], SIZE[case["dtype"]]
    if op == "router":
        n = c["tokens"] * c["experts"]
        return dict(bytes=n * b + c["tokens"] * c["topk"] * 8 + (4 * c["experts"] if c["bias"] else 0),
                    flops=3 * n)
    if op == "router_backward":
        n = c["tokens"] * c["experts"]
        return dict(bytes=2 * n * b + c["tokens"] * c["topk"] * 8, flops=3 * n)
    if op in ("sort", "sort_backward", "unsort", "unsort_backward"):
        entries = c["tokens"] * c["topk"] * (1.0 - c["dropped"])
        rows, toks = entries * c["hidden"] * b, c["tokens"] * c["hidden"] * b
        moved = rows + toks + c["tokens"] * c["topk"] * 4
        flops = entries * c["hidden"] * (1 if op in ("unsort", "sort_backward") else 0)
        if c["weighted"]:
            moved += c["tokens"] * c["topk"] * 4
            flops += entries * c["hidden"]
            if op == "unsort_backward":
                moved += rows + c["tokens"] * c["topk"] * 4
                flops += 2 * entries * c["hidden"]
            if op == "sort_backward":
                moved += toks + c["tokens"] * c["topk"] * 4
                flops += 2 * entries * c["hidden"]
        return dict(bytes=int(moved), flops=int(flops))
    if op == "matvec":
        return dict(bytes=int(c["n"] * c["k"] * 9 / 16 + c["tokens"] * (c["n"] + c["k"]) * b + 4),
                    flops=2 * c["tokens"] * c["n"] * c["k"])
    entries = c["tokens"] * c["topk"] * (1.0 - c["dropped"])
    # experts that at least one of the tokens picked, on average
    hit = c["experts"] * (1.0 - (1.0 - (1.0 - c["dropped"]) * c["topk"] / c["experts"]) ** c["tokens"])
    if op == "expert_matvec":
        nk = c["n"] * c["k"]
        moved = hit * nk * 9 / 16 + c["tokens"] * c["k"] * b + c["tokens"] * c["topk"] * (4 + c["n"] * b)
        return dict(bytes=int(moved), flops=int(2 * entries * nk))
    nk = 3 * c["hidden"] * c["inter"]
    moved = hit * nk * 9 / 16 + 2 * c["tokens"] * c["hidden"] * b + c["tokens"] * c["topk"] * 8
    return dict(bytes=int(moved), flops=int(2 * entries * nk))


# ---- the definitions in binary64 ----------------------------------------------

def _matrix64(w, e):
    """Matrix e of the weights in binary64, from the code and scale bytes."""
    c = w["codes"][e].to(torch.int64)
    c = torch.stack((c % 16, c // 16), dim=2).reshape(c.shape[0], -1)
    m, sign = c % 8, 1.0 - 2.0 * (c // 8).double()
    mag = torch.where(m < 2, 0.5 * m.double(),
                      (1.0 + 0.5 * (m % 2).double()) * torch.pow(2.0, (m // 2 - 1).double()))
    b = w["scales"][e].to(torch.int64)
    ex, fr = b // 8, (b % 8).double()
    sb = torch.where(ex == 0, fr * 2.0 ** -9, (1.0 + fr / 8) * torch.pow(2.0, (ex - 7).double()))
    return sign * mag * sb.repeat_interleave(16, dim=1) * w["outer"][e].double()


def _experts64(s, c, one):
    """one(e, tokens, slots) for every expert some entry names, scattered into
    a [T, k, n] result; entries not routed stay zero."""
    out = None
    for e in range(c["experts"]):
        t, j = torch.nonzero(s["idx"] == e, as_tuple=True)
        if t.numel() == 0:
            continue
        y = one(e, t, j)
        if out is None:
            out = torch.zeros((*s["idx"].shape, y.shape[1]), dtype=torch.float64, device="cuda")
        out[t, j] = y
    return out


def exact(case, seed):
    s, c, op = prepare(case, seed), case, case["op"]
    if op in ("router", "router_backward"):
        z = s["logits"].double()
        if op == "router":
            key = s["logits"].float()
            key = (key if s["bias"] is None else key + s["bias"]).double()
            # descending key, ascending index among equals
            at = torch.argsort(-key, dim=1, stable=True)[:, :c["topk"]]
            ok = key.gather(1, at) > -math.inf
        else:
            at, ok = s["idx"].long().clamp(min=0), s["idx"] >= 0
        sel = z.gather(1, at)
        top = sel.masked_fill(~ok, -math.inf).amax(1, keepdim=True).clamp(min=-1e300)
        if c["score"] == 0:
            # the shift cancels in every quotient
            top = z.amax(1, keepdim=True).clamp(min=-1e300) if not c["renorm"] else top
            up = torch.exp(sel - top) * ok
            total = up.sum(1, keepdim=True) if c["renorm"] else torch.exp(z - top).sum(1, keepdim=True)
            p = up / total.clamp(min=1e-300)
        else:
            up = ok / (1.0 + torch.exp(-sel.clamp(min=-700.0)))
            p = up / up.sum(1, keepdim=True).clamp(min=1e-300) if c["renorm"] else up
        if op == "router":
            return torch.where(ok, at, torch.full_like(at, -1)).to(torch.int32), p
        dp = s["dprob"].double() * ok
        mean = (p * dp).sum(1, keepdim=True)
        dz = torch.zeros_like(z)
        if c["score"] == 0 and not c["renorm"]:
            dz = -torch.exp(z - top) / torch.exp(z - top).sum(1, keepdim=True).clamp(min=1e-300) * mean
            dl = p * dp
        elif c["score"] == 0:
            dl = p * (dp - mean)
        else:
            slope = 1.0 / (1.0 + torch.exp(sel.clamp(min=-700.0)))
            dl = p * (dp - mean) * slope if c["renorm"] else p * dp * slope
        return dz.scatter_add_(1, at, torch.where(ok, dl, torch.zeros_like(dl)))
    if op in ("matvec", "expert_matvec", "decode"):
        x = s["x"].double()
        if op == "matvec":
            return torch.matmul(x, _matrix64(s["w"], 0).t().contiguous())
        if op == "expert_matvec":
            y = _experts64(s, c, lambda e, t, j: torch.matmul(x[t], _matrix64(s["w"], e).t().contiguous()))
            return y if y is not None else torch.zeros((c["tokens"], c["topk"], c["n"]),
                                                       dtype=torch.float64, device="cuda")

        def layer(e, t, j):
            h = torch.matmul(x[t], _matrix64(s["w1"], e).t().contiguous())
            g, u = h[:, :c["inter"]], h[:, c["inter"]:]
            d = g / (1.0 + torch.exp(-g)) * u * s["prob"][t, j].double().unsqueeze(1)
            return torch.matmul(d, _matrix64(s["w2"], e).t().contiguous())

        y = _experts64(s, c, layer)
        return y.sum(1) if y is not None else torch.zeros_like(x)
    if c["tokens"] * c["topk"] * c["hidden"] > 1 << 30:
        return None
    dst = s["dst_row"].long()
    t, j = torch.nonzero(dst >= 0, as_tuple=True)
    r = dst[t, j]
    if op in ("sort", "unsort_backward"):
        rows = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        rows[r] = s["tok"].double()[t]
        dprob = None
        if s["prob"] is not None:
            rows[r] *= s["prob"].double()[t, j].unsqueeze(1)
            if op == "unsort_backward":
                dprob = torch.zeros(dst.shape, dtype=torch.float64, device="cuda")
                dprob[t, j] = torch.linalg.vecdot(s["rows"].double()[r], s["tok"].double()[t])
        return rows if op == "sort" else (rows, dprob)
    vals = s["rows"].double()[r]
    dprob = None
    if c["weighted"]:
        if op == "sort_backward":
            dprob = torch.zeros(dst.shape, dtype=torch.float64, device="cuda")
            dprob[t, j] = torch.linalg.vecdot(vals, s["tok"].double()[t])
        vals = vals * s["prob"].double()[t, j].unsqueeze(1)
    y = torch.zeros((c["tokens"], c["hidden"]), dtype=torch.float64, device="cuda")
    y.index_add_(0, t, vals)
    return y if op == "unsort" else (y, dprob)
