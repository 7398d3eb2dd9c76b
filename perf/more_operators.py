"""Measured cases of the operators that train beside frozen NVFP4 weights:
low-rank adapters of many requests beside a shared NVFP4 projection (a few new
tokens), the same adapters on long batches with their gradients, and the
orthogonalised update of a weight's gradient by Newton-Schulz products.

A case names an operator and its sizes.  prepare() makes what a program holds
before the call; run() makes one call, either of the package's entry points
(own) or in plain torch operations in binary32; exact() is the definition in
binary64.  Sizes follow the Qwen3-30B-A3B-shaped layer of workloads.py (hidden
2048, QKV projection 5120 wide, 128 experts of intermediate 768); the odd ones
are generic.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
# E2M1 values of the codes 0..7 (bit 3 is the sign)
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# the quintic's coefficients of the usual orthogonalised update
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


def listed():
    return [
        # the QKV projection of one new token with its request's adapter: pure latency
        dict(name="lora_matvec_t1_qkv", op="lora_matvec", tokens=1, n=5120, k=2048, rank=16,
             adapters=8, bare=0.0, tiled=True, dtype="bf16"),
        # 64 requests' new tokens at a large projection, nearly every one with its own adapter
        dict(name="lora_matvec_t64_n16384", op="lora_matvec", tokens=64, n=16384, k=4096, rank=32,
             adapters=64, bare=0.1, tiled=False, dtype="bf16"),
        # sizes that no tile divides, some requests without an adapter
        dict(name="lora_matvec_t7_odd", op="lora_matvec", tokens=7, n=1001, k=1040, rank=9,
             adapters=3, bare=0.3, tiled=False, dtype="fp32"),
        # prompts of 24 requests on their adapters, added to the projection's output
        dict(name="lora_forward_t4096", op="lora_forward", tokens=4096, n=5120, k=2048, rank=16,
             adapters=16, requests=24, bare=0.1, base=True, train=False, dtype="bf16"),
        # odd widths and rank, in training (a x is kept for the way back)
        dict(name="lora_forward_t1003_odd", op="lora_forward", tokens=1003, n=1111, k=1999, rank=24,
             adapters=5, requests=11, bare=0.2, base=False, train=True, dtype="fp16"),
        # gradients of a training batch that holds four adapters' sequences
        dict(name="lora_backward_t8192", op="lora_backward", tokens=8192, n=5120, k=2048, rank=16,
             adapters=4, requests=16, bare=0.0, base=True, dtype="bf16"),
        # one adapter of a large rank on a long batch
        dict(name="lora_backward_t32768_r64", op="lora_backward", tokens=32768, n=5120, k=2048,
             rank=64, adapters=1, requests=8, bare=0.0, base=True, dtype="bf16"),
        # odd sizes in binary32, some tokens without an adapter, one adapter without tokens
        dict(name="lora_backward_t517_odd", op="lora_backward", tokens=517, n=1111, k=777, rank=9,
             adapters=6, requests=7, bare=0.2, base=False, dtype="fp32"),
        # the update of 64 adapters' down projections
        dict(name="newton_schulz_e64_16x2048", op="newton_schulz", batch=64, rows=16, cols=2048,
             signal=16, dtype="fp32", out="fp32", steps=5),
        # odd sizes, every digit of binary32 kept
        dict(name="newton_schulz_e4_1000x2047", op="newton_schulz", batch=4, rows=1000, cols=2047,
             signal=300, dtype="fp32", out="fp32", steps=5),
        # one dense projection's update in bf16
        dict(name="newton_schulz_5120x2048", op="newton_schulz", batch=1, rows=5120, cols=2048,
             signal=512, dtype="bf16", out="bf16", steps=5),
        # the update of every expert's down projection from its binary32 gradient
        dict(name="newton_schulz_e128_2048x768", op="newton_schulz", batch=128, rows=2048, cols=768,
             signal=256, dtype="fp32", out="bf16", steps=5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the listed ones' ranges."""
    op = rng.choice(["lora_matvec", "lora_forward", "lora_backward", "newton_schulz"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    rank = rng.choice([4, 8, 16, 16, 32, 64, rng.randint(1, 64)])
    bare = rng.choice([0.0, 0.0, 0.2])
    if op == "lora_matvec":
        tiled = rng.random() < 0.5
        n, k = _log(rng, 32, 16384), _log(rng, 64, 4096)
        n, k = ((n + 31) // 32 * 32, (k + 127) // 128 * 128) if tiled else (n, (k + 15) // 16 * 16)
        return dict(op=op, tokens=_log(rng, 1, 64), n=n, k=k, rank=rank, adapters=_log(rng, 1, 64),
                    bare=bare, tiled=tiled, dtype=dtype)
    if op in ("lora_forward", "lora_backward"):
        n, k = _log(rng, 64, 5120), _log(rng, 64, 5120)
        if rng.random() < 0.6:
            n, k = (n + 7) // 8 * 8, (k + 7) // 8 * 8
        tokens = min(_log(rng, 1, 32768), (1 << 27) // (n + k))
        c = dict(op=op, tokens=tokens, n=n, k=k, rank=rank,
                 adapters=_log(rng, 1, 32), requests=min(tokens, _log(rng, 1, 64)), bare=bare,
                 base=rng.random() < 0.7, dtype=dtype)
        if op == "lora_forward":
            c["train"] = rng.random() < 0.5
        return c
    rows, cols = _log(rng, 8, 4096), _log(rng, 8, 4096)
    if rng.random() < 0.6:
        rows, cols = (rows + 7) // 8 * 8, (cols + 7) // 8 * 8
    one = _products(rows, cols, 5)
    batch = max(1, min(_log(rng, 1, 128), int(2.5e12 / one)))
    return dict(op=op, batch=batch, rows=rows, cols=cols, signal=max(1, min(rows, cols) // rng.choice([1, 2, 4])),
                dtype=dtype, out=rng.choice([dtype, "bf16"]), steps=5)


# ---- inputs ----------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std


def _weights(g, n, k, tiled):
    """One NVFP4 weight matrix of N(0, 0.02) values: codes, E4M3 block scales
    and an outer scale, row-major and, if asked, in the tiled layout."""
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    w = _normal(g, n, k // 16, 16, std=0.02)
    outer = (w.abs().amax() / 2688.0).reshape(1)
    s8 = (w.abs().amax(dim=2) / (6.0 * outer)).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = (s8.float() * outer).unsqueeze(-1)
    q = torch.bucketize(w.abs() / d.clamp(min=1e-30), edges).to(torch.uint8)
    q = (q | ((w < 0).to(torch.uint8) << 3)).view(n, k // 2, 2)
    codes, scales = (q[..., 0] | (q[..., 1] << 4)).contiguous(), s8.view(torch.uint8)
    held = (codes, scales)
    if tiled:
        t = codes.view(n // 32, 32, k // 128, 2, 2, 16).permute(0, 2, 4, 3, 1, 5)
        s = scales.view(n // 32, 32, k // 128, 2, 4).permute(0, 2, 3, 1, 4)
        held = (t.contiguous().view(codes.shape), s.contiguous().view(scales.shape))
    return dict(codes=codes, scales=scales, outer=outer, layout=int(tiled), as_held=held)


def _adapter_of(g, c):
    """Every token's adapter: one a token, or one a request of consecutive
    tokens; -1 for a share of them that has none."""
    t, of = c["tokens"], c.get("requests", c["tokens"])
    ids = torch.randint(0, c["adapters"], (of,), generator=g, device="cuda")
    if c["bare"]:               # (the first one has an adapter)
        gone = torch.rand(of, generator=g, device="cuda") < c["bare"]
        gone[0] = False
        ids = torch.where(gone, -torch.ones_like(ids), ids)
    if "requests" in c:
        if c["adapters"] > 4:       # an adapter that no token uses
            ids = torch.where(ids == 3, torch.full_like(ids, 2), ids)
        start = torch.zeros(t, dtype=torch.long, device="cuda")
        start[torch.randint(0, t, (of - 1,), generator=g, device="cuda")] = 1
        start[0] = 0
        ids = ids[torch.cumsum(start, 0)]
    return ids.to(torch.int32).contiguous()


def _gradients(g, c):
    """Gradients as training gives them: a few strong directions (a product of
    `signal` directions of falling weight) over a floor of noise."""
    fall = torch.arange(1, c["signal"] + 1, device="cuda", dtype=torch.float32).rsqrt()
    left = _normal(g, c["batch"], c["rows"], c["signal"]) * fall
    x = torch.bmm(left, _normal(g, c["batch"], c["signal"], c["cols"]))
    x = x / math.sqrt(c["signal"]) + _normal(g, *x.shape, std=0.3)
    return x * 1e-3


def prepare(case, seed):
    g, c, op = _gen(seed), case, case["op"]
    t = DTYPES[c["dtype"]]
    s = dict(case=case)
    if op == "newton_schulz":
        s["g"] = _gradients(g, c).to(t)
        return s
    s["x"] = _normal(g, c["tokens"], c["k"]).to(t)
    s["a"] = _normal(g, c["adapters"], c["rank"], c["k"], std=c["k"] ** -0.5).to(t)
    s["b"] = _normal(g, c["adapters"], c["n"], c["rank"], std=0.1).to(t)
    # alpha / rank of every adapter
    s["scale"] = torch.rand(c["adapters"], generator=g, device="cuda") * 3.0 + 0.5
    s["ids"] = _adapter_of(g, c)
    if op == "lora_matvec":
        s["w"] = _weights(g, c["n"], c["k"], c["tiled"])
        return s
    if op == "lora_forward":
        s["base"] = _normal(g, c["tokens"], c["n"]).to(t) if c["base"] else None
        return s
    s["dy"] = _normal(g, c["tokens"], c["n"], std=0.1).to(t)
    s["base"] = _normal(g, c["tokens"], c["k"], std=0.1).to(t) if c["base"] else None
    s["h"] = _down(s["x"], s["a"], s["ids"]).view(c["tokens"], c["adapters"], c["rank"]).sum(1)
    return s


# ---- one call ----------------------------------------------------------------

def run(state):
    return (_own if own else _plain)(state, state["case"])


def _own(s, c):
    from nvfp4_w4a4_quantized_amd import ops
    op = c["op"]
    if op == "lora_matvec":
        w = ops.NvFp4Weights(*(v.unsqueeze(0) for v in s["w"]["as_held"]), s["w"]["outer"],
                             layout=s["w"]["layout"])
        return ops.nvfp4_lora_matvec(s["x"], w, s["a"], s["b"], s["ids"], scale=s["scale"])
    if op == "lora_forward":
        if c["train"]:
            return ops.lora_forward(s["x"], s["a"], s["b"], s["ids"], scale=s["scale"],
                                    base=s["base"], return_h=True)
        return ops.lora_forward(s["x"], s["a"], s["b"], s["ids"], scale=s["scale"], base=s["base"])
    if op == "lora_backward":
        return ops.lora_backward(s["dy"], s["x"], s["a"], s["b"], s["ids"], scale=s["scale"],
                                 h=s["h"], base=s["base"])
    return ops.newton_schulz(s["g"], steps=c["steps"], coefficients=COEFFICIENTS, eps=EPS,
                             out_dtype=DTYPES[c["out"]])


def _mask(ids, adapters, rank):
    """One in the columns of a token's own adapter: [T, adapters * rank]."""
    hot = ids.unsqueeze(1) == torch.arange(adapters, device=ids.device)
    return hot.float().repeat_interleave(rank, dim=1)


def _down(x, a, ids):
    """Every adapter's a x at once, zero but for a token's own: [T, S * R]."""
    adapters, rank, k = a.shape
    h = torch.mm(x.float(), a.float().view(adapters * rank, k).t().contiguous())
    return h * _mask(ids, adapters, rank)


def _up(b):
    """The adapters' b under each other: [S * R, N]."""
    return b.float().permute(0, 2, 1).reshape(-1, b.shape[1]).contiguous()


def _plain(s, c):
    op = c["op"]
    t = DTYPES[c["dtype"]]
    if op == "newton_schulz":
        x = s["g"].float()
        tall = c["rows"] > c["cols"]
        if tall:
            x = x.transpose(1, 2).contiguous()
        norm = s["g"].double().square().sum(dim=(1, 2), keepdim=True).sqrt()
        x = (x / (norm + EPS)).float()
        a, b, d = COEFFICIENTS
        # a step needs the one before it
        for _ in range(c["steps"]):
            p = torch.bmm(x, x.transpose(1, 2).contiguous())
            x = a * x + torch.bmm(b * p + d * torch.bmm(p, p), x)
        if tall:
            x = x.transpose(1, 2).contiguous()
        return x.to(DTYPES[c["out"]])
    scale = s["scale"].repeat_interleave(c["rank"])
    if op in ("lora_matvec", "lora_forward"):
        h = _down(s["x"], s["a"], s["ids"])
        y = torch.mm(h * scale, _up(s["b"]))
        if op == "lora_matvec":
            grid = torch.tensor(GRID + tuple(-v for v in GRID), device=y.device)
            w = s["w"]
            q = grid[torch.stack((w["codes"] & 15, w["codes"] >> 4), dim=-1).int()]
            q = q.view(*w["scales"].shape, 16) * w["scales"].view(torch.float8_e4m3fn).float().unsqueeze(-1)
            q = (q * w["outer"]).view(c["n"], c["k"])
            return (y + torch.mm(q, s["x"].float().t().contiguous()).t()).to(t).contiguous()
        if c["base"]:
            y = y + s["base"].float()
        if c["train"]:
            return y.to(t), h.view(c["tokens"], c["adapters"], c["rank"]).sum(1)
        return y.to(t)
    dy, x = s["dy"].float(), s["x"].float()
    mask = _mask(s["ids"], c["adapters"], c["rank"])
    up = torch.mm(dy, _up(s["b"]).t().contiguous()) * mask * scale       # the gradient of a x
    h = s["h"].repeat(1, c["adapters"]) * mask * scale
    dx = torch.mm(up, s["a"].float().view(-1, c["k"]))
    if c["base"]:
        dx = dx + s["base"].float()
    da = torch.mm(up.t().contiguous(), x).view(c["adapters"], c["rank"], c["k"])
    db = torch.mm(h.t().contiguous(), dy).view(c["adapters"], c["rank"], c["n"])
    return dx.to(t), da, db.transpose(1, 2).contiguous()


def _products(rows, cols, steps):
    """Operations of the iteration: the products over the short side n, each
    symmetric one half, step by step or, where the other side is much longer,
    on the n x n matrices alone with one product at either end."""
    n, m = min(rows, cols), max(rows, cols)
    return min(steps * (3 * n * n * m + n ** 3), 3 * n * n * m + 4 * steps * n ** 3)


def work(case):
    """Bytes that have to move and operations that have to be done."""
    c, op, b = case, case["op"], SIZE[case["dtype"]]
    if op == "newton_schulz":
        e = c["batch"] * c["rows"] * c["cols"]
        return dict(bytes=e * (b + SIZE[c["out"]]), flops=c["batch"] * _products(c["rows"], c["cols"], c["steps"]))
    t, n, k, r = c["tokens"], c["n"], c["k"], c["rank"]
    live = t * (1.0 - c["bare"])
    # adapters that at least one token uses, on average
    of = c.get("requests", t) * (1.0 - c["bare"])
    used = c["adapters"] * (1.0 - (1.0 - 1.0 / c["adapters"]) ** of)
    flops = 2 * live * r * (n + k)
    moved = used * r * (n + k) * b + 4 * t
    if op == "lora_matvec":
        return dict(bytes=int(moved + n * k * 9 / 16 + t * (n + k) * b), flops=int(flops + 2 * t * n * k))
    if op == "lora_forward":
        moved += live * k * b + t * n * b * (2 if c["base"] else 1) + (4 * t * r if c["train"] else 0)
        return dict(bytes=int(moved), flops=int(flops))
    moved += live * (n + k) * b + t * k * b * (2 if c["base"] else 1) + 4 * live * r
    return dict(bytes=int(moved + 4 * c["adapters"] * r * (n + k)), flops=int(2 * flops))


# ---- the definitions in binary64 ----------------------------------------------

def _matrix64(w):
    """The weight matrix in binary64, from the code and scale bytes."""
    c = w["codes"].to(torch.int64)
    c = torch.stack((c % 16, c // 16), dim=2).reshape(c.shape[0], -1)
    m, sign = c % 8, 1.0 - 2.0 * (c // 8).double()
    mag = torch.where(m < 2, 0.5 * m.double(),
                      (1.0 + 0.5 * (m % 2).double()) * torch.pow(2.0, (m // 2 - 1).double()))
    b = w["scales"].to(torch.int64)
    ex, fr = b // 8, (b % 8).double()
    sb = torch.where(ex == 0, fr * 2.0 ** -9, (1.0 + fr / 8) * torch.pow(2.0, (ex - 7).double()))
    return sign * mag * sb.repeat_interleave(16, dim=1) * w["outer"].double()


def exact(case, seed):
    s, c, op = prepare(case, seed), case, case["op"]
    if op == "newton_schulz":
        out = torch.empty(s["g"].shape, dtype=torch.float64, device="cuda")
        a, b, d = COEFFICIENTS
        for e in range(c["batch"]):
            v = s["g"][e].double()
            v = v / (torch.linalg.matrix_norm(v) + EPS)
            for _ in range(c["steps"]):
                # on the shorter side, from whichever side the matrix has it
                if c["rows"] <= c["cols"]:
                    w = torch.matmul(v, v.t().contiguous())
                    v = a * v + torch.matmul(b * w + d * torch.matmul(w, w), v)
                else:
                    w = torch.matmul(v.t().contiguous(), v)
                    v = a * v + torch.matmul(v, b * w + d * torch.matmul(w, w))
            out[e] = v
        return out
    x = s["x"].double()
    t, n, k = c["tokens"], c["n"], c["k"]
    zeros = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")  # noqa: E731
    if op in ("lora_matvec", "lora_forward"):
        y, h = zeros(t, n), zeros(t, c["rank"])
        if op == "lora_matvec":
            y += torch.matmul(x, _matrix64(s["w"]).t().contiguous())
        elif c["base"]:
            y += s["base"].double()
        for e in range(c["adapters"]):
            at = torch.nonzero(s["ids"] == e).view(-1)
            if at.numel():
                h[at] = torch.matmul(x[at], s["a"][e].double().t().contiguous())
                y[at] += s["scale"][e].double() * torch.matmul(h[at], s["b"][e].double().t().contiguous())
        return (y, h) if op == "lora_forward" and c["train"] else y
    dx = s["base"].double() if c["base"] else zeros(t, k)
    da, db = zeros(*s["a"].shape), zeros(*s["b"].shape)
    for e in range(c["adapters"]):
        at = torch.nonzero(s["ids"] == e).view(-1)
        if at.numel():
            dy = s["dy"][at].double() * s["scale"][e].double()
            up = torch.matmul(dy, s["b"][e].double())
            dx[at] += torch.matmul(up, s["a"][e].double())
            da[e] = torch.matmul(up.t().contiguous(), x[at])
            db[e] = torch.matmul(dy.t().contiguous(), s["h"][at].double())
    return dx, da, db
