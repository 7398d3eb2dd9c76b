"""Plain binary64 definitions of the low-rank adapters, on the CPU, for the
tests, with the magnitudes that the error bounds go by."""
import torch

ULP = 2.0 ** -24


def picks(ids, adapters):
    """Every token's adapter as a row of zeros with at most a one."""
    return (ids.long().unsqueeze(1) == torch.arange(adapters)).double()


def forward(x, a, b, ids, scale, base, w=None):
    """(y, |y|'s bound, h, |h|'s bound): sums of the values and of their
    magnitudes; a token's own adapter alone enters its row."""
    T, S, R, N = x.shape[0], a.shape[0], a.shape[1], b.shape[1]
    h, hm = torch.zeros(T, R, dtype=torch.float64), torch.zeros(T, R, dtype=torch.float64)
    y = torch.zeros(T, N, dtype=torch.float64) if base is None else base.double().clone()
    ym = y.abs()
    if w is not None:
        y, ym = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    for s in range(S):
        at = torch.nonzero(ids == s).view(-1)
        if at.numel() == 0:
            continue
        c = 1.0 if scale is None else float(scale[s])
        xs, A, B = x[at].double(), a[s].double(), b[s].double()
        h[at], hm[at] = xs @ A.t(), xs.abs() @ A.abs().t()
        y[at] += c * (h[at] @ B.t())
        ym[at] += abs(c) * (hm[at] @ B.abs().t())
    return y, ym, h, hm


def backward(dy, x, a, b, ids, scale, h, base):
    """((dx, bound), (da, bound), (db, bound)) with h the forward's."""
    S = a.shape[0]
    dx = torch.zeros(x.shape, dtype=torch.float64) if base is None else base.double().clone()
    dxm = dx.abs()
    da, db = torch.zeros(a.shape, dtype=torch.float64), torch.zeros(b.shape, dtype=torch.float64)
    dam, dbm = da.clone(), db.clone()
    for s in range(S):
        at = torch.nonzero(ids == s).view(-1)
        if at.numel() == 0:
            continue
        c = 1.0 if scale is None else float(scale[s])
        d, xs, A, B = dy[at].double(), x[at].double(), a[s].double(), b[s].double()
        g, gm = c * (d @ B), abs(c) * (d.abs() @ B.abs())
        dx[at] += g @ A
        dxm[at] += gm @ A.abs()
        da[s], dam[s] = g.t() @ xs, gm.t() @ xs.abs()
        db[s], dbm[s] = c * (d.t() @ h[at].double()), abs(c) * (d.abs().t() @ h[at].double().abs())
    return (dx, dxm), (da, dam), (db, dbm)


def make_ids(gen, T, S, kind):
    """Adapters of T tokens: 'runs' of requests, 'random', 'one', 'none', or
    'wild' ids far outside."""
    if kind == "none":
        return torch.full((T,), -1, dtype=torch.int32)
    if kind == "one":
        return torch.full((T,), S - 1, dtype=torch.int32)
    ids = torch.randint(0, S, (T,), generator=gen)
    if kind == "runs":
        ids = ids[torch.cumsum((torch.rand(T, generator=gen) < 0.05).long(), 0).clamp(max=T - 1)]
        ids = torch.where(ids == S // 2, torch.full_like(ids, -1), ids)
    if kind == "wild":
        out = torch.tensor([-1, S, S + 1, 2 ** 31 - 1, -2 ** 31, -5])
        ids = torch.where(torch.rand(T, generator=gen) < 0.4,
                          out[torch.randint(0, 6, (T,), generator=gen)], ids)
    return ids.to(torch.int32)


def newton_schulz(g, steps, coefficients, eps, scale=1.0):
    """The orthogonalised update, from the definition, on g's device."""
    a, b, c = coefficients
    x = g.double()
    tall = x.shape[-2] > x.shape[-1]
    x = x / (x.square().sum(dim=(-2, -1), keepdim=True).sqrt() + eps)
    for _ in range(steps):
        xt = x.transpose(-2, -1).contiguous()
        if tall:
            s = torch.matmul(xt, x)
            x = a * x + torch.matmul(x, b * s + c * torch.matmul(s, s))
        else:
            s = torch.matmul(x, xt)
            x = a * x + torch.matmul(b * s + c * torch.matmul(s, s), x)
    return scale * x
