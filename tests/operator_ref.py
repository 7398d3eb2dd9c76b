"""Plain binary64 definitions of the operators on unquantized tensors, on the
CPU, for the tests.  They share no code with the kernels: routing through
sorts, products through decoded matrices, gradients from the formulas."""
import numpy as np
import torch

GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# half the distance of the smallest values: what rounding loses below the normal range
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}


def log_sigmoid(z):
    return torch.clamp(z, max=0.0) - torch.log1p(torch.exp(-z.abs()))


def softmax_rows(v):
    """Softmax in binary64; a row of -inf alone gives zeros."""
    m = v.max(dim=1, keepdim=True).values
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    e = torch.exp(v - m)
    s = e.sum(dim=1, keepdim=True)
    return torch.where(s > 0, e / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(e))


def router_ids(logits, topk, bias=None):
    """Descending keys, equal ones by ascending id; -1 where none is left."""
    key = logits.float()
    if bias is not None:
        key = key + bias.float()
    key = torch.where(torch.isnan(key), torch.full_like(key, -np.inf), key).numpy()
    order = np.argsort(-key.astype(np.float64), axis=1, kind="stable")[:, :topk]
    picked = np.take_along_axis(key, order, axis=1)
    return torch.from_numpy(np.where(picked > -np.inf, order, -1).astype(np.int32))


def router_weights(logits, ids, score, renorm, scale=1.0):
    z = logits.double()
    ok = (ids >= 0) & (ids < z.shape[1])
    sel = z.gather(1, ids.clamp(0, z.shape[1] - 1).long())
    if renorm:
        v = sel if score == 0 else log_sigmoid(sel)
        w = softmax_rows(torch.where(ok, v, torch.full_like(v, -np.inf)))
    elif score == 0:
        w = softmax_rows(z).gather(1, ids.clamp(0, z.shape[1] - 1).long())
    else:
        w = torch.exp(log_sigmoid(sel))
    return scale * torch.where(ok, w, torch.zeros_like(w))


def router_gradient(logits, ids, dprob, score, renorm, scale=1.0):
    z = logits.double()
    E = z.shape[1]
    ok = (ids >= 0) & (ids < E)
    at = ids.clamp(0, E - 1).long()
    dw = scale * torch.where(ok, dprob.double(), torch.zeros(ids.shape, dtype=torch.float64))
    q = router_weights(logits, ids, score, renorm)
    mean = (q * dw).sum(1, keepdim=True)
    sel = z.gather(1, at)
    out = torch.zeros_like(z)
    if score == 0 and not renorm:
        out -= softmax_rows(z) * mean
        dl = q * dw
    elif score == 0:
        dl = q * (dw - mean)
    elif renorm:
        dl = q * (dw - mean) * torch.exp(log_sigmoid(-sel))
    else:
        dl = dw * torch.exp(log_sigmoid(sel) + log_sigmoid(-sel))
    return out.scatter_add_(1, at, torch.where(ok, dl, torch.zeros_like(dl)))


def routing(ids, experts, align):
    """dst_row, row_src, offsets and the number of rows, as moe_permute."""
    T, k = ids.shape
    flat = ids.reshape(-1).numpy()
    cap = T * k + experts * (align - 1)
    dst = np.full(T * k, -1, np.int32)
    src = np.full(cap, -1, np.int32)
    offs = np.zeros(experts + 1, np.int32)
    row = 0
    for e in range(experts):
        at = np.flatnonzero(flat == e)
        dst[at] = row + np.arange(at.size)
        src[row:row + at.size] = at // k
        row += -(-at.size // align) * align
        offs[e + 1] = row
    return (torch.from_numpy(dst.reshape(T, k)), torch.from_numpy(src), torch.from_numpy(offs), row)


def decode(codes, scales, gscale):
    """NVFP4 weights [G, N, K] in binary64."""
    c = codes.cpu().numpy()
    c = np.stack((c & 15, c >> 4), axis=-1).reshape(*c.shape[:-1], -1)
    mag = np.array(GRID)[c & 7] * np.where(c & 8, -1.0, 1.0)
    b = scales.cpu().numpy().astype(np.int64)
    ex, fr = b >> 3, (b & 7).astype(np.float64)
    s = np.where(ex == 0, fr * 2.0 ** -9, (1.0 + fr / 8.0) * np.exp2(ex - 7.0))
    w = mag * np.repeat(s, 16, axis=-1)
    return torch.from_numpy(w * gscale.cpu().double().numpy()[:, None, None])


def make_weights(rng, groups, n, k, std=0.02):
    """Random NVFP4 weights as bytes: any code, block scales in the middle of
    the E4M3 range with a few zeros, subnormals and largest ones."""
    codes = torch.from_numpy(rng.integers(0, 256, (groups, n, k // 2), dtype=np.uint8))
    sc = rng.integers(40, 90, (groups, n, k // 16)).astype(np.uint8)
    odd = rng.random(sc.shape)
    sc[odd < 0.02] = 0
    sc[(odd >= 0.02) & (odd < 0.04)] = 3
    sc[(odd >= 0.04) & (odd < 0.05)] = 0x7E
    gs = torch.from_numpy((std / 8 * (0.5 + rng.random(groups))).astype(np.float32))
    return codes, torch.from_numpy(sc), gs


def tile_weights(codes, scales):
    """The documented byte permutation of the tiled layout, element by element."""
    G, n, kh = codes.shape
    c, s = codes.numpy(), scales.numpy()
    t = c.reshape(G, n // 32, 32, kh // 64, 2, 2, 16).transpose(0, 1, 3, 5, 4, 2, 6)
    u = s.reshape(G, n // 32, 32, kh // 64, 2, 4).transpose(0, 1, 3, 4, 2, 5)
    return (torch.from_numpy(np.ascontiguousarray(t).reshape(c.shape)),
            torch.from_numpy(np.ascontiguousarray(u).reshape(s.shape)))


def expert_products(x, ids, w, by_entry=False):
    """[T, k, n] products and the sums of their terms' magnitudes."""
    T, k = ids.shape
    G, n, K = w.shape
    y = torch.zeros((T, k, n), dtype=torch.float64)
    mag = torch.zeros_like(y)
    x = x.double().cpu()
    for e in range(G):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            rows = x.view(T, k, K)[t, j] if by_entry else x[t]
            y[t, j] = rows @ w[e].t()
            mag[t, j] = rows.abs() @ w[e].abs().t()
    return y, mag


def outside(got, ref, lim):
    """Where `got` is not the rounding to its type of a value within `lim` of
    ref.  A binary16 result is infinite exactly from 65520 on (half a step
    above the largest value, 65504), so an infinity of ref's sign is right
    where |ref| + lim reaches that."""
    g = got.cpu().double()
    tol = lim + STEP[got.dtype] * 1.0001 * ref.abs() + TINY[got.dtype]
    bad = ~((g - ref).abs() <= tol)
    if got.dtype == torch.float16:
        bad &= ~(torch.isinf(g) & (g.sign() == ref.sign()) & (ref.abs() + lim >= 65520.0))
    return bad
