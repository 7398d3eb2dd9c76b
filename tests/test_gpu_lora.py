"""lora_forward, lora_backward and nvfp4_lora_matvec against binary64.

Tolerances, with u = 2^-24 and |.| sums of magnitudes: h is a binary32 sum of K
products, (K + 16) u |a||x|.  y adds R products of h to base: (K + R + 24) u
(|base| + c |b||a||x|), then the output type's half step.  nvfp4_lora_matvec
adds the projection's (K + 16) u |w||x|, inside the same bound on the joined
magnitudes.  The way back alike: g as h with N products, dx as y; da sums T
products of g and x, (N + T + 40) u |g||x|, db T products of dy and c h,
(T + 24) u c |dy||h| (with h computed again, K + 16 more)."""
import pytest
import torch

import adapter_ref as A
import operator_ref as R
from gpu_util import say

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
INF = float("inf")


def make(T, K, N, rank, S, kind, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed + T + K + N + rank)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return dict(x=n(T, K).to(dtype), a=(n(S, rank, K) * K ** -0.5).to(dtype), b=n(S, N, rank).to(dtype),
                ids=A.make_ids(gen, T, S, kind), scale=torch.rand(S, generator=gen) * 3 - 0.5,
                base=n(T, N).to(dtype), dy=n(T, N).to(dtype), dbase=n(T, K).to(dtype))


def check(got, ref, lim, what):
    bad = R.outside(got, ref, lim)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside"


def cuda(c, *names):
    return [c[n].cuda() if isinstance(c[n], torch.Tensor) else c[n] for n in names]


SHAPES = [
    # T, K, N, rank, S, ids
    (1, 1, 1, 1, 1, "one"), (1, 16, 5, 3, 2, "random"), (1, 2048, 640, 16, 4, "random"),
    (2, 33, 17, 16, 1, "one"), (5, 129, 300, 17, 3, "wild"), (17, 1000, 257, 9, 5, "random"),
    (64, 512, 1024, 32, 40, "random"), (65, 100, 64, 33, 2, "runs"), (256, 256, 256, 16, 3, "runs"),
    (256, 72, 40, 8, 1, "one"), (255, 4100, 31, 4, 300, "random"), (257, 264, 520, 16, 4, "runs"),
    (300, 777, 511, 24, 6, "wild"), (512, 64, 96, 64, 2, "random"), (700, 130, 258, 100, 3, "runs"),
    (333, 96, 64, 256, 2, "runs"), (40, 96, 65, 256, 4, "random"), (1030, 48, 56, 5, 9, "none"),
    (1500, 320, 192, 12, 1, "one"), (2100, 40, 24, 2, 1000, "random"),
    # several chunks of every adapter, of some; whole pieces and 32 ranks, 64, 128
    (3000, 24, 40, 6, 20, "random"), (900, 64, 128, 32, 9, "runs"), (2050, 128, 256, 64, 5, "runs"),
    (600, 256, 512, 128, 3, "runs")]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,K,N,rank,S,kind", SHAPES)
def test_forward(T, K, N, rank, S, kind, dtype):
    from nvfp4_w4a4_quantized_amd import ops
    c = make(T, K, N, rank, S, kind, dtype)
    x, a, b, ids, scale, base = cuda(c, "x", "a", "b", "ids", "scale", "base")
    lim = (K + rank + 24) * A.ULP
    y, ym, h, hm = A.forward(c["x"], c["a"], c["b"], c["ids"], c["scale"], c["base"])
    say("lora_forward", T, K, N, rank, S, kind, dtype)
    got, gh = ops.lora_forward(x, a, b, ids, scale=scale, base=base, return_h=True)
    check(got, y, lim * ym, "with base")
    check(gh, h, (K + 16) * A.ULP * hm, "h")
    y, ym, _, _ = A.forward(c["x"], c["a"], c["b"], c["ids"], None, None)
    check(ops.lora_forward(x, a, b, ids, out_dtype=torch.float32), y, lim * ym, "plain, binary32 out")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,K,N,rank,S,kind", SHAPES)
def test_backward(T, K, N, rank, S, kind, dtype):
    from nvfp4_w4a4_quantized_amd import ops
    c = make(T, K, N, rank, S, kind, dtype, 1)
    dy, x, a, b, ids, scale, base = cuda(c, "dy", "x", "a", "b", "ids", "scale", "dbase")
    h = A.forward(c["x"], c["a"], c["b"], c["ids"], None, None)[2].float()
    say("lora_backward", T, K, N, rank, S, kind, dtype)
    for given, sc, bs, more in ((h, c["scale"], c["dbase"], 0), (None, None, None, K + 16)):
        (dx, dxm), (da, dam), (db, dbm) = A.backward(c["dy"], c["x"], c["a"], c["b"], c["ids"], sc, h, bs)
        if given is None:
            # h computed again: its error goes by the magnitudes under it
            hm = A.forward(c["x"], c["a"], c["b"], c["ids"], None, None)[3]
            dbm = A.backward(c["dy"], c["x"], c["a"], c["b"], c["ids"], sc, hm, bs)[2][1]
        got = ops.lora_backward(dy, x, a, b, ids, scale=scale if sc is not None else None,
                                h=None if given is None else h.cuda(),
                                base=base if bs is not None else None)
        check(got[0], dx, (N + rank + 24) * A.ULP * dxm, "dx")
        check(got[1], da, (N + T + 40) * A.ULP * dam, "da")
        check(got[2], db, (T + 24 + more) * A.ULP * dbm, "db")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,K,N,rank,S,kind,tiled", [
    (1, 16, 1, 1, 1, "one", False), (1, 256, 96, 16, 4, "random", True), (1, 2048, 5120, 16, 8, "random", True),
    (3, 112, 33, 9, 2, "wild", False), (16, 640, 160, 64, 5, "random", True),
    (7, 1040, 1001, 9, 3, "random", False), (64, 1040, 257, 32, 64, "random", False),
    (64, 256, 32800, 16, 10, "random", True), (8, 384, 24576, 5, 2, "none", True),
    (300, 256, 64, 16, 3, "runs", True), (33, 48, 70, 200, 2, "random", False)])
def test_matvec(T, K, N, rank, S, kind, tiled, dtype):
    import numpy as np
    from nvfp4_w4a4_quantized_amd import ops
    codes, scales, gs = R.make_weights(np.random.default_rng(T + K + N), 1, N, K)
    w = ops.NvFp4Weights(codes.cuda(), scales.cuda(), gs.cuda())
    w = w.packed() if tiled else w
    c = make(T, K, N, rank, S, kind, dtype, 2)
    y, ym, _, _ = A.forward(c["x"], c["a"], c["b"], c["ids"], c["scale"], None, R.decode(codes, scales, gs)[0])
    for out in {dtype, torch.float32}:
        say("nvfp4_lora_matvec", T, K, N, rank, S, kind, tiled, dtype, out)
        got = ops.nvfp4_lora_matvec(*cuda(c, "x"), w, *cuda(c, "a", "b", "ids"), scale=c["scale"].cuda(),
                                    out_dtype=out)
        check(got, y, (K + rank + 40) * A.ULP * ym, f"{dtype} -> {out}")


def test_tokens_without_an_adapter_keep_their_rows():
    """Ids that are no adapter, near and far: the base's bits, or zeros."""
    from nvfp4_w4a4_quantized_amd import ops
    for T in (3, 400):
        c = make(T, 100, 70, 8, 2, "none", torch.bfloat16)
        x, a, b, base = cuda(c, "x", "a", "b", "base")
        ids = torch.tensor([-1, 2, 2 ** 31 - 1, -2 ** 31] * 100, dtype=torch.int32)[:T].cuda()
        y, h = ops.lora_forward(x, a, b, ids, base=base, return_h=True)
        assert torch.equal(y, base) and not bool(h.any())
        assert not bool(ops.lora_forward(x, a, b, ids).any())
        dx, da, db = ops.lora_backward(base, x, a, b, ids, base=x)
        assert torch.equal(dx, x) and not bool(da.any()) and not bool(db.any())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [6, 330])
def test_infinities_and_nan_stay_with_their_token(T, dtype):
    """A token's infinity or NaN reaches its own rows and its adapter's
    gradients alone; one in an adapter nobody uses reaches nothing."""
    from nvfp4_w4a4_quantized_amd import ops
    K, N, rank, S = 70, 90, 5, 4
    c = make(T, K, N, rank, S, "runs", dtype, 3)
    c["ids"] = (torch.arange(T) * 3 // T).to(torch.int32)       # adapters 0, 1, 2; 3 is idle
    c["ids"][1] = -1
    c["a"][3], c["b"][3] = float("nan"), INF
    c["x"][0, 7], c["x"][1, 3], c["dy"][0, 11], c["dy"][1, 2] = INF, float("nan"), float("nan"), INF
    c["a"], c["b"] = c["a"].abs() + 0.01, c["b"].abs() + 0.01   # (no 0 * inf, no inf - inf)
    x, a, b, ids, base, dy = cuda(c, "x", "a", "b", "ids", "base", "dy")
    y, h = ops.lora_forward(x, a, b, ids, base=base, return_h=True)
    assert bool((y[0] == INF).all()) and bool((h[0] == INF).all())
    assert torch.equal(y[1], base[1]) and not bool(h[1].any())
    assert bool(torch.isfinite(y[2:]).all())
    dx, da, db = ops.lora_backward(dy, x, a, b, ids, h=h)
    assert bool(torch.isnan(dx[0]).all()) and not bool(dx[1].any()) and bool(torch.isfinite(dx[2:]).all())
    assert bool(torch.isnan(da[0]).all()) and bool(torch.isnan(db[0, 11]).all())
    assert bool(torch.isfinite(da[1:]).all()) and bool(torch.isfinite(db[1:]).all())
    assert not bool(da[3].any()) and not bool(db[3].any())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rank", [8, 48])
@pytest.mark.parametrize("T", [12, 400])
def test_a_broken_adapter_reaches_its_own_tokens_alone(T, rank, dtype):
    """An adapter full of NaN and infinities beside others, token by token."""
    from nvfp4_w4a4_quantized_amd import ops
    K, N, S = 72, 128, 3
    c = make(T, K, N, rank, S, "random", dtype, 7)
    c["ids"] = (torch.arange(T) % 4 - 1).to(torch.int32)
    x, a, b, ids, base, dy = cuda(c, "x", "a", "b", "ids", "base", "dy")
    want, h = ops.lora_forward(x, a, b, ids, base=base, return_h=True)
    back = ops.lora_backward(dy, x, a, b, ids, h=h)
    a[1], b[1] = float("nan"), INF
    own = (ids == 1)
    y, h2 = ops.lora_forward(x, a, b, ids, base=base, return_h=True)
    assert torch.equal(y[~own], want[~own]) and torch.equal(h2[~own], h[~own])
    assert not bool(torch.isfinite(y[own]).any())
    dx, da, db = ops.lora_backward(dy, x, a, b, ids, h=h)
    assert torch.equal(dx[~own], back[0][~own]) and not bool(torch.isfinite(dx[own]).any())
    for s in (0, 2):
        assert torch.equal(da[s], back[1][s]) and torch.equal(db[s], back[2][s])


def spread(t, left, right):
    """The same rows inside wider ones full of NaN, at an odd offset."""
    wide = torch.full((t.shape[0], left + t.shape[1] + right), float("nan"), dtype=t.dtype, device="cuda")
    wide[:, left:left + t.shape[1]] = t
    return wide[:, left:left + t.shape[1]]


def shifted(t):
    """A dense copy that starts one element behind an aligned address."""
    flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    out = flat[1:].view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,K,N,rank", [(9, 131, 77, 7), (290, 131, 77, 7), (290, 128, 64, 16)])
def test_strided_rows_odd_addresses_and_in_place(T, K, N, rank, dtype):
    from nvfp4_w4a4_quantized_amd import ops
    c = make(T, K, N, rank, 3, "runs", dtype, 4)
    x, a, b, ids, scale, base, dy, dbase = cuda(c, "x", "a", "b", "ids", "scale", "base", "dy", "dbase")
    want, h = ops.lora_forward(x, a, b, ids, scale=scale, base=base, return_h=True)
    back = ops.lora_backward(dy, x, a, b, ids, scale=scale, h=h, base=dbase)
    sx, sa, sb, sid = spread(x, 3, 2), shifted(a), shifted(b), shifted(ids)
    got = ops.lora_forward(sx, sa, sb, sid, scale=shifted(scale), base=spread(base, 1, 4),
                           out=shifted(base))
    assert torch.equal(got, want)
    inplace = shifted(base)
    assert ops.lora_forward(x, a, b, ids, scale=scale, base=inplace, out=inplace) is inplace
    assert torch.equal(inplace, want)
    again = ops.lora_backward(spread(dy, 5, 1), sx, sa, sb, sid, scale=scale, h=shifted(h),
                              base=spread(dbase, 1, 2))
    for p, q in zip(again, back):
        assert torch.equal(p, q)
    dx = dbase.clone()
    assert torch.equal(ops.lora_backward(dy, x, a, b, ids, scale=scale, h=h, base=dx, out=dx)[0], back[0])
    assert torch.equal(dx, back[0])


def test_no_tokens():
    from nvfp4_w4a4_quantized_amd import ops
    c = make(0, 20, 30, 4, 2, "none", torch.bfloat16)
    x, a, b, ids, dy = cuda(c, "x", "a", "b", "ids", "dy")
    assert ops.lora_forward(x, a, b, ids).shape == (0, 30)
    dx, da, db = ops.lora_backward(dy, x, a, b, ids)
    assert dx.shape == (0, 20) and not bool(da.any()) and not bool(db.any())


def test_rows_far_apart():
    """Row offsets past 31 bits of elements."""
    from nvfp4_w4a4_quantized_amd import ops
    T, K, N, ld = 66, 40, 24, 1 << 25
    c = make(T, K, N, 4, 2, "runs", torch.bfloat16, 5)
    x, a, b, ids, dy = cuda(c, "x", "a", "b", "ids", "dy")
    far = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda").view(T, ld)
    far[:, :K], far[:, 64:64 + N] = x, dy
    want, back = ops.lora_forward(x, a, b, ids), ops.lora_backward(dy, x, a, b, ids)
    assert torch.equal(ops.lora_forward(far[:, :K], a, b, ids), want)
    for p, q in zip(ops.lora_backward(far[:, 64:64 + N], far[:, :K], a, b, ids), back):
        assert torch.equal(p, q)


def test_a_dirty_workspace_changes_nothing():
    from nvfp4_w4a4_quantized_amd import ops
    c = make(400, 90, 50, 6, 3, "runs", torch.bfloat16, 6)
    x, a, b, ids, dy = cuda(c, "x", "a", "b", "ids", "dy")
    want, back = ops.lora_forward(x, a, b, ids), ops.lora_backward(dy, x, a, b, ids)
    n = ops.lora_backward_workspace_size(torch.bfloat16, 400, 90, 50, 3, 6)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    for p, q in zip(ops.lora_backward(dy, x, a, b, ids, workspace=ws), back):
        assert torch.equal(p, q)
    n = ops.lora_forward_workspace_size(400, 90, 6)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(ops.lora_forward(x, a, b, ids, workspace=ws), want)
