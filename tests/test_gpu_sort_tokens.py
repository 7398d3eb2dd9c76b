"""moe_sort_tokens, moe_unsort_tokens and their gradients against binary64.

Tolerances: copies are exact.  A weighted row is one binary32 product rounded
to the type: 2^-24 |v| plus the type's half step.  A token's sum of k
products: 2 k 2^-24 of the sum of magnitudes plus the half step.  A weight's
gradient, a binary32 sum of H products in some order: (H + 2) 2^-24 of the
sum of magnitudes."""
import numpy as np
import pytest
import torch

import operator_ref as R
from gpu_util import say

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def make_case(rng, T, k, E, align, dropped, dtype, H):
    ids = np.stack([rng.choice(E, k, replace=False) for _ in range(T)]) if T else np.zeros((0, k))
    ids = ids.astype(np.int32).reshape(T, k)
    if dropped:
        ids[rng.random((T, k)) < dropped] = -1
        if T > 2:
            ids[T // 2] = -1                # a token with no rows
    ids = torch.from_numpy(ids)
    dst, src, offs, end = R.routing(ids, E, align)
    cap = src.numel()
    t = dict(ids=ids, dst=dst, src=src, offs=offs, end=end, cap=cap,
             x=torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).to(dtype),
             rows=torch.from_numpy(rng.standard_normal((cap, H)).astype(np.float32)).to(dtype),
             prob=torch.from_numpy(rng.random((T, k)).astype(np.float32)))
    # what lies behind the last row and in rows no entry names must not matter
    named = torch.zeros(cap, dtype=torch.bool)
    named[dst[dst >= 0].long()] = True
    t["rows"][~named] = float("nan")
    if dropped:
        t["prob"][ids < 0] = float("nan")
    return t


def sums_ref(c, weighted):
    """y and the sums of magnitudes of its terms."""
    ok = c["dst"] >= 0
    r = c["rows"].double()[c["dst"].clamp(min=0).long()] if c["cap"] else torch.zeros(
        (*c["dst"].shape, c["x"].shape[1]), dtype=torch.float64)
    r = torch.where(ok.unsqueeze(-1), r, torch.zeros_like(r))
    w = torch.where(ok, c["prob"].double(), torch.zeros(c["dst"].shape, dtype=torch.float64))
    v = r * w.unsqueeze(-1) if weighted else r
    return r, v.sum(1), v.abs().sum(1)


def rows_ref(c, weighted):
    t, j = torch.nonzero(c["dst"] >= 0, as_tuple=True)
    out = torch.zeros((c["end"], c["x"].shape[1]), dtype=torch.float64)
    v = c["x"].double()[t]
    out[c["dst"][t, j].long()] = v * c["prob"].double()[t, j].unsqueeze(1) if weighted else v
    return out


def dots_ref(c):
    r, _, _ = sums_ref(c, False)
    p = r * c["x"].double().unsqueeze(1)
    return p.sum(-1), p.abs().sum(-1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,H,align,dropped", [
    (1, 1, 1, 1, 1, 0.0), (1, 8, 128, 2048, 1, 0.0), (5, 2, 3, 7, 16, 0.0), (64, 4, 60, 1111, 16, 0.1),
    (33, 9, 12, 513, 1, 0.2), (70, 20, 24, 64, 128, 0.3), (3, 3, 1000, 40, 2, 0.5),
    (257, 8, 16, 2056, 1, 0.0), (0, 4, 8, 96, 16, 0.0), (10, 17, 40, 4099, 4, 0.1),
    (6, 8, 16, 9000, 1, 0.0), (300, 10, 20, 4100, 16, 0.1)])
def test_sort_and_unsort(T, k, E, H, align, dropped, dtype):
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(T * 31 + H)
    c = make_case(rng, T, k, E, align, dropped, dtype, H)
    d = {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in c.items()}
    if T:
        meta = ops.moe_permute(None, d["ids"], torch.nan_to_num(d["prob"]), E, align=align)
        assert torch.equal(meta["dst_row"], d["dst"]) and torch.equal(meta["offsets"], d["offs"])
        assert torch.equal(meta["row_src"][:c["end"]], d["src"][:c["end"]])
    step, tiny = R.STEP[dtype], R.TINY[dtype]
    for weighted in (False, True):
        say("sort", T, k, E, H, align, dropped, dtype, weighted)
        prob = d["prob"] if weighted else None
        # rows behind the last expert's keep what the buffer held
        out = torch.full((c["cap"], H), 7.0, dtype=dtype, device="cuda")
        rows = ops.moe_sort_tokens(d["x"], d["dst"], d["src"], d["offs"], prob=prob, out=out)
        assert rows is out
        got = rows.cpu().double()
        ref = rows_ref(c, weighted)
        assert bool((got[c["end"]:] == 7.0).all())
        if weighted:
            lim = (step + 2.0 ** -24) * 1.0001 * ref.abs() + tiny
            assert bool(((got[:c["end"]] - ref).abs() <= lim).all())
        else:
            assert torch.equal(got[:c["end"]], ref)
        y = ops.moe_unsort_tokens(d["rows"], d["dst"], prob=prob)
        r, ref, mag = sums_ref(c, weighted)
        lim = 2 * k * 2.0 ** -24 * mag + step * 1.0001 * ref.abs() + tiny
        assert bool(((y.cpu().double() - ref).abs() <= lim).all())
        # gradients: the other movement, and the weights' dot products
        dref, dmag = dots_ref(c)
        dlim = (H + 2) * 2.0 ** -24 * dmag + 2.0 ** -126
        dx, none = ops.moe_sort_tokens_backward(d["rows"], d["dst"], prob=prob)
        assert none is None and torch.equal(dx, y)
        dx, dprob = ops.moe_sort_tokens_backward(d["rows"], d["dst"], x=d["x"], prob=prob)
        assert torch.equal(dx, y)
        assert bool(((dprob.cpu().double() - dref).abs() <= dlim).all())
        out2 = torch.full((c["cap"], H), 7.0, dtype=dtype, device="cuda")
        dr, none = ops.moe_unsort_tokens_backward(d["x"], d["dst"], d["src"], d["offs"], prob=prob,
                                                  out=out2)
        assert none is None and torch.equal(dr, rows)
        dr, dprob2 = ops.moe_unsort_tokens_backward(d["x"], d["dst"], d["src"], d["offs"],
                                                    rows=d["rows"], prob=prob, out=out2)
        assert torch.equal(dr, rows)
        assert bool(((dprob2.cpu().double() - dref).abs() <= dlim).all())
        again = ops.moe_unsort_tokens_backward(d["x"], d["dst"], d["src"], d["offs"],
                                               rows=d["rows"], prob=prob, out=out2)[1]
        assert torch.equal(again, dprob2)


@pytest.mark.parametrize("dtype", DTYPES)
def test_strided_rows(dtype):
    """Row distances beyond the width and rows that start at any element."""
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(9)
    T, k, E, H = 40, 3, 9, 203
    c = make_case(rng, T, k, E, 4, 0.1, dtype, H)
    d = {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in c.items()}
    xw = torch.full((T, H + 29), float("nan"), dtype=dtype, device="cuda")
    rw = torch.full((c["cap"], H + 5), float("nan"), dtype=dtype, device="cuda")
    xs, rs = xw[:, 3:3 + H], rw[:, 1:1 + H]
    xs.copy_(d["x"])
    rs.copy_(d["rows"])
    m = (d["dst"], d["src"], d["offs"])
    n = c["end"]
    assert torch.equal(ops.moe_sort_tokens(xs, *m, prob=d["prob"])[:n],
                       ops.moe_sort_tokens(d["x"], *m, prob=d["prob"])[:n])
    assert torch.equal(ops.moe_unsort_tokens(rs, d["dst"], prob=d["prob"]),
                       ops.moe_unsort_tokens(d["rows"], d["dst"], prob=d["prob"]))
    for a, b in ((ops.moe_sort_tokens_backward(rs, d["dst"], x=xs, prob=d["prob"]),
                  ops.moe_sort_tokens_backward(d["rows"], d["dst"], x=d["x"], prob=d["prob"])),):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a = ops.moe_unsort_tokens_backward(xs, *m, rows=rs, prob=d["prob"])
    b = ops.moe_unsort_tokens_backward(d["x"], *m, rows=d["rows"], prob=d["prob"])
    assert torch.equal(a[0][:n], b[0][:n]) and torch.equal(a[1], b[1])


def test_padding_in_trimmed_row_arrays():
    """Row arrays cut to the last offset still get their padding rows zeroed,
    though they hold fewer rows than there are entries."""
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(11)
    c = make_case(rng, 50, 4, 8, 8, 0.6, torch.bfloat16, 72)
    n = c["end"]
    assert n < 200
    src = c["src"][:n].contiguous().cuda()
    out = torch.full((n, 72), 5.0, dtype=torch.bfloat16, device="cuda")
    ops.moe_sort_tokens(c["x"].cuda(), c["dst"].cuda(), src, c["offs"].cuda(), out=out)
    assert torch.equal(out.cpu().double(), rows_ref(c, False))


def test_rows_out_of_range_are_skipped():
    from nvfp4_w4a4_quantized_amd import ops
    x = torch.randn(4, 48, device="cuda")
    dst = torch.tensor([[0, 5], [-7, 1], [2, 1 << 30], [6, 3]], dtype=torch.int32, device="cuda")
    src = torch.tensor([0, 1, 2, 3, -1], dtype=torch.int32, device="cuda")
    offs = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    rows = ops.moe_sort_tokens(x, dst, src, offs)
    assert torch.equal(rows[:4], x) and bool((rows[4] == 0).all())
    y, dp = ops.moe_sort_tokens_backward(rows, dst, x=x)
    assert torch.equal(y, x)
    assert bool((dp.cpu()[dst.cpu().ge(5) | dst.cpu().lt(0)] == 0).all())


def test_infinities_reach_their_own_token_only():
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(12)
    c = make_case(rng, 20, 3, 6, 1, 0.0, torch.float32, 100)
    c["rows"][int(c["dst"][4, 1])] = float("inf")
    y = ops.moe_unsort_tokens(c["rows"].cuda(), c["dst"].cuda(), prob=c["prob"].cuda()).cpu()
    assert bool(torch.isinf(y[4]).all())
    keep = torch.arange(20) != 4
    assert bool(torch.isfinite(y[keep]).all())


def test_weight_gradients_against_differences():
    """The movements are linear in the weights: differences of the forward
    with step 1 are exact up to its binary32 roundings."""
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(13)
    T, k, H = 6, 3, 50
    c = make_case(rng, T, k, 7, 1, 0.0, torch.float32, H)
    d = {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in c.items()}
    dprob = ops.moe_unsort_tokens_backward(d["x"], d["dst"], d["src"], d["offs"], rows=d["rows"],
                                           prob=d["prob"])[1].cpu().double()
    base = ops.moe_unsort_tokens(d["rows"], d["dst"], prob=d["prob"]).cpu().double()
    for j in range(k):
        up = d["prob"].clone()
        up[:, j] += 1.0
        y = ops.moe_unsort_tokens(d["rows"], d["dst"], prob=up).cpu().double()
        num = ((y - base) * c["x"].double()).sum(1)
        assert float((num - dprob[:, j]).abs().max()) < 1e-3   # H * 2^-22 * |y x|, |y x| < 30


def test_more_than_two_to_the_31_elements():
    """Rows whose offsets pass 31 bits: the last tokens' rows, both ways."""
    from nvfp4_w4a4_quantized_amd import ops
    T, k, H = 270_000, 8, 1024
    x = torch.randn((T, H), device="cuda").bfloat16()
    row = torch.arange(T * k, dtype=torch.int32, device="cuda")
    dst = (T * k - 1 - row).view(T, k).contiguous()
    src = (torch.flip(row, (0,)) // k).to(torch.int32)
    offs = torch.tensor([0, T * k], dtype=torch.int32, device="cuda")
    prob = torch.full((T, k), 0.125, device="cuda")
    rows = ops.moe_sort_tokens(x, dst, src, offs)
    for r in (0, 1, T * k // 2, T * k - 1):
        assert torch.equal(rows[r], x[int(src[r])])
    y = ops.moe_unsort_tokens(rows, dst, prob=prob)
    assert torch.equal(y, x)
    drows, dprob = ops.moe_unsort_tokens_backward(x, dst, src, offs, rows=rows, prob=prob)
    assert torch.equal(drows[T * k - 1], (x[0].float() * 0.125).bfloat16())
    ref = (x[-4:].double() ** 2).sum(1, keepdim=True).expand(4, k)
    assert bool(((dprob[-4:].double() - ref).abs() <= (H + 2) * 2.0 ** -24 * ref).all())
