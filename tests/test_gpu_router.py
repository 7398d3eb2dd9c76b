"""moe_router and its gradient against their binary64 definitions.

Tolerances: a weight is a quotient of binary32 exponentials.  With r the
largest |l - max| among the terms that count, the two roundings of the
argument, that of log2 e and the exponential's own error move a term by at
most (2.5 r + 4) 2^-24 relative (r capped at 104: beyond it the term is
zero), the n-term sum by n 2^-24, the quotient and the scale by 2 2^-24:
together below (2 R + n + 16) 2^-24 with R = r + max |l| >= 1.5 r.  A weight
below the normal range may be flushed to zero, 2^-126 off; the gradient
multiplies that error by at most |dw| + sum q |dw| <= 2 max |dw|.  log s(l) carries one more rounding of its magnitude,
which R covers.  The gradient multiplies two such values with binary32
differences of dw, so its error is below twice that, relative to
q (|dw| + sum q |dw|); the result's type adds its half step."""
import numpy as np
import pytest
import torch

import operator_ref as R
from gpu_util import say

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def make_logits(rng, T, E, dtype, kind):
    z = rng.standard_normal((T, E)).astype(np.float32)
    if kind == "ties":
        z = np.round(z * 2) / 2            # many equal keys, both zeros among them
        z[z == 0] *= np.where(rng.random((z == 0).sum()) < 0.5, 1.0, -1.0).astype(np.float32)
    elif kind == "masked":
        z[rng.random((T, E)) < 0.6] = -np.inf
        z[T // 2] = -np.inf                # nothing left
        if T > 2:
            z[1] = -np.inf
            z[1, E - 1] = 0.25             # one left
    elif kind == "lowest":
        low = torch.finfo(dtype).min
        z[rng.random((T, E)) < 0.5] = low
        z[T // 2] = low                    # all the type's lowest value: not masked
    elif kind == "wide":
        z *= 60.0
    return torch.from_numpy(z).to(dtype)


def bound(logits, ids, score, renorm):
    z = logits.double()
    z = torch.where(torch.isfinite(z) & (z.abs() < 1e30), z, torch.zeros_like(z))
    n = ids.shape[1] if renorm else z.shape[1]
    r = min(104.0, float((z.max() - z.min()).abs()) + float(z.abs().max()))
    return (2 * r + n + 16) * 2.0 ** -24


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["plain", "ties", "masked", "lowest", "wide"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 128, 8), (3, 7, 7), (65, 60, 4), (130, 129, 6),
                                   (37, 257, 9), (9, 1000, 20), (5, 1024, 1),
                                   (6, 100, 40), (4, 1024, 200), (3, 256, 256),
                                   # the other lanes and experts per lane
                                   (50, 8, 2), (33, 16, 16), (20, 17, 4), (41, 64, 6),
                                   (12, 300, 12), (8192, 130, 3), (8200, 290, 5)])
def test_router_matches_the_definition(T, E, k, kind, dtype):
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(T * 1000 + E + k)
    logits = make_logits(rng, T, E, dtype, kind)
    dev = logits.cuda()
    dprob = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32))
    ids = R.router_ids(logits, k)
    for score in (0, 1):
        for renorm in (False, True):
            scale = 2.5 if renorm else 1.0
            say("router", T, E, k, kind, dtype, score, renorm)
            got_ids, got = ops.moe_router(dev, k, score=score, renormalize=renorm, scale=scale)
            assert torch.equal(got_ids.cpu(), ids)
            ref = R.router_weights(logits, ids, score, renorm, scale)
            tol = bound(logits, ids, score, renorm)
            err = (got.cpu().double() - ref).abs()
            assert bool((err <= tol * ref.abs() + scale * 2.0 ** -126).all()), float(err.max())
            dz = ops.moe_router_backward(dprob.cuda(), dev, got_ids, score=score,
                                         renormalize=renorm, scale=scale)
            assert dz.dtype == dtype
            refd = R.router_gradient(logits, ids, dprob, score, renorm, scale)
            q = R.router_weights(logits, ids, score, renorm)
            dw = scale * dprob.double().abs()
            lim = torch.zeros(T, E, dtype=torch.float64)
            ok = ids >= 0
            size = q * (dw + (q * dw).sum(1, keepdim=True))
            lim.scatter_add_(1, ids.clamp(min=0).long(), torch.where(ok, size, torch.zeros_like(size)))
            if score == 0 and not renorm:
                lim += R.softmax_rows(logits.double()) * (q * dw).sum(1, keepdim=True)
            err = (dz.cpu().double() - refd).abs()
            lim = 2 * tol * lim + R.STEP[dtype] * refd.abs() * 1.0001 + R.TINY[dtype] * 1.0001
            lim += 2 * float(dw.max()) * 2.0 ** -126       # flushed weights (see above)
            assert bool((err <= lim).all()), float((err - lim).max())


@pytest.mark.parametrize("E", [60, 300])
def test_router_bias_counts_for_the_choice_alone(E):
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(E)
    logits = make_logits(rng, 50, E, torch.float32, "plain")
    bias = torch.from_numpy(rng.standard_normal(E).astype(np.float32) * 2)
    bias[3] = -np.inf                       # masks the expert
    ids = R.router_ids(logits, 5, bias)
    assert not bool((ids == 3).any())
    for score, renorm in ((0, False), (0, True), (1, True)):
        got_ids, got = ops.moe_router(logits.cuda(), 5, bias=bias.cuda(), score=score,
                                      renormalize=renorm)
        assert torch.equal(got_ids.cpu(), ids)
        ref = R.router_weights(logits, ids, score, renorm)
        assert bool(((got.cpu().double() - ref).abs() <= bound(logits, ids, score, renorm) * ref).all())


@pytest.mark.parametrize("E", [40, 500])
def test_rows_with_nan_or_infinity(E):
    """Their weights and gradients are NaN, the ids valid; other rows unchanged."""
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(E + 1)
    logits = make_logits(rng, 70, E, torch.float32, "plain")
    clean = logits.clone()
    logits[5, 7] = float("nan")
    logits[6, 9] = float("inf")
    logits[7, :] = float("nan")
    dprob = torch.from_numpy(rng.standard_normal((70, 4)).astype(np.float32))
    bad = torch.zeros(70, dtype=torch.bool)
    bad[5:8] = True
    for score in (0, 1):
        for renorm in (False, True):
            i0, w0 = ops.moe_router(clean.cuda(), 4, score=score, renormalize=renorm)
            i1, w1 = ops.moe_router(logits.cuda(), 4, score=score, renormalize=renorm)
            assert bool(torch.isnan(w1.cpu()[bad]).all())
            assert torch.equal(i0.cpu()[~bad], i1.cpu()[~bad])
            assert torch.equal(w0.cpu()[~bad], w1.cpu()[~bad])
            assert bool(((i1 >= -1) & (i1 < E)).all())
            d = ops.moe_router_backward(dprob.cuda(), logits.cuda(), i1, score=score,
                                        renormalize=renorm).cpu()
            assert bool(torch.isnan(d[bad]).all()) and not bool(torch.isnan(d[~bad]).any())


def test_gradient_against_differences():
    """Central differences of the binary64 weights, h = 1e-6: their own error
    is about h^2 and 2^-52 / h, far below the binary32 bound."""
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(2)
    T, E, k = 4, 12, 3
    logits = make_logits(rng, T, E, torch.float32, "plain")
    dprob = torch.from_numpy(rng.standard_normal((T, k)).astype(np.float32))
    ids = R.router_ids(logits, k)
    h = 1e-6
    for score in (0, 1):
        for renorm in (False, True):
            num = torch.zeros(T, E, dtype=torch.float64)
            for e in range(E):
                up, dn = logits.double().clone(), logits.double().clone()
                up[:, e] += h
                dn[:, e] -= h
                f = [(R.router_weights(z, ids, score, renorm, 1.5) * dprob.double()).sum(1)
                     for z in (up, dn)]
                num[:, e] = (f[0] - f[1]) / (2 * h)
            got = ops.moe_router_backward(dprob.cuda(), logits.cuda(), ids.cuda(), score=score,
                                          renormalize=renorm, scale=1.5)
            assert float((got.cpu().double() - num).abs().max()) < 1e-5


def test_foreign_and_repeated_ids_in_the_gradient():
    """Ids out of range are skipped, one named twice counts twice."""
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(3)
    logits = make_logits(rng, 3, 20, torch.float32, "plain")
    ids = torch.tensor([[4, 4, 7], [-5, 20, 2], [1 << 30, -1, 99]], dtype=torch.int32)
    dprob = torch.from_numpy(rng.standard_normal((3, 3)).astype(np.float32))
    for score in (0, 1):
        for renorm in (False, True):
            got = ops.moe_router_backward(dprob.cuda(), logits.cuda(), ids.cuda(), score=score,
                                          renormalize=renorm).cpu().double()
            ref = R.router_gradient(logits, ids, dprob, score, renorm)
            assert float((got - ref).abs().max()) < 1e-5


def test_strided_logits_and_no_tokens():
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(4)
    for dtype in DTYPES:
        wide = make_logits(rng, 33, 151, dtype, "plain").cuda()
        part = wide[:, 3:123]               # row distance 151, rows at odd addresses
        i0, w0 = ops.moe_router(part, 6)
        i1, w1 = ops.moe_router(part.contiguous(), 6)
        assert torch.equal(i0, i1) and torch.equal(w0, w1)
        d = torch.ones_like(w0)
        assert torch.equal(ops.moe_router_backward(d, part, i0),
                           ops.moe_router_backward(d, part.contiguous(), i1))
        i, w = ops.moe_router(wide[:0], 6)
        assert i.shape == (0, 6) and w.shape == (0, 6)
        assert ops.moe_router_backward(w, wide[:0], i).shape == (0, 151)


def test_many_tokens():
    """More tokens than one pass of the grid's groups, checked as a whole."""
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(5)
    logits = make_logits(rng, 20001, 128, torch.bfloat16, "ties")
    ids, w = ops.moe_router(logits.cuda(), 8)
    ref = R.router_ids(logits, 8)
    assert torch.equal(ids.cpu(), ref)
    rw = R.router_weights(logits, ref, 0, True)
    assert bool(((w.cpu().double() - rw).abs() <= bound(logits, ref, 0, True) * rw).all())


def test_more_than_two_to_the_31_logits():
    from nvfp4_w4a4_quantized_amd import ops
    T, E = 2_200_000, 1000
    logits = torch.randn((T, E), device="cuda", dtype=torch.bfloat16)
    ids, w = ops.moe_router(logits, 4)
    tail = logits[-5:].contiguous()
    i1, w1 = ops.moe_router(tail, 4)
    assert torch.equal(ids[-5:], i1) and torch.equal(w[-5:], w1)
    dz = ops.moe_router_backward(w, logits, ids, renormalize=False)
    assert torch.equal(dz[-5:], ops.moe_router_backward(w1, tail, i1, renormalize=False))
