"""moe_router with a bias on the scores (softmax or sigmoid over all experts).

The picks are compared through binary64 keys: a pick may come after, or an
expert be left out for, one whose key is larger by no more than both keys'
errors.  A key's error: the binary32 score's, (6 M + E + 16) 2^-24 relative with
M the row's largest |l| (each exponential's argument is rounded, at most 2 M, and
its product with log2 e; the sum of E terms; the quotient) and 2^-126 where it
is flushed, and the key's rounding, 2^-24 of it."""
import numpy as np
import pytest
import torch

import operator_ref as R
from gpu_util import say

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def scores(logits, score):
    z = logits.double()
    return R.softmax_rows(z) if score == 0 else torch.exp(R.log_sigmoid(z))


def check_picks(ids, logits, bias, score):
    z = logits.double()
    s = scores(logits, score)
    key = s + bias.double()
    m = torch.where(torch.isfinite(z), z.abs(), torch.zeros_like(z)).amax(1, keepdim=True)
    err = (6 * m + z.shape[1] + 16) * 2.0 ** -24 * s + 2.0 ** -24 * key.abs() + 2.0 ** -126
    gone = torch.isinf(z) & (z < 0) | torch.isinf(key)
    key = torch.where(gone, torch.full_like(key, -np.inf), key)
    err = torch.where(gone, torch.zeros_like(err), err)
    ids = ids.cpu().long()
    ok = ids >= 0
    left = (~gone).sum(1)
    assert torch.equal(ok.sum(1), torch.clamp(left, max=ids.shape[1]))
    assert bool((ok[:, :-1] | ~ok[:, 1:]).all())            # those left over come last
    at = ids.clamp(min=0)
    pk, pe = key.gather(1, at), err.gather(1, at)
    assert bool((pk[ok] > -np.inf).all())
    down = pk[:, 1:] - pe[:, 1:] <= pk[:, :-1] + pe[:, :-1]
    assert bool((down | ~ok[:, 1:]).all())
    # distinct, and no better expert left out
    seen = torch.zeros(key.shape, dtype=torch.long).scatter_add_(1, at, ok.long())
    assert int(seen.max()) <= 1
    rest = torch.where(seen > 0, torch.full_like(key, -np.inf), key - err).amax(1)
    last = torch.where(ok, pk + pe, torch.full_like(pk, np.inf)).amin(1)
    assert bool((rest <= last).all())


def check_weights(got, logits, ids, score, renorm, scale):
    z = logits.double()
    z = torch.where(torch.isfinite(z), z, torch.zeros_like(z))
    ref = R.router_weights(logits, ids.cpu(), score, renorm, scale)
    r = float(z.max() - z.min()) + float(z.abs().max())
    tol = (2 * min(r, 104.0) + z.shape[1] + 16) * 2.0 ** -24
    err = (got.cpu().double() - ref).abs()
    assert bool((err <= tol * ref.abs() + scale * 2.0 ** -126).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (7, 8, 2), (65, 16, 16), (50, 60, 4), (33, 128, 8),
                                   (20, 130, 6), (9, 300, 12), (5, 1000, 20), (4, 1024, 200),
                                   (3, 256, 256), (8192, 130, 3), (8200, 290, 5)])
def test_picks_and_weights(T, E, k, dtype):
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(T + E + k)
    z = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32) * 3).to(dtype)
    z[rng.random((T, E)) < 0.2] = -np.inf
    if T > 4:
        z[T // 2] = -np.inf                                 # nothing left
    for score in (0, 1):
        # as large as the scores differ, so that both count
        bias = torch.from_numpy(rng.standard_normal(E).astype(np.float32) * (0.3 if score else 0.5 / E))
        if E > 4:
            bias[2] = -np.inf
            bias[3] = 10.0                                  # picked wherever it is not masked
        for renorm in (False, True):
            scale = 2.5 if renorm else 1.0
            say("router, score bias", T, E, k, dtype, score, renorm)
            ids, w = ops.moe_router(z.cuda(), k, score=score, renormalize=renorm, scale=scale,
                                    score_bias=bias.cuda())
            check_picks(ids, z, bias, score)
            check_weights(w, z, ids, score, renorm, scale)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("E", [2, 40, 500])
def test_score_and_logit_bias_rank_differently(E, score):
    """Logits 4 and 2 with a bias of 0.5 on the second: 4 against 2.5 on the
    logit, 0.982 against 1.381 (sigmoid) on the score; softmax of the two with a
    bias of 0.9: 4 against 2.9, 0.881 against 1.019."""
    from nvfp4_w4a4_quantized_amd import ops
    z = torch.full((3, E), -60.0)
    z[:, E - 2], z[:, E - 1] = 4.0, 2.0
    bias = torch.zeros(E)
    bias[E - 1] = 0.5 if score else 0.9
    on_logit, _ = ops.moe_router(z.cuda(), 1, bias=bias.cuda(), score=score)
    on_score, w = ops.moe_router(z.cuda(), 1, score_bias=bias.cuda(), score=score, renormalize=False)
    assert bool((on_logit == E - 2).all()) and bool((on_score == E - 1).all())
    check_weights(w, z, on_score, score, False, 1.0)


@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("E", [16, 128, 300])
def test_equal_keys_by_ascending_id(E, score):
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(E)
    z = torch.from_numpy(rng.integers(0, 2, (40, E)).astype(np.float32))
    bias = torch.zeros(E)
    ids, _ = ops.moe_router(z.cuda(), 6, score=score, score_bias=bias.cuda())
    assert torch.equal(ids.cpu(), R.router_ids(z, 6))       # the score rises with the logit
    ids, _ = ops.moe_router(torch.full((3, E), 90.0).cuda(), 6, score=score, score_bias=bias.cuda())
    assert torch.equal(ids.cpu(), torch.arange(6, dtype=torch.int32).expand(3, 6))


def test_zero_bias_is_no_bias_for_separated_logits():
    """Softmax and sigmoid rise with the logit: with distinct keys the picks are
    the unbiased ones."""
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(7)
    z = torch.stack([torch.from_numpy(rng.permutation(64).astype(np.float32)) / 8 for _ in range(30)])
    bias = torch.zeros(64)
    for score in (0, 1):
        a, wa = ops.moe_router(z.cuda(), 8, score=score)
        b, wb = ops.moe_router(z.cuda(), 8, score=score, score_bias=bias.cuda())
        assert torch.equal(a, b) and torch.equal(wa, wb)


@pytest.mark.parametrize("E", [40, 500])
def test_rows_with_nan_or_infinity(E):
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(E + 1)
    z = torch.from_numpy(rng.standard_normal((20, E)).astype(np.float32))
    clean = z.clone()
    z[5, 7], z[6, 9] = float("nan"), float("inf")
    z[7] = float("nan")
    bias = torch.from_numpy(rng.standard_normal(E).astype(np.float32)).cuda()
    bad = torch.zeros(20, dtype=torch.bool)
    bad[5:8] = True
    for score in (0, 1):
        for renorm in (False, True):
            i0, w0 = ops.moe_router(clean.cuda(), 4, score=score, renormalize=renorm, score_bias=bias)
            i1, w1 = ops.moe_router(z.cuda(), 4, score=score, renormalize=renorm, score_bias=bias)
            assert bool(torch.isnan(w1.cpu()[bad]).all())
            assert torch.equal(i0.cpu()[~bad], i1.cpu()[~bad])
            assert torch.equal(w0.cpu()[~bad], w1.cpu()[~bad])
            assert bool(((i1 >= -1) & (i1 < E)).all())


def test_strides_streams_and_capture():
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(4)
    bias = torch.from_numpy(rng.standard_normal(120).astype(np.float32) * 0.2).cuda()
    wide = torch.from_numpy(rng.standard_normal((33, 151)).astype(np.float32)).bfloat16().cuda()
    part = wide[:, 3:123]

    def step():
        return ops.moe_router(part, 6, score=1, score_bias=bias)
    want = ops.moe_router(part.contiguous(), 6, score=1, score_bias=bias)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step()
    for _ in range(3):
        wide.copy_(torch.from_numpy(rng.standard_normal((33, 151)).astype(np.float32)))
        want = [t.clone() for t in step()]
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(held[0], want[0]) and torch.equal(held[1], want[1])
    i, w = ops.moe_router(part[:0], 6, score_bias=bias)
    assert i.shape == (0, 6) and w.shape == (0, 6)


def test_gradient_takes_the_picks():
    """The bias has no part in the weights, so the gradient is that of the same
    ids without it."""
    from nvfp4_w4a4_quantized_amd import ops
    rng = np.random.default_rng(9)
    z = torch.from_numpy(rng.standard_normal((12, 30)).astype(np.float32))
    bias = torch.from_numpy(rng.standard_normal(30).astype(np.float32))
    dw = torch.from_numpy(rng.standard_normal((12, 4)).astype(np.float32))
    for score in (0, 1):
        for renorm in (False, True):
            ids, _ = ops.moe_router(z.cuda(), 4, score=score, renormalize=renorm, score_bias=bias.cuda())
            dz = ops.moe_router_backward(dw.cuda(), z.cuda(), ids, score=score, renormalize=renorm)
            ref = R.router_gradient(z, ids.cpu(), dw, score, renorm)
            assert float((dz.cpu().double() - ref).abs().max()) < 1e-5


def test_refused_arguments():
    from nvfp4_w4a4_quantized_amd import ops
    from nvfp4_w4a4_quantized_amd._lib import NvFp4Error
    z = torch.zeros(4, 8, device="cuda")
    b = torch.zeros(8, device="cuda")
    for kind, kw in ((ValueError, dict(bias=b, score_bias=b)), (ValueError, dict(score_bias=b[:7])),
                     (TypeError, dict(score_bias=b.double())), (NvFp4Error, dict(score_bias=b.cpu()))):
        with pytest.raises(kind):
            ops.moe_router(z, 2, **kw)
