"""The adapters where a value is infinite: what the definition's own arithmetic
gives, the sign of an infinity included, for every type.

Finite values are held to the bounds of test_gpu_lora.py: (K + rank + 24) 2^-24 of
the magnitudes forward, N in K's place and T products more on the way back, then
the output's half step."""
import pytest
import torch

import adapter_ref as A
import operator_ref as R
from gpu_util import say
from test_gpu_lora import cuda, make

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
INF = float("inf")


def same(got, ref, lim, what):
    """NaN where ref has one, its infinities with their signs, and the rest of it
    within lim and got's rounding."""
    g = got.cpu().double()
    finite = torch.isfinite(ref)
    assert torch.equal(torch.isnan(g), torch.isnan(ref)), f"{what}: NaN in other places"
    odd = ~finite & ~torch.isnan(ref)
    assert torch.equal(g[odd], ref[odd]), f"{what}: other infinities"
    bad = R.outside(got.cpu()[finite], ref[finite], lim[finite])
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} outside"


def positive(c, *names):
    """No zeros and one sign, so that no 0 * inf and no inf - inf is meant."""
    for n in names:
        c[n] = c[n].abs() + 0.125
    return c


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rank", [1, 8, 16, 20, 48, 100])
@pytest.mark.parametrize("T", [1, 5, 300])
def test_infinities_of_b(T, rank, dtype):
    """Rows of x with one element make h a value of x's type, whose lower parts are
    zero in every split."""
    from nvfp4_w4a4_quantized_amd import ops
    K, N, S = 40, 130, 3
    c = positive(make(T, K, N, rank, S, "random", dtype, 11), "x", "a")
    c["x"][::2] = 0
    c["x"][::2, 5] = 1
    c["ids"] = (torch.arange(T) % 4).to(torch.int32)            # (3: without an adapter)
    c["scale"] = torch.tensor([1.5, -0.75, 1.0])
    for s in range(2):
        c["b"][s, 3 + s, 0], c["b"][s, 64, rank - 1], c["b"][s, 129, rank // 2] = INF, -INF, INF
    x, a, b, ids, base = cuda(c, "x", "a", "b", "ids", "base")
    for scale in (None, c["scale"]):
        y, ym, _, _ = A.forward(c["x"], c["a"], c["b"], c["ids"], scale, c["base"])
        assert not bool(torch.isnan(y).any()) and (~torch.isfinite(y)).sum() == 3 * int((c["ids"] < 2).sum())
        say("lora_forward", T, rank, dtype, scale is None)
        got = ops.lora_forward(x, a, b, ids, scale=None if scale is None else scale.cuda(), base=base)
        same(got, y, (K + rank + 24) * A.ULP * ym, "y")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rank", [3, 16, 24, 48, 100])
@pytest.mark.parametrize("T", [4, 300, 1500])
def test_infinities_on_the_way_back(T, rank, dtype):
    """One in a, x and dy each: dx's columns, da's and db's."""
    from nvfp4_w4a4_quantized_amd import ops
    K, N, S = 72, 136, 3
    c = positive(make(T, K, N, rank, S, "random", dtype, 12), "dy", "b")
    c["ids"] = (torch.arange(T) % 4).to(torch.int32)
    h = make(T, rank, 1, 1, 1, "one", dtype, 13)["x"].float()   # (values of the type, of either sign)
    h = torch.where(h == 0, torch.ones_like(h), h)
    c["dy"][1::2] = 0                                           # g is one value of b there
    c["dy"][1::2, 9] = 1
    c["a"][0, 0, 7], c["x"][1, 11], c["dy"][2, 20] = -INF, INF, INF
    c["x"][c["x"] == 0] = 1
    dy, x, a, b, ids = cuda(c, "dy", "x", "a", "b", "ids")
    (dx, dxm), (da, dam), (db, dbm) = A.backward(c["dy"], c["x"], c["a"], c["b"], c["ids"], None, h, None)
    assert bool(torch.isinf(dx[0, 7])) and bool(torch.isinf(da[1, :, 11]).all())
    assert bool(torch.isinf(db[2, 20]).all()) and bool(torch.isinf(da[2]).all())
    say("lora_backward", T, rank, dtype)
    got = ops.lora_backward(dy, x, a, b, ids, h=h.cuda())
    same(got[0], dx, (N + rank + 24) * A.ULP * dxm, "dx")
    same(got[1], da, (N + T + 40) * A.ULP * dam, "da")
    same(got[2], db, (T + 24) * A.ULP * dbm, "db")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rank", [5, 20, 40, 100])
@pytest.mark.parametrize("T", [4, 200, 300])
def test_an_infinite_scale(T, rank, dtype):
    """With positive values every product of it is one infinity, whatever the rank
    is padded to."""
    from nvfp4_w4a4_quantized_amd import ops
    K, N, S = 40, 88, 2
    c = positive(make(T, K, N, rank, S, "random", dtype, 14), "x", "a", "b", "dy")
    c["ids"] = (torch.arange(T) % 3).to(torch.int32)
    c["scale"] = torch.tensor([INF, -2.0])
    x, a, b, ids, base, dy, scale = cuda(c, "x", "a", "b", "ids", "base", "dy", "scale")
    y, ym, h, _ = A.forward(c["x"], c["a"], c["b"], c["ids"], c["scale"], c["base"])
    say("infinite scale", T, rank, dtype)
    same(ops.lora_forward(x, a, b, ids, scale=scale, base=base), y, (K + rank + 24) * A.ULP * ym, "y")
    (dx, dxm), (da, dam), (db, dbm) = A.backward(c["dy"], c["x"], c["a"], c["b"], c["ids"], c["scale"],
                                                 h.float(), None)
    assert bool((dx[0] == INF).all()) and bool((da[0] == INF).all()) and bool((db[0] == INF).all())
    got = ops.lora_backward(dy, x, a, b, ids, scale=scale, h=h.float().cuda())
    same(got[0], dx, (N + rank + 24) * A.ULP * dxm, "dx")
    same(got[1], da, (N + T + 40) * A.ULP * dam, "da")
    same(got[2], db, (T + 24) * A.ULP * dbm, "db")
