"""The adapters and the update where a launch takes its larger shapes: long batches
whose workgroups walk several turns of columns with the base a turn ahead, and
batches of different matrices on every tile, in every orientation.  Tolerances are
those of test_gpu_lora.py and test_gpu_newton_schulz.py."""
import numpy as np
import pytest
import torch

import adapter_ref as A
import operator_ref as R
import test_gpu_newton_schulz as NS
from gpu_util import say
from test_gpu_lora import check, cuda, make

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rank", [16, 24, 40])
@pytest.mark.parametrize("N", [4104, 4352])
def test_forward_of_a_long_batch(N, rank, dtype):
    """Two turns of 256 columns a workgroup, whole pieces and others."""
    from nvfp4_w4a4_quantized_amd import ops
    T, K, S = 4100, 40, 5
    c = make(T, K, N, rank, S, "runs", dtype, 21)
    x, a, b, ids, scale, base = cuda(c, "x", "a", "b", "ids", "scale", "base")
    lim = (K + rank + 24) * A.ULP
    y, ym, _, _ = A.forward(c["x"], c["a"], c["b"], c["ids"], c["scale"], c["base"])
    say("lora_forward", T, K, N, rank, dtype)
    got = ops.lora_forward(x, a, b, ids, scale=scale, base=base)
    check(got, y, lim * ym, "with base")
    assert ops.lora_forward(x, a, b, ids, scale=scale, base=base, out=base) is base
    assert torch.equal(base, got)
    z = c["base"].double()
    check(ops.lora_forward(x, a, b, ids, scale=scale), y - z, lim * (ym - z.abs()), "without base")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rank", [16, 40])
def test_backward_of_a_long_batch(rank, dtype):
    from nvfp4_w4a4_quantized_amd import ops
    T, K, N, S = 4100, 4352, 24, 3
    c = make(T, K, N, rank, S, "runs", dtype, 22)
    dy, x, a, b, ids, scale, base = cuda(c, "dy", "x", "a", "b", "ids", "scale", "dbase")
    h = A.forward(c["x"], c["a"], c["b"], c["ids"], None, None)[2].float()
    (dx, dxm), (da, dam), (db, dbm) = A.backward(c["dy"], c["x"], c["a"], c["b"], c["ids"], c["scale"], h,
                                                 c["dbase"])
    say("lora_backward", T, K, N, rank, dtype)
    got = ops.lora_backward(dy, x, a, b, ids, scale=scale, h=h.cuda(), base=base, out=base)
    assert got[0] is base
    check(got[0], dx, (N + rank + 24) * A.ULP * dxm, "dx")
    check(got[1], da, (N + T + 40) * A.ULP * dam, "da")
    check(got[2], db, (T + 24) * A.ULP * dbm, "db")


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_projection_of_a_long_batch(dtype):
    """The base in binary32, two turns of columns."""
    from nvfp4_w4a4_quantized_amd import ops
    T, K, N, rank, S = 4100, 128, 4352, 16, 4
    parts = R.make_weights(np.random.default_rng(3), 1, N, K)
    w = ops.NvFp4Weights(*(t.cuda() for t in parts)).packed()
    c = make(T, K, N, rank, S, "runs", dtype, 23)
    y, ym, _, _ = A.forward(c["x"], c["a"], c["b"], c["ids"], c["scale"], None, R.decode(*parts)[0])
    say("nvfp4_lora_matvec", T, K, N, rank, dtype)
    got = ops.nvfp4_lora_matvec(*cuda(c, "x"), w, *cuda(c, "a", "b", "ids"), scale=c["scale"].cuda())
    check(got, y, (K + rank + 40) * A.ULP * ym, "y")


# matrices of 300 have three symmetric 256 x 256 tiles, four 256 x 128 ones and six
# others: by their number every product takes each shape that there is for its type
@pytest.mark.parametrize("out", DTYPES)
@pytest.mark.parametrize("E,n,m", [(40, 300, 520), (66, 300, 520), (66, 520, 300), (90, 300, 520),
                                   (90, 520, 300), (180, 300, 520), (180, 520, 300), (180, 257, 261),
                                   (70, 385, 383)])
def test_batches_of_different_matrices(E, n, m, out):
    from nvfp4_w4a4_quantized_amd import ops
    g = NS.gradient(E, n, m, "signal", torch.float32, 9)
    say("newton_schulz", E, n, m, out)
    got = ops.newton_schulz(g, out_dtype=out)
    NS.check(got, A.newton_schulz(g, 5, NS.USUAL, 1e-7), 5, f"{E} x {n} x {m} -> {out}")
    assert torch.equal(ops.newton_schulz(g, out_dtype=out), got)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,m", [(2300, 2200), (2200, 5000), (4100, 2050)])
def test_one_matrix_of_many_tiles(n, m, out):
    from nvfp4_w4a4_quantized_amd import ops
    g = NS.gradient(1, n, m, "signal", torch.float32, 10)
    say("newton_schulz", n, m, out)
    NS.check(ops.newton_schulz(g, out_dtype=out), A.newton_schulz(g, 5, NS.USUAL, 1e-7), 5, f"{n} x {m}")
