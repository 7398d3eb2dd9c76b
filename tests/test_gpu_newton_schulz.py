"""newton_schulz against binary64.

Tolerances are of the Frobenius norm, per matrix.  bf16 results: a rounding to
11 bits is 2e-4 off in the mean square (half a step, uniform over a binade).
Where X is near orthogonal (all of it at the end, the errors before are
multiplied by |a + 3 b + 5 c| = 0.72) a step's roundings of X and P in P X and of
A make 2e-4 sqrt(2 |P|^2 + (1.7 (b + 2 c))^2) = 8e-4 with |P| <= 2.8; the steps
together up to twice that, and twice again for the spread of singular values:
4e-3.  float32 and fp16 results: binary32 sums of K products wander by sqrt(K)
2^-24 (4e-6 at 4096), four times that as above: 2e-5.  X's own 22 bits, 2^-22 of
|X0| = 1, grow by a per step where a singular value is zero: a^steps 2^-22.
Then the output's half step."""
import math

import pytest
import torch

import adapter_ref as A
import operator_ref as R
from gpu_util import say

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
USUAL = (3.4445, -4.7750, 2.0315)


def gradient(E, n, m, kind, dtype, seed=0):
    gen = torch.Generator().manual_seed(seed + 3 * n + m)
    x = torch.randn(E, n, m, generator=gen)
    k = max(1, min(n, m) // 3)
    if kind == "one":
        x = torch.randn(E, n, 1, generator=gen) @ torch.randn(E, 1, m, generator=gen)
    if kind == "signal":
        fall = torch.arange(1, k + 1).float().rsqrt()
        x = (torch.randn(E, n, k, generator=gen) * fall) @ torch.randn(E, k, m, generator=gen) + 0.3 * x
    return (x * 1e-3 if dtype != torch.float16 else x).to(dtype).cuda()


def check(got, ref, steps, what, coefficients=USUAL, scale=1.0, first=1.0):
    """got within the tolerance of every matrix of ref; first: |X0|."""
    assert got.shape == ref.shape
    got, ref = got.reshape(-1, *got.shape[-2:]), ref.reshape(-1, *ref.shape[-2:])
    grow = abs(coefficients[0]) ** steps * 2.0 ** -22 * first * abs(scale)
    for e in range(got.shape[0]):
        r = float(ref[e].norm())
        d = float((got[e].double() - ref[e]).norm())
        tol = (4e-3 if got.dtype == torch.bfloat16 else 2e-5) * r + grow
        tol += R.STEP[got.dtype] * r + R.TINY[got.dtype] * math.sqrt(ref[e].numel())
        assert d <= tol, f"{what}: matrix {e} off by {d:.3g} of {r:.3g}, tolerance {tol:.3g}"


SHAPES = [(1, 1, 1), (3, 1, 7), (2, 9, 1), (1, 5, 5), (64, 16, 100), (5, 33, 17), (1, 64, 64), (2, 65, 64),
          (3, 16, 2048), (2, 2048, 16), (2, 40, 1111), (2, 63, 130), (2, 100, 99), (1, 128, 129),
          (3, 129, 128), (1, 200, 700), (2, 333, 250), (1, 256, 1024), (1, 700, 257), (1, 513, 515),
          (2, 768, 300), (1, 1000, 1003)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("E,n,m", SHAPES)
def test_sizes(E, n, m, dtype):
    from nvfp4_w4a4_quantized_amd import ops
    g = gradient(E, n, m, "signal", dtype)
    ref = A.newton_schulz(g, 5, USUAL, 1e-7)
    for out in DTYPES:
        say("newton_schulz", E, n, m, dtype, out)
        got = ops.newton_schulz(g, out_dtype=out)
        assert got.dtype == out
        check(got, ref, 5, f"{E} x {n} x {m} {dtype} -> {out}")


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,m", [(4, 50), (48, 20), (150, 200), (300, 140)])
@pytest.mark.parametrize("kind", ["noise", "one", "signal"])
def test_kinds_and_steps(kind, n, m, out):
    from nvfp4_w4a4_quantized_amd import ops
    g = gradient(2, n, m, kind, torch.float32, 1)
    for steps in (1, 2, 5, 7):
        say("newton_schulz", kind, n, m, out, steps)
        got = ops.newton_schulz(g, steps=steps, out_dtype=out, scale=-0.25)
        check(got, A.newton_schulz(g, steps, USUAL, 1e-7, -0.25), steps, f"{kind} {steps}", scale=0.25)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,m", [(8, 24), (90, 70), (140, 400)])
def test_other_coefficients(n, m, out):
    from nvfp4_w4a4_quantized_amd import ops
    g = gradient(1, n, m, "noise", torch.float32, 2)[0]
    for co, steps in (((1.5, -0.5, 0.0), 12), ((1.875, -1.25, 0.375), 9), ((2.0, -1.5, 0.5), 8),
                      ((1.0, 0.0, 0.0), 3), ((-3.4445, 4.7750, -2.0315), 5)):
        say("newton_schulz", n, m, out, co)
        got = ops.newton_schulz(g, steps=steps, coefficients=co, eps=0.0, out_dtype=out)
        check(got, A.newton_schulz(g, steps, co, 0.0), steps, f"{co}", co)


@pytest.mark.parametrize("out", DTYPES)
@pytest.mark.parametrize("n,m", [(6, 40), (80, 30), (130, 150), (260, 90)])
def test_large_and_small_gradients(n, m, out):
    """Norms whose squares leave binary32, and norms far below eps, which leave
    X0 short of unit length: every digit of the result's stays."""
    from nvfp4_w4a4_quantized_amd import ops
    g = gradient(1, n, m, "noise", torch.float32, 3)[0] * 1e3
    for factor in (1e30, 1e-25, 1e-11, 1e-14, 3e-9):
        s = g * factor
        ref = A.newton_schulz(s, 5, USUAL, 1e-7, 1.0)
        first = float(s.double().norm() / (s.double().norm() + 1e-7))
        # (scaled up so that fp16 can hold the result)
        scale = 2.0 ** max(0, math.floor(-math.log2(first)) - 9)
        say("newton_schulz", n, m, out, factor)
        got = ops.newton_schulz(s, out_dtype=out, scale=scale)
        check(got, ref * scale, 5, f"norm times {factor}", scale=scale, first=first)


@pytest.mark.parametrize("n,m", [(7, 33), (150, 140)])
def test_zeros_infinities_and_nan_stay_in_their_matrix(n, m):
    from nvfp4_w4a4_quantized_amd import ops
    g = gradient(6, n, m, "noise", torch.float32, 4)
    want = {out: ops.newton_schulz(g, out_dtype=out) for out in DTYPES}
    g[1] = 0
    g[2, n // 2, m // 3] = float("inf")
    g[4, 0, 0] = float("nan")
    for eps in (1e-7, 0.0):
        for out in DTYPES:
            got = ops.newton_schulz(g, out_dtype=out, eps=eps)
            assert not bool(got[1].any())
            assert bool(torch.isnan(got[2]).all()) and bool(torch.isnan(got[4]).all())
            if eps:
                for e in (0, 3, 5):
                    assert torch.equal(got[e], want[out][e])
            assert bool(torch.isfinite(got[[0, 3, 5]]).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,m", [(20, 61), (130, 77), (96, 256)])
def test_strides_odd_addresses_and_in_place(n, m, dtype):
    from nvfp4_w4a4_quantized_amd import ops
    g = gradient(3, n, m, "noise", dtype, 5)
    want = ops.newton_schulz(g)
    wide = torch.full((4, n + 3, m + 5), float("nan"), dtype=dtype, device="cuda")
    wide[1:, 1:n + 1, 3:m + 3] = g
    assert torch.equal(ops.newton_schulz(wide[1:, 1:n + 1, 3:m + 3]), want)
    one = g[1].contiguous()
    assert torch.equal(ops.newton_schulz(one), want[1])
    assert torch.equal(ops.newton_schulz(one.expand(3, n, m))[2], want[1])
    odd = torch.empty(g.numel() + 1, dtype=dtype, device="cuda")[1:].view(g.shape)
    odd.copy_(g)
    assert ops.newton_schulz(odd, out=odd) is odd
    assert torch.equal(odd, want)


def test_a_dirty_workspace_changes_nothing():
    from nvfp4_w4a4_quantized_amd import ops
    for n, m in ((24, 90), (140, 170)):
        for out in (torch.float32, torch.bfloat16):
            g = gradient(3, n, m, "noise", torch.float32, 6)
            size = ops.newton_schulz_workspace_size(3, n, m, out)
            ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
            assert torch.equal(ops.newton_schulz(g, out_dtype=out, workspace=ws),
                               ops.newton_schulz(g, out_dtype=out))


def test_more_matrices_than_are_taken_at_once():
    """A batch of more than one workspace's matrices.  (The tiles, and so the
    order of the sums, go by the number of matrices taken together: the first
    ones agree in every bit, all of them within the tolerance.)"""
    from nvfp4_w4a4_quantized_amd import ops
    g = gradient(1, 512, 2048, "noise", torch.bfloat16, 7)
    most = 4 * (1 << 30) // (8 * 512 * 2048 + 8 * 512 * 512)
    got = ops.newton_schulz(g.expand(most + 3, 512, 2048))
    assert bool((got[:most] == got[0]).all()) and bool((got[most:] == got[most]).all())
    ref = A.newton_schulz(g, 5, USUAL, 1e-7)
    for e in (0, most):
        check(got[e], ref[0], 5, f"matrix {e}")


def test_no_matrices():
    from nvfp4_w4a4_quantized_amd import ops
    assert ops.newton_schulz(torch.empty(0, 5, 6, device="cuda")).shape == (0, 5, 6)


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,m", [(64, 5000), (2048, 768), (1300, 4100)])
def test_large(n, m, out):
    from nvfp4_w4a4_quantized_amd import ops
    g = gradient(2, n, m, "signal", torch.float32, 8)
    say("newton_schulz", n, m, out)
    check(ops.newton_schulz(g, out_dtype=out), A.newton_schulz(g, 5, USUAL, 1e-7), 5, f"{n} x {m}")
