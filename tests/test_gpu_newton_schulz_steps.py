"""newton_schulz of bf16 results over more steps, and with other coefficients, than
the upper 11 bits of the products carry.

Tolerances, relative to the norm of a matrix: the rounding to bf16, no element's
half step being above 2^-8, and binary32 products, 2e-5 after five steps and
growing with the square root of their number (each step turns the singular vectors
by its own roundings): 8e-5 after 64.  X's last bit, 2^-22 of its unit length, is
2e-5 of the smallest singular values here, which are a hundredth of that length.
1e-4 holds both."""
import pytest
import torch

import adapter_ref as A
from gpu_util import say

pytestmark = pytest.mark.gpu
USUAL = (3.4445, -4.7750, 2.0315)
TOL = 2.0 ** -8 + 1e-4


def noise(E, n, m, seed):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(E, n, m, generator=gen) * 1e-3).cuda()


def off(got, ref):
    return (got.double() - ref).norm(dim=(-2, -1)) / ref.norm(dim=(-2, -1))


@pytest.mark.parametrize("steps", [7, 20, 40, 64])
@pytest.mark.parametrize("E,n,m", [(1, 256, 400), (3, 400, 256), (90, 150, 300)])
def test_more_steps_in_bf16(E, n, m, steps):
    from nvfp4_w4a4_quantized_amd import ops
    g = noise(E, n, m, n + steps)
    say("newton_schulz bf16", E, n, m, steps)
    d = off(ops.newton_schulz(g, steps=steps, out_dtype=torch.bfloat16), A.newton_schulz(g, steps, USUAL, 1e-7))
    assert bool((d <= TOL).all()), f"{steps} steps: {float(d.max()):.3g}"


def test_products_that_cancel_in_bf16():
    """One direction, whose length a + b + c = 2^-9 leaves: the sum's terms are 500
    times the result, and lose nothing of it beyond 22 bits of each, four of them
    (500 * 4 * 2^-22)."""
    from nvfp4_w4a4_quantized_amd import ops
    gen = torch.Generator().manual_seed(5)
    g = torch.randn(120, 1, generator=gen) @ torch.randn(1, 300, generator=gen)
    co = (1.0, 0.0, -1.0 + 2.0 ** -9)
    say("newton_schulz bf16 cancelling")
    got = ops.newton_schulz(g.cuda(), steps=1, coefficients=co, eps=0.0, out_dtype=torch.bfloat16)
    d = off(got, A.newton_schulz(g.cuda(), 1, co, 0.0))
    assert bool(d <= 2.0 ** -8 + 500 * 4 * 2.0 ** -22), f"{float(d):.3g}"
