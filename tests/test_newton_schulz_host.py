"""newton_schulz's definition by singular values, and calls that its range refuses
(no GPU needed)."""
import pytest
import torch

import adapter_ref as A
from test_operators_host import F, L, UNSUPPORTED, WS_SMALL  # noqa: F401

USUAL = (3.4445, -4.7750, 2.0315)


def call(L, steps, coefficients, rows=80, cols=96, out=0):  # noqa: F811
    return L.newton_schulz(F, 0, 2, rows, cols, cols, rows * cols, steps, *coefficients, 1e-7, 1.0, out,
                           F, F, 0, None)


@pytest.mark.parametrize("out", [0, 1, 2])
def test_coefficients_that_lose_small_singular_values(L, out):  # noqa: F811
    """A singular value far below one shrinks by |a| a step: past 2^-8 in all, X's two
    parts no longer hold its digits beside the large ones'.  Matrices of a short
    side up to 64 are binary64 and take any."""
    for steps, co in ((9, (0.5, 0.0, 0.0)), (2, (0.0, 0.0, 1.0)), (1, (0.003, 0.5, 0.0)), (5, (-0.3, 0.1, 0.0)),
                      (20, (0.5, 0.0, 0.0))):
        assert call(L, steps, co, out=out) == UNSUPPORTED, (steps, co)
        assert call(L, steps, co, rows=96, cols=65, out=out) == UNSUPPORTED, (steps, co)
        assert call(L, steps, co, rows=64, out=out) == WS_SMALL, (steps, co)
        assert call(L, steps, co, rows=500, cols=7, out=out) == WS_SMALL, (steps, co)
    for steps, co in ((8, (0.5, 0.0, 0.0)), (1, (0.004, 0.5, 0.0)), (64, (1.0, 0.0, 0.0)),
                      (64, (1.5, -0.5, 0.0)), (64, USUAL), (3, (-1.0, 0.0, 1.0))):
        assert call(L, steps, co, out=out) == WS_SMALL, (steps, co)


@pytest.mark.parametrize("coefficients,steps", [(USUAL, 1), (USUAL, 5), ((1.5, -0.5, 0.0), 4),
                                                ((-2.0, 1.5, -0.5), 3)])
@pytest.mark.parametrize("shape", [(12, 40), (40, 12), (2, 9, 9)])
def test_the_definition_by_singular_values(shape, coefficients, steps):
    """The update keeps the singular vectors and takes every singular value through
    the odd polynomial: U p(p(..(S / (|G| + eps)))) V^T, in no product of matrices
    of the definition's own.  Sums of 40 products in binary64, each step's errors
    multiplied by at most 3.5: 1e-11."""
    a, b, c = coefficients
    gen = torch.Generator().manual_seed(7)
    g = torch.randn(*shape, generator=gen, dtype=torch.float64)
    u, s, vt = torch.linalg.svd(g, full_matrices=False)
    s = s / (s.square().sum(-1, keepdim=True).sqrt() + 1e-3)
    for _ in range(steps):
        s = a * s + b * s ** 3 + c * s ** 5
    got = A.newton_schulz(g, steps, coefficients, 1e-3, 0.5)
    assert torch.allclose(got, 0.5 * (u * s.unsqueeze(-2)) @ vt, rtol=0, atol=1e-11)
    if coefficients == USUAL and steps == 5:
        assert bool((s < 1.21).all())
