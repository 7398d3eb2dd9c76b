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
