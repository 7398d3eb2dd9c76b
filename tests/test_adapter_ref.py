"""The adapters' binary64 definitions against autograd and differences, and the
operators' refusals (no GPU needed)."""
import ctypes as C

import pytest
import torch

import adapter_ref as A
from nvfp4_w4a4_quantized_amd import ops
from nvfp4_w4a4_quantized_amd._lib import NvFp4Error, Weights
from test_operators_host import F, INVALID, L, ODD, UNSUPPORTED, WS_SMALL, change  # noqa: F401


@pytest.mark.parametrize("kind", ["runs", "random", "wild", "none"])
def test_gradients_against_autograd_and_differences(kind):
    T, K, N, R, S = 12, 7, 5, 3, 4
    gen = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, a, b, dy, base = n(T, K), n(S, R, K), n(S, N, R), n(T, N), n(T, K)
    ids, scale = A.make_ids(gen, T, S, kind), n(S).float()
    (dx, _), (da, _), (db, _) = A.backward(dy, x, a, b, ids, scale,
                                           A.forward(x, a, b, ids, scale, None)[2], base)
    leaves = [t.clone().requires_grad_() for t in (x, a, b)]

    def loss(x, a, b):
        hot = A.picks(ids, S)
        h = torch.einsum("tk,srk,ts->tr", x, a, hot)
        y = torch.einsum("tr,snr,ts->tn", h, b, hot * scale.double())
        return (y * dy).sum()

    grads = torch.autograd.grad(loss(*leaves), leaves)
    for got, want in zip((dx - base, da, db), grads):
        assert torch.allclose(got, want, rtol=1e-12, atol=1e-12)
    for t, g in ((0, dx - base), (1, da), (2, db)):
        step = n(*g.shape) * 1e-4
        ends = [loss(*[v + f * step if i == t else v for i, v in enumerate((x, a, b))]) for f in (1, -1)]
        # (the loss is linear in each leaf: the difference is exact but for roundings)
        assert abs((ends[0] - ends[1]) / 2 - (g * step).sum()) < 1e-12


def test_forward_refusals(L):  # noqa: F811
    # x, dtype, T, k, ld, ids, a, b, scale, S, rank, n, base, ld_base, out_dtype, out, h, ws, bytes, s
    good = [F, 1, 4, 48, 48, F, F, F, None, 3, 8, 40, None, 40, 1, F, None, F, 1 << 30, None]
    for i, v in ((0, None), (0, ODD), (1, 3), (2, -1), (3, 0), (4, 47), (5, None), (5, ODD), (6, None),
                 (6, ODD), (7, None), (7, ODD), (8, ODD), (9, 0), (10, 0), (11, 0), (12, ODD),
                 (14, 3), (15, None), (15, ODD), (16, ODD), (17, None), (17, C.c_void_p(0x1008))):
        assert L.lora_forward(*change(good, i, v)) == INVALID, (i, v)
    assert L.lora_forward(*change(change(good, 12, F), 13, 39)) == INVALID
    for i, v in ((2, (1 << 24) + 1), (9, 1025), (10, 257), (11, (1 << 18) + 1)):
        assert L.lora_forward(*change(good, i, v)) == UNSUPPORTED, (i, v)
    assert L.lora_forward(*change(change(good, 3, 1 << 19), 4, 1 << 19)) == UNSUPPORTED
    assert L.lora_forward(*change(good, 18, L.lora_forward_workspace_size(4, 48, 8) - 1)) == WS_SMALL
    assert L.lora_forward(*change(good, 2, 0)) == 0
    assert L.lora_forward_workspace_size(4, 48, 257) == 0


def test_backward_refusals(L):  # noqa: F811
    # dy, dtype, T, n, ld, x, k, ld_x, ids, a, b, scale, S, rank, h, base, ld_base, dx, da, db, ws, bytes, s
    good = [F, 1, 4, 40, 40, F, 48, 48, F, F, F, None, 3, 8, None, None, 48, F, F, F, F, 1 << 30, None]
    for i, v in ((0, None), (0, ODD), (1, 3), (2, -1), (3, 0), (4, 39), (5, None), (5, ODD), (6, 0),
                 (7, 47), (8, None), (8, ODD), (9, None), (10, None), (11, ODD), (12, 0), (13, 0),
                 (14, ODD), (15, ODD), (17, None), (17, ODD), (18, None), (18, ODD), (19, None),
                 (19, ODD), (20, None), (20, C.c_void_p(0x1008))):
        assert L.lora_backward(*change(good, i, v)) == INVALID, (i, v)
    assert L.lora_backward(*change(change(good, 15, F), 16, 47)) == INVALID
    for i, v in ((2, (1 << 24) + 1), (12, 1025), (13, 257)):
        assert L.lora_backward(*change(good, i, v)) == UNSUPPORTED, (i, v)
    size = L.lora_backward_workspace_size(1, 4, 48, 40, 3, 8)
    assert L.lora_backward(*change(good, 21, size - 1)) == WS_SMALL
    assert L.lora_backward_workspace_size(3, 4, 48, 40, 3, 8) == 0


def test_backward_refuses_more_threads_than_a_launch_takes(L):  # noqa: F811
    """2^32 threads: tokens * rank (h computed again), and the tiles of 64 x 64 that
    A and B are transposed in, 1024 threads each and one more for the sort."""
    good = [F, 1, 4, 40, 40, F, 48, 48, F, F, F, None, 3, 8, None, None, 48, F, F, F, F, 1 << 30, None]
    many = change(change(good, 2, 1 << 24), 13, 256)
    assert L.lora_backward(*many) == UNSUPPORTED
    assert L.lora_backward_workspace_size(1, 1 << 24, 48, 40, 3, 256) == 0
    assert L.lora_backward(*change(many, 13, 255)) == WS_SMALL
    # 1024 adapters of 4 x (512 + 512) tiles, 2^22 in all; 4 x (512 + 511) are taken
    for k, n, want in ((1 << 15, 1 << 15, UNSUPPORTED), (1 << 15, (1 << 15) - 64, WS_SMALL)):
        wide = [F, 1, 4, n, n, F, k, k, F, F, F, None, 1024, 256, None, None, k, F, F, F, F, 1 << 30, None]
        assert L.lora_backward(*wide) == want, (k, n)
        assert (L.lora_backward_workspace_size(1, 4, k, n, 1024, 256) == 0) == (want == UNSUPPORTED)


def test_matvec_refusals(L):  # noqa: F811
    w = Weights(0x1000, 0x1000, 0x1000, 0)
    # x, dtype, T, ld, w, n, k, ids, a, b, scale, S, rank, out_dtype, out, ws, bytes, s
    good = [F, 1, 4, 256, C.byref(w), 64, 256, F, F, F, None, 3, 8, 1, F, F, 1 << 30, None]
    for i, v in ((0, None), (0, ODD), (1, 3), (2, -1), (3, 255), (4, None), (5, 0), (6, 24), (7, None),
                 (7, ODD), (8, None), (9, ODD), (10, ODD), (11, 0), (12, 0), (13, 3), (14, None),
                 (14, ODD), (15, None), (15, C.c_void_p(0x1008))):
        assert L.nvfp4_lora_matvec(*change(good, i, v)) == INVALID, (i, v)
    for i, v in ((2, 65537), (11, 1025), (12, 257), (5, (1 << 18) + 1)):
        assert L.nvfp4_lora_matvec(*change(good, i, v)) == UNSUPPORTED, (i, v)
    size = L.nvfp4_lora_matvec_workspace_size(4, 64, 256, 8)
    assert L.nvfp4_lora_matvec(*change(good, 16, size - 1)) == WS_SMALL
    assert L.nvfp4_lora_matvec(*change(good, 2, 0)) == 0


def test_python_checks():
    x = torch.zeros(4, 48, dtype=torch.bfloat16)
    t = torch.zeros(2, 8, 48, dtype=torch.bfloat16)
    for call in (lambda: ops.lora_forward(x, t, t, x), lambda: ops.lora_backward(x, x, t, t, x),
                 lambda: ops.nvfp4_lora_matvec(x, ops.NvFp4Weights(x, x, x), t, t, x)):
        with pytest.raises(NvFp4Error):
            call()
    with pytest.raises(TypeError):
        ops.lora_forward([1.0], t, t, x)
    with pytest.raises(TypeError):
        ops.nvfp4_lora_matvec(x, x, t, t, x)


def test_newton_schulz_refusals(L):  # noqa: F811
    # g, dtype, batch, rows, cols, ld_row, ld_batch, steps, a, b, c, eps, scale, out_dtype, out, ws, bytes, s
    good = [F, 0, 2, 40, 60, 60, 2400, 5, 3.4445, -4.775, 2.0315, 1e-7, 1.0, 1, F, F, 1 << 40, None]
    inf, nan = float("inf"), float("nan")
    for i, v in ((0, None), (0, ODD), (1, 3), (2, -1), (3, 0), (4, 0), (5, 59), (6, -1), (7, 0), (8, nan),
                 (9, inf), (10, -inf), (11, -1.0), (11, nan), (11, inf), (12, nan), (12, inf), (13, 3),
                 (14, None), (14, ODD), (15, None), (15, C.c_void_p(0x1008))):
        assert L.newton_schulz(*change(good, i, v)) == INVALID, (i, v)
    for i, v in ((2, (1 << 20) + 1), (3, 16385), (7, 65), (8, 9.0), (9, 40.0), (10, -30.0)):
        assert L.newton_schulz(*change(good, i, v)) == UNSUPPORTED, (i, v)
    assert L.newton_schulz(*change(change(good, 4, 16385), 5, 16385)) == UNSUPPORTED
    for code in (0, 1, 2):
        size = L.newton_schulz_workspace_size(2, 40, 60, code)
        assert L.newton_schulz(*change(change(good, 13, code), 16, size - 1)) == WS_SMALL
    assert L.newton_schulz(*change(good, 2, 0)) == 0
    assert L.newton_schulz_workspace_size(0, 40, 60, 1) == 0
    assert L.newton_schulz_workspace_size(2, 40, 16385, 1) == 0


def test_newton_schulz_brings_singular_values_near_one():
    """The definition itself: the usual coefficients take every singular value
    that is not far below the largest to [0.68, 1.21], on either side."""
    gen = torch.Generator().manual_seed(1)
    for shape in ((12, 40), (40, 12), (2, 9, 9)):
        g = torch.randn(*shape, generator=gen, dtype=torch.float64)
        x = A.newton_schulz(g, 5, (3.4445, -4.7750, 2.0315), 1e-7)
        s0, s1 = torch.linalg.svdvals(g), torch.linalg.svdvals(x)
        kept = (s0 > 0.05 * s0.amax(-1, keepdim=True)).flip(-1)
        assert bool(((s1 < 1.21) & (s1 > 0.68)).all()) or bool(((s1 > 0.68).sum(-1) >= kept.sum(-1)).all())
        p = A.newton_schulz(-2.0 * g.transpose(-2, -1), 5, (3.4445, -4.7750, 2.0315), 0.0)
        assert torch.allclose(p.transpose(-2, -1), -x, atol=1e-5)


def test_newton_schulz_python_checks():
    for call in (lambda: ops.newton_schulz(torch.zeros(3, 4)),):
        with pytest.raises(NvFp4Error):
            call()
    with pytest.raises(TypeError):
        ops.newton_schulz([1.0])
