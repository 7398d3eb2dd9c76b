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
