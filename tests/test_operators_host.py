"""Refusals of the operators on unquantized tensors: every invalid argument is
rejected on the host before any HIP call (no GPU needed)."""
import ctypes as C
import os

import pytest
import torch

from nvfp4_w4a4_quantized_amd import _lib, ops
from nvfp4_w4a4_quantized_amd._lib import NvFp4Error, Weights

INVALID, UNSUPPORTED, WS_SMALL = 1, 2, 4
F = C.c_void_p(0x1000)       # never dereferenced: validation fails first
ODD = C.c_void_p(0x1001)
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("library not built (run __graft_entry__.build())")
    return _lib.lib()


def change(good, i, v):
    a = list(good)
    a[i] = v
    return a


def test_router(L):
    # logits, dtype, tokens, experts, ld, bias, topk, score, renorm, scale, idx, prob, stream
    good = [F, 1, 4, 60, 60, None, 6, 0, 1, 1.0, F, F, None]
    for i, v in ((0, None), (0, ODD), (1, 3), (1, -1), (2, -1), (3, 0), (3, 1025), (4, 59), (5, ODD),
                 (6, 0), (6, 61), (7, 2), (8, 2), (9, NAN), (9, INF), (10, None), (10, ODD),
                 (11, None), (11, ODD), (2, 1 << 40)):
        assert L.moe_router(*change(good, i, v)) == INVALID, (i, v)
    # logits, dtype, tokens, experts, ld, idx, dprob, topk, score, renorm, scale, dlogits, stream
    good = [F, 0, 4, 60, 60, F, F, 6, 0, 1, 1.0, F, None]
    for i, v in ((0, None), (1, 3), (2, -1), (3, 0), (3, 1025), (4, 59), (5, None), (5, ODD),
                 (6, None), (6, ODD), (7, 0), (7, 61), (8, -1), (9, -1), (10, NAN), (11, None),
                 (11, ODD), (2, 1 << 40)):
        assert L.moe_router_backward(*change(good, i, v)) == INVALID, (i, v)


def test_sort_and_unsort(L):
    # x, dtype, T, H, ld, dst, prob, k, row_src, offsets, E, cap, rows, stream
    good = [F, 1, 4, 48, 48, F, None, 2, F, F, 8, 8, F, None]
    for i, v in ((0, None), (0, ODD), (1, 3), (2, -1), (3, 0), (4, 47), (5, None), (5, ODD), (6, ODD),
                 (7, 0), (8, None), (9, None), (9, ODD), (10, 0), (10, 1025), (11, -1),
                 (11, 1 << 31), (12, None), (12, ODD), (2, 1 << 31)):
        assert L.moe_sort_tokens(*change(good, i, v)) == INVALID, (i, v)
    # drows, dtype, T, H, ld_rows, cap, dst, prob, k, x, ld_x, dx, dprob, stream
    good = [F, 1, 4, 48, 48, 8, F, None, 2, F, 48, F, F, None]
    for i, v in ((0, None), (0, ODD), (1, -1), (2, -1), (3, 0), (4, 47), (5, -1), (5, 1 << 31),
                 (6, None), (7, ODD), (8, 0), (9, None), (9, ODD), (10, 47), (11, None), (11, ODD),
                 (12, ODD)):
        assert L.moe_sort_tokens_backward(*change(good, i, v)) == INVALID, (i, v)
    # rows, dtype, T, H, ld_rows, cap, dst, prob, k, y, stream
    good = [F, 2, 4, 48, 48, 8, F, None, 2, F, None]
    for i, v in ((0, None), (0, ODD), (1, 7), (2, -1), (3, 0), (4, 47), (5, -1), (6, None), (6, ODD),
                 (7, ODD), (8, 0), (9, None), (9, ODD)):
        assert L.moe_unsort_tokens(*change(good, i, v)) == INVALID, (i, v)
    # dy, dtype, T, H, ld_dy, dst, prob, k, row_src, offsets, E, cap, rows, ld_rows, drows, dprob, s
    good = [F, 0, 4, 48, 48, F, None, 2, F, F, 8, 8, F, 48, F, F, None]
    for i, v in ((0, None), (0, ODD), (1, 3), (2, -1), (3, 0), (4, 47), (5, None), (7, 0), (8, None),
                 (9, None), (10, 0), (11, -1), (12, None), (12, ODD), (13, 47), (14, None),
                 (14, ODD), (15, ODD)):
        assert L.moe_unsort_tokens_backward(*change(good, i, v)) == INVALID, (i, v)
    assert L.moe_sort_tokens(*change(change([F, 1, 4, 48, 48, F, None, 2, F, F, 8, 8, F, None],
                                            3, 1 << 32), 4, 1 << 32)) == UNSUPPORTED


def test_matvec(L):
    w, tiled = Weights(0x1000, 0x1000, 0x1000, 0), Weights(0x1000, 0x1000, 0x1000, 1)
    # x, dtype, T, ld, w, n, k, out_dtype, out, stream
    good = [F, 1, 4, 256, C.byref(w), 64, 256, 1, F, None]
    for i, v in ((0, None), (0, ODD), (1, 3), (2, -1), (3, 255), (4, None),
                 (4, C.byref(Weights(0, 0x1000, 0x1000, 0))), (4, C.byref(Weights(0x1000, 0, 0x1000, 0))),
                 (4, C.byref(Weights(0x1000, 0x1000, 0, 0))), (4, C.byref(Weights(0x1000, 0x1000, 0x1001, 0))),
                 (4, C.byref(Weights(0x1000, 0x1000, 0x1000, 2))),
                 (4, C.byref(Weights(0x1008, 0x1000, 0x1000, 1))), (5, 0), (6, 8), (6, 250), (7, 3),
                 (8, None), (8, ODD)):
        assert L.nvfp4_matvec(*change(good, i, v)) == INVALID, (i, v)
    for n, k, x in ((1 << 24, 256, w), (64, 16400, w), (48, 256, tiled), (64, 144, tiled)):
        a = [F, 1, 4, k, C.byref(x), n, k, 1, F, None]
        assert L.nvfp4_matvec(*a) == UNSUPPORTED, (n, k)
    assert L.nvfp4_matvec(*change(good, 2, 65537)) == UNSUPPORTED
    # x, dtype, T, ld, by_entry, idx, topk, w, E, n, k, out_dtype, out, stream
    good = [F, 1, 4, 256, 0, F, 2, C.byref(w), 8, 64, 256, 1, F, None]
    for i, v in ((0, None), (0, ODD), (1, -1), (2, -1), (3, 255), (4, 2), (5, None), (5, ODD), (6, 0),
                 (7, None), (8, 0), (8, 1025), (9, 0), (10, 24), (11, 3), (12, None), (12, ODD)):
        assert L.nvfp4_expert_matvec(*change(good, i, v)) == INVALID, (i, v)
    assert L.nvfp4_expert_matvec(*change(good, 2, 2049)) == UNSUPPORTED


def test_decode(L):
    w, tiled = Weights(0x1000, 0x1000, 0x1000, 0), Weights(0x1000, 0x1000, 0x1000, 1)
    # x, dtype, T, H, I, ld, idx, prob, topk, E, w1, w2, y, ws, ws_bytes, stream
    good = [F, 1, 4, 256, 128, 256, F, F, 2, 8, C.byref(w), C.byref(w), F, F, 1 << 30, None]
    for i, v in ((0, None), (0, ODD), (1, 3), (2, -1), (5, 255), (6, None), (6, ODD), (7, None),
                 (7, ODD), (8, 0), (8, 9), (9, 0), (9, 1025), (10, None), (11, None), (12, None),
                 (12, ODD), (13, None), (13, C.c_void_p(0x1008))):
        assert L.moe_expert_decode(*change(good, i, v)) == INVALID, (i, v)
    for i, v in ((2, 2049), (3, 200), (3, 16400), (4, 8), (4, 100), (4, 16400)):
        a = change(good, i, v)
        a[5] = max(a[5], a[3])
        assert L.moe_expert_decode(*a) == UNSUPPORTED, (i, v)
    a = change(change(good, 4, 48), 10, C.byref(tiled))      # 2 * 48 rows are not whole tiles
    assert L.moe_expert_decode(*a) == UNSUPPORTED
    size = L.moe_expert_decode_workspace_size(4, 256, 128, 2)
    assert size >= 8 * (128 * 4 + 256 * 4)
    assert L.moe_expert_decode(*change(good, 14, size - 1)) == WS_SMALL
    assert L.moe_expert_decode_workspace_size(2049, 256, 128, 2) == 0
    assert L.moe_expert_decode(*change(good, 2, 0)) == 0     # no tokens: nothing to do


def test_python_checks():
    """The binding refuses host tensors, other dtypes, shapes and layouts."""
    x = torch.zeros(4, 48, dtype=torch.bfloat16)
    for call in (lambda: ops.moe_router(x, 2), lambda: ops.moe_unsort_tokens(x, x),
                 lambda: ops.nvfp4_matvec(x, ops.NvFp4Weights(x, x, x)),
                 lambda: ops.moe_sort_tokens(x, x, x, x)):
        with pytest.raises(NvFp4Error):
            call()
    with pytest.raises(TypeError):
        ops.moe_router([1.0], 1)
    with pytest.raises(TypeError):
        ops.nvfp4_matvec(x, x)


def test_router_score_bias(L):
    # logits, dtype, tokens, experts, ld, score bias, topk, score, renorm, scale, idx, prob, stream
    good = [F, 1, 4, 60, 60, F, 6, 1, 1, 1.0, F, F, None]
    for i, v in ((0, None), (0, ODD), (1, 3), (2, -1), (3, 0), (3, 1025), (4, 59), (5, None), (5, ODD),
                 (6, 0), (6, 61), (7, 2), (8, 2), (9, NAN), (10, None), (11, ODD), (2, 1 << 40)):
        assert L.moe_router_score_bias(*change(good, i, v)) == INVALID, (i, v)
