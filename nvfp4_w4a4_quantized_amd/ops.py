"""Python entry points with the names of the C ABI (include/nvfp4moe.h).

Each function validates tensor devices/dtypes, allocates the outputs with
torch on the input's device, and calls the library on the current stream.
bf16 activations may be passed as torch.bfloat16 or as int16/uint16 bit
patterns; codes and scales are uint8, outer scales float32, indices int32.
"""
from __future__ import annotations

import ctypes as C

import torch

from ._lib import (BackwardIntermediates, Intermediates, NvFp4Error, SinglePassIntermediates,
                   Weights, check, lib, ptr, stream_handle)

__all__ = ["nvfp4_quantize", "moe_rows_capacity", "moe_permute", "moe_permute_noalloc",
           "w4a4_grouped_gemm",
           "w4a4_grouped_gemm_swiglu", "moe_combine", "moe_expert_forward",
           "moe_expert_forward_workspace_size", "moe_expert_forward_single_pass",
           "moe_expert_forward_single_pass_workspace_size", "moe_expert_backward",
           "moe_expert_backward_workspace_size", "SINGLE_PASS_TILE", "NvFp4Weights",
           "StageTimer", "BackwardTimer", "moe_router", "moe_router_backward",
           "moe_sort_tokens", "moe_sort_tokens_backward", "moe_unsort_tokens",
           "moe_unsort_tokens_backward", "nvfp4_matvec", "nvfp4_expert_matvec",
           "moe_expert_decode", "moe_expert_decode_workspace_size", "lora_forward",
           "lora_forward_workspace_size", "lora_backward", "lora_backward_workspace_size",
           "nvfp4_lora_matvec", "nvfp4_lora_matvec_workspace_size", "newton_schulz",
           "newton_schulz_workspace_size"]

SINGLE_PASS_TILE = 256   # intermediate columns per online-scale tile of the single-pass layer

_BF16_LIKE = (torch.bfloat16, torch.int16, torch.uint16)


def _need(t, dtypes, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise NvFp4Error(f"{name} must be a device tensor (got {t.device})")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


class NvFp4Weights:
    """NVFP4 expert weights: codes [G, N, K/2] u8, scales [G, N, K/16] u8,
    gscale [G] f32 (one outer scale per expert matrix).  layout 0 is
    row-major; layout 1 holds the same bytes in the grouped GEMM's tiled
    order (nvfp4_pack_weights), the tensor shapes unchanged."""

    def __init__(self, codes, scales, gscale, layout: int = 0):
        self.codes, self.scales, self.gscale = codes, scales, gscale
        self.layout = layout

    def packed(self) -> "NvFp4Weights":
        """The tiled copy of row-major weights (static weights: done once)."""
        if self.layout != 0:
            raise ValueError("weights are already in the tiled layout")
        G, N, kh = self.codes.shape
        pc = torch.empty_like(self.codes)
        ps = torch.empty_like(self.scales)
        check(lib().nvfp4_pack_weights(ptr(self.codes), ptr(self.scales), G, N, kh * 2, ptr(pc),
                                       ptr(ps), stream_handle()), "nvfp4_pack_weights")
        return NvFp4Weights(pc, ps, self.gscale, layout=1)

    @classmethod
    def quantize(cls, w_bf16: torch.Tensor, block_rule: int = 0,
                 blocks_2d: bool = False) -> "NvFp4Weights":
        """Quantizes bf16 weights [G, N, K] with one outer scale per expert
        (block_rule: see nvfp4_quantize; blocks_2d: 16x16 blocks, N % 16 == 0)."""
        G, N, K = w_bf16.shape
        offs = (torch.arange(G + 1, dtype=torch.int32, device=w_bf16.device) * N)
        codes, scales, gscale = nvfp4_quantize(w_bf16.reshape(G * N, K),
                                               scale_domain=2 if blocks_2d else 1,
                                               block_rule=block_rule,
                                               group_offsets=offs)
        return cls(codes.view(G, N, K // 2), scales.view(G, N, K // 16), gscale)

    def c_struct(self) -> Weights:
        return Weights(self.codes.data_ptr(), self.scales.data_ptr(), self.gscale.data_ptr(),
                       self.layout)


def nvfp4_quantize(x, scale_domain: int = 0, group_offsets=None, amax_in=None,
                   block_rule: int = 0, out=None):
    """NVFP4 quantization of a bf16 [rows, k] matrix.  Returns (codes, scales,
    global_scales) with global_scales per row (domain 0) or per group (1).
    block_rule 0: every block maximum maps to 6; 1 / 2: Four-Over-Six with the
    block error measured as a sum of squares / of absolute values.  `out` may
    supply the three output tensors (contiguous, of those shapes)."""
    _need(x, _BF16_LIKE, "x")
    rows, k = x.shape
    dev = x.device
    ng = 0
    if scale_domain in (1, 2):
        _need(group_offsets, (torch.int32,), "group_offsets")
        ng = group_offsets.numel() - 1
    shapes = ((rows, k // 2), (rows, k // 16), (ng if scale_domain in (1, 2) else rows,))
    if out is None:
        codes = torch.empty(shapes[0], dtype=torch.uint8, device=dev)
        scales = torch.empty(shapes[1], dtype=torch.uint8, device=dev)
        gs = torch.empty(shapes[2], dtype=torch.float32, device=dev)
    else:
        codes, scales, gs = out
        for t, n, d, shp in ((codes, "codes", torch.uint8, shapes[0]),
                             (scales, "scales", torch.uint8, shapes[1]),
                             (gs, "global_scales", torch.float32, shapes[2])):
            _need(t, (d,), n)
            if tuple(t.shape) != shp:
                raise ValueError(f"{n}: shape {tuple(t.shape)}, expected {shp}")
    if amax_in is not None:
        _need(amax_in, (torch.float32,), "amax_in")
    check(lib().nvfp4_quantize(ptr(x), rows, k, k, scale_domain, ptr(group_offsets), ng,
                               ptr(amax_in), block_rule, ptr(codes), ptr(scales), ptr(gs),
                               stream_handle()),
          "nvfp4_quantize")
    return codes, scales, gs


def moe_rows_capacity(tokens: int, topk: int, num_experts: int, align: int = 1) -> int:
    return int(lib().moe_rows_capacity(tokens, topk, num_experts, align))


def moe_permute(x, topk_idx, topk_prob, num_experts: int, align: int = 1, block_rule: int = 0,
                workspace=None, library=None):
    """Routing metadata + per-token quantize-scatter.  x may be None (metadata
    only).  Returns a dict of device tensors.  `workspace`: a uint8 device
    tensor of at least moe_permute_workspace_size bytes (allocated here when
    None); `library`: the loaded library to call (the release build by
    default, _lib.debug_lib() for the precondition-checking build)."""
    L = library if library is not None else lib()
    _need(topk_idx, (torch.int32,), "topk_idx")
    _need(topk_prob, (torch.float32,), "topk_prob")
    T, k = topk_idx.shape
    dev = topk_idx.device
    cap = moe_rows_capacity(T, k, num_experts, align)
    out = dict(
        offsets=torch.empty(num_experts + 1, dtype=torch.int32, device=dev),
        dst_row=torch.empty((T, k), dtype=torch.int32, device=dev),
        row_src=torch.empty(cap, dtype=torch.int32, device=dev),
        row_prob=torch.empty(cap, dtype=torch.float32, device=dev))
    H = 0
    if x is not None:
        _need(x, _BF16_LIKE, "x")
        H = x.shape[1]
        out["codes"] = torch.empty((cap, H // 2), dtype=torch.uint8, device=dev)
        out["scales"] = torch.empty((cap, H // 16), dtype=torch.uint8, device=dev)
        out["gscale"] = torch.empty(cap, dtype=torch.float32, device=dev)
    wsb = int(L.moe_permute_workspace_size(T, k, num_experts))
    ws = workspace if workspace is not None else torch.empty(max(wsb, 256), dtype=torch.uint8,
                                                             device=dev)
    _need(ws, (torch.uint8,), "workspace")
    check(L.moe_permute(ptr(x), T, H, ptr(topk_idx), ptr(topk_prob), k, num_experts, align,
                            block_rule, ptr(out["offsets"]), ptr(out["dst_row"]), ptr(out["row_src"]),
                            ptr(out["row_prob"]), ptr(out.get("codes")), ptr(out.get("scales")),
                            ptr(out.get("gscale")), ptr(ws), ws.numel(), stream_handle()),
          "moe_permute")
    return out


def moe_permute_noalloc(x, topk_idx, topk_prob, num_experts: int, align: int = 1,
                        block_rule: int = 0, out=None):
    """moe_permute through the entry point that allocates nothing: the routing
    scratch is the library's static device array.  `out`: a dict of output
    tensors shaped as moe_permute returns them (allocated here when None;
    the library call itself allocates nothing).  Returns that dict."""
    _need(topk_idx, (torch.int32,), "topk_idx")
    _need(topk_prob, (torch.float32,), "topk_prob")
    T, k = topk_idx.shape
    dev = topk_idx.device
    cap = moe_rows_capacity(T, k, num_experts, align)
    H = 0
    if x is not None:
        _need(x, _BF16_LIKE, "x")
        H = x.shape[1]
    if out is None:
        out = dict(
            offsets=torch.empty(num_experts + 1, dtype=torch.int32, device=dev),
            dst_row=torch.empty((T, k), dtype=torch.int32, device=dev),
            row_src=torch.empty(cap, dtype=torch.int32, device=dev),
            row_prob=torch.empty(cap, dtype=torch.float32, device=dev))
        if x is not None:
            out["codes"] = torch.empty((cap, H // 2), dtype=torch.uint8, device=dev)
            out["scales"] = torch.empty((cap, H // 16), dtype=torch.uint8, device=dev)
            out["gscale"] = torch.empty(cap, dtype=torch.float32, device=dev)
    check(lib().moe_permute_noalloc(ptr(x), T, H, ptr(topk_idx), ptr(topk_prob), k, num_experts,
                                    align, block_rule, ptr(out["offsets"]), ptr(out["dst_row"]),
                                    ptr(out["row_src"]), ptr(out["row_prob"]),
                                    ptr(out.get("codes")), ptr(out.get("scales")),
                                    ptr(out.get("gscale")), stream_handle()),
          "moe_permute_noalloc")
    return out


def _gemm_common(a_codes, a_scales, a_gscale, b, group_offsets):
    for t, n, d in ((a_codes, "a_codes", (torch.uint8,)), (a_scales, "a_scales", (torch.uint8,)),
                    (a_gscale, "a_gscale", (torch.float32,)), (b.codes, "b_codes", (torch.uint8,)),
                    (b.scales, "b_scales", (torch.uint8,)), (b.gscale, "b_gscale", (torch.float32,)),
                    (group_offsets, "group_offsets", (torch.int32,))):
        _need(t, d, n)
    G, N, kh = b.codes.shape
    return a_codes.shape[0], G, N, kh * 2


def w4a4_grouped_gemm(a_codes, a_scales, a_gscale, b: NvFp4Weights, group_offsets,
                      out_dtype=torch.float32, out=None):
    rows_cap, G, N, K = _gemm_common(a_codes, a_scales, a_gscale, b, group_offsets)
    code = 0 if out_dtype == torch.float32 else 1
    if out is None:
        out = torch.empty((rows_cap, N), dtype=out_dtype, device=a_codes.device)
    else:
        _need(out, (out_dtype,), "out")
        if tuple(out.shape) != (rows_cap, N):
            raise ValueError(f"out: shape {tuple(out.shape)}, expected {(rows_cap, N)}")
    check(lib().w4a4_grouped_gemm(ptr(a_codes), ptr(a_scales), ptr(a_gscale), rows_cap,
                                  ptr(b.codes), ptr(b.scales), ptr(b.gscale), ptr(group_offsets),
                                  G, N, K, b.layout, code, ptr(out), stream_handle()),
          "w4a4_grouped_gemm")
    return out


def w4a4_grouped_gemm_swiglu(a_codes, a_scales, a_gscale, b: NvFp4Weights, group_offsets,
                             row_prob, with_c: bool = False):
    """FC1 with the weighted SwiGLU epilogue.  Returns (D bf16 [cap, I],
    amax f32 [cap], C f32 [cap, 2I] or None)."""
    rows_cap, G, N2, K = _gemm_common(a_codes, a_scales, a_gscale, b, group_offsets)
    _need(row_prob, (torch.float32,), "row_prob")
    inter = N2 // 2
    dev = a_codes.device
    d = torch.empty((rows_cap, inter), dtype=torch.bfloat16, device=dev)
    amax = torch.zeros(rows_cap, dtype=torch.float32, device=dev)
    c = torch.empty((rows_cap, N2), dtype=torch.float32, device=dev) if with_c else None
    check(lib().w4a4_grouped_gemm_swiglu(ptr(a_codes), ptr(a_scales), ptr(a_gscale), rows_cap,
                                         ptr(b.codes), ptr(b.scales), ptr(b.gscale),
                                         ptr(group_offsets), G, inter, K, b.layout,
                                         ptr(row_prob), ptr(d),
                                         ptr(amax), ptr(c), stream_handle()),
          "w4a4_grouped_gemm_swiglu")
    return d, amax, c


def moe_combine(y_rows, dst_row):
    _need(y_rows, (torch.float32, torch.bfloat16), "y_rows")
    _need(dst_row, (torch.int32,), "dst_row")
    T, k = dst_row.shape
    H = y_rows.shape[1]
    y = torch.empty((T, H), dtype=torch.bfloat16, device=y_rows.device)
    check(lib().moe_combine(ptr(y_rows), 0 if y_rows.dtype == torch.float32 else 1, ptr(dst_row),
                            T, k, H, ptr(y), stream_handle()), "moe_combine")
    return y


def moe_expert_forward_workspace_size(tokens, hidden, inter, topk, num_experts, align=1) -> int:
    return int(lib().moe_expert_forward_workspace_size(tokens, hidden, inter, topk, num_experts,
                                                       align))


class StageTimer:
    """Six HIP events recorded by moe_expert_forward at its stage boundaries:
    route+quantize, FC1+SwiGLU, requantize, FC2, combine."""

    NAMES = ("route_quantize", "fc1_swiglu", "requantize", "fc2", "combine")

    def __init__(self):
        L = lib()
        self.events = (C.c_void_p * 6)()
        for i in range(6):
            h = C.c_void_p()
            check(L.nvfp4_event_create(C.byref(h)), "nvfp4_event_create")
            self.events[i] = h.value

    def elapsed_ms(self):
        out = {}
        ms = C.c_float()
        for i, n in enumerate(self.NAMES):
            check(lib().nvfp4_event_elapsed_ms(self.events[i], self.events[i + 1], C.byref(ms)),
                  "nvfp4_event_elapsed_ms")
            out[n] = ms.value
        return out

    def close(self):
        for i in range(6):
            if self.events[i]:
                lib().nvfp4_event_destroy(self.events[i])
                self.events[i] = None


def moe_expert_forward(x, topk_idx, topk_prob, num_experts: int, inter: int,
                       w1: NvFp4Weights, w2: NvFp4Weights, align: int = 1, workspace=None,
                       debug: bool = False, fc1_out: bool = False, y_rows_f32: bool = False,
                       timer: StageTimer | None = None, y=None, act_block_rule: int = 0,
                       act_scale_domain: int = 0, library=None):
    """The whole expert layer.  Returns y (bf16 [T, H]); with debug=True also a
    dict of the intermediates (allocated here, written by the library).
    act_scale_domain: 0 one activation outer scale per token, 1 per tensor.
    `library`: the loaded library to call (release build by default)."""
    L = library if library is not None else lib()
    _need(x, _BF16_LIKE, "x")
    _need(topk_idx, (torch.int32,), "topk_idx")
    _need(topk_prob, (torch.float32,), "topk_prob")
    T, H = x.shape
    k = topk_idx.shape[1]
    dev = x.device
    wsb = int(L.moe_expert_forward_workspace_size(T, H, inter, k, num_experts, align))
    if workspace is None:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=dev)
    if y is None:
        y = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    dbg = None
    inter_t = None
    if debug:
        cap = moe_rows_capacity(T, k, num_experts, align)
        e = lambda shape, dt: torch.empty(shape, dtype=dt, device=dev)  # noqa: E731
        inter_t = dict(
            expert_offsets=e(num_experts + 1, torch.int32), dst_row=e((T, k), torch.int32),
            row_src=e(cap, torch.int32), row_prob=e(cap, torch.float32),
            a1_codes=e((cap, H // 2), torch.uint8), a1_scales=e((cap, H // 16), torch.uint8),
            a1_gscale=e(cap, torch.float32), d=e((cap, inter), torch.bfloat16),
            amax_d=e(cap, torch.float32), a2_codes=e((cap, inter // 2), torch.uint8),
            a2_scales=e((cap, inter // 16), torch.uint8), a2_gscale=e(cap, torch.float32),
            y_rows=e((cap, H), torch.bfloat16))
        if fc1_out:
            inter_t["fc1_out"] = e((cap, 2 * inter), torch.float32)
        if y_rows_f32:
            inter_t["y_rows_f32"] = e((cap, H), torch.float32)
        dbg = Intermediates(**{n: t.data_ptr() for n, t in inter_t.items()})
    ev = timer.events if timer is not None else None
    check(L.moe_expert_forward(ptr(x), T, H, inter, ptr(topk_idx), ptr(topk_prob), k,
                                   num_experts, align, act_block_rule, act_scale_domain,
                                   C.byref(w1.c_struct()),
                                   C.byref(w2.c_struct()), ptr(y), ptr(workspace),
                                   workspace.numel(), C.byref(dbg) if dbg is not None else None,
                                   C.cast(ev, C.c_void_p) if ev is not None else None,
                                   stream_handle()), "moe_expert_forward")
    if debug:
        return y, inter_t
    return y


class SinglePassTimer(StageTimer):
    """Four HIP events recorded by moe_expert_forward_single_pass: routing +
    quantize, the fused FC1 -> SwiGLU -> quantize -> FC2 kernel, combine."""

    NAMES = ("route_quantize", "fused_fc1_fc2", "combine")

    def __init__(self):
        L = lib()
        self.events = (C.c_void_p * 4)()
        for i in range(4):
            h = C.c_void_p()
            check(L.nvfp4_event_create(C.byref(h)), "nvfp4_event_create")
            self.events[i] = h.value

    def close(self):
        for i in range(4):
            if self.events[i]:
                lib().nvfp4_event_destroy(self.events[i])
                self.events[i] = None


def moe_expert_forward_single_pass_workspace_size(tokens, hidden, inter, topk, num_experts,
                                                  align=1) -> int:
    return int(lib().moe_expert_forward_single_pass_workspace_size(tokens, hidden, inter, topk,
                                                                   num_experts, align))


def moe_expert_forward_single_pass(x, topk_idx, topk_prob, num_experts: int, inter: int,
                                   w1: NvFp4Weights, w2: NvFp4Weights, align: int = 1,
                                   workspace=None, debug: bool = False, fc1_out: bool = False,
                                   y_rows_f32: bool = False, timer=None, y=None):
    """The expert layer with the single-pass FC1 -> SwiGLU -> quantize -> FC2
    kernel (online amax compensation, tiles of SINGLE_PASS_TILE columns).
    Returns y (bf16 [T, H]); with debug=True also a dict of the intermediates:
    routing maps, a1 rows, fc1_out (if asked), p (bf16 weighted SwiGLU),
    a2_codes / a2_scales (the online quantization), gs_tiles, y_rows (bf16, or
    y_rows_f32 if asked)."""
    _need(x, _BF16_LIKE, "x")
    _need(topk_idx, (torch.int32,), "topk_idx")
    _need(topk_prob, (torch.float32,), "topk_prob")
    T, H = x.shape
    k = topk_idx.shape[1]
    dev = x.device
    wsb = moe_expert_forward_single_pass_workspace_size(T, H, inter, k, num_experts, align)
    if workspace is None:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=dev)
    if y is None:
        y = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
    dbg = None
    inter_t = None
    if debug:
        cap = moe_rows_capacity(T, k, num_experts, align)
        nt = (inter + SINGLE_PASS_TILE - 1) // SINGLE_PASS_TILE
        e = lambda shape, dt: torch.zeros(shape, dtype=dt, device=dev)  # noqa: E731
        inter_t = dict(
            expert_offsets=e(num_experts + 1, torch.int32), dst_row=e((T, k), torch.int32),
            row_src=e(cap, torch.int32), row_prob=e(cap, torch.float32),
            a1_codes=e((cap, H // 2), torch.uint8), a1_scales=e((cap, H // 16), torch.uint8),
            a1_gscale=e(cap, torch.float32), p=e((cap, inter), torch.bfloat16),
            a2_codes=e((cap, inter // 2), torch.uint8), a2_scales=e((cap, inter // 16), torch.uint8),
            gs_tiles=e((cap, nt), torch.float32), y_rows=e((cap, H), torch.bfloat16))
        if fc1_out:
            inter_t["fc1_out"] = e((cap, 2 * inter), torch.float32)
        if y_rows_f32:
            inter_t["y_rows_f32"] = e((cap, H), torch.float32)
        dbg = SinglePassIntermediates(**{n: t.data_ptr() for n, t in inter_t.items()})
    ev = timer.events if timer is not None else None
    check(lib().moe_expert_forward_single_pass(
        ptr(x), T, H, inter, ptr(topk_idx), ptr(topk_prob), k, num_experts, align,
        C.byref(w1.c_struct()), C.byref(w2.c_struct()), ptr(y), ptr(workspace), workspace.numel(),
        C.byref(dbg) if dbg is not None else None,
        C.cast(ev, C.c_void_p) if ev is not None else None, stream_handle()),
        "moe_expert_forward_single_pass")
    if debug:
        return y, inter_t
    return y



class BackwardTimer(StageTimer):
    """Eight HIP events recorded by moe_expert_backward around its stages, in
    the order they run: the dgrad tile tables, FC2 dgrad, the SwiGLU
    backward, FC1 dgrad, the dx / dprob reductions, FC2 wgrad, FC1 wgrad."""

    NAMES = ("tables", "fc2_dgrad", "swiglu_bwd", "fc1_dgrad", "reduce", "fc2_wgrad",
             "fc1_wgrad")

    def __init__(self):
        L = lib()
        self.events = (C.c_void_p * 8)()
        for i in range(8):
            h = C.c_void_p()
            check(L.nvfp4_event_create(C.byref(h)), "nvfp4_event_create")
            self.events[i] = h.value

    def close(self):
        for i in range(8):
            if self.events[i]:
                lib().nvfp4_event_destroy(self.events[i])
                self.events[i] = None


def moe_expert_backward_workspace_size(rows_cap, hidden, inter, num_experts) -> int:
    return int(lib().moe_expert_backward_workspace_size(rows_cap, hidden, inter, num_experts))


def moe_expert_backward(dy, x, fc1_out, d, expert_offsets, row_src, row_prob, dst_row,
                        w1, w2, workspace=None, debug: bool = False,
                        dx_rows_f32: bool = False, timer: BackwardTimer | None = None,
                        out=None):
    """Gradients of the expert layer (straight-through, BF16 GEMMs).
    dy, x: bf16 [T, H]; fc1_out: fp32 [cap, 2I] and d: bf16 [cap, I], the
    forward's FC1 output and FC2 input; the forward's routing arrays; w1 bf16
    [E, 2I, H], w2 bf16 [E, H, I].  Returns dict(dx, dw1, dw2, dprob); with
    debug=True a second dict of the intermediates (dd, dc, dp_rows, dx_rows,
    and dx_rows_f32 if asked).  `out`: optional dict of preallocated outputs
    with those four names."""
    for t, n in ((dy, "dy"), (x, "x"), (d, "d"), (w1, "w1"), (w2, "w2")):
        _need(t, _BF16_LIKE, n)
    _need(fc1_out, (torch.float32,), "fc1_out")
    _need(row_prob, (torch.float32,), "row_prob")
    for t, n in ((expert_offsets, "expert_offsets"), (row_src, "row_src"), (dst_row, "dst_row")):
        _need(t, (torch.int32,), n)
    T, H = dy.shape
    E = w1.shape[0]
    inter = w2.shape[2]
    k = dst_row.shape[1]
    cap = d.shape[0]
    if (tuple(x.shape) != (T, H) or tuple(fc1_out.shape) != (cap, 2 * inter)
            or tuple(d.shape) != (cap, inter) or tuple(w1.shape) != (E, 2 * inter, H)
            or tuple(w2.shape) != (E, H, inter) or expert_offsets.numel() != E + 1
            or row_src.numel() < cap or row_prob.numel() < cap or dst_row.shape[0] != T):
        raise NvFp4Error("moe_expert_backward: inconsistent shapes")
    dev = dy.device
    L = lib()
    wsb = int(L.moe_expert_backward_workspace_size(cap, H, inter, E))
    if workspace is None:
        workspace = torch.empty(max(wsb, 1), dtype=torch.uint8, device=dev)
    if out is None:
        out = dict(dx=torch.empty((T, H), dtype=torch.bfloat16, device=dev),
                   dw1=torch.empty((E, 2 * inter, H), dtype=torch.float32, device=dev),
                   dw2=torch.empty((E, H, inter), dtype=torch.float32, device=dev),
                   dprob=torch.empty((T, k), dtype=torch.float32, device=dev))
    dbg = None
    inter_t = None
    if debug:
        e = lambda shape, dt: torch.empty(shape, dtype=dt, device=dev)  # noqa: E731
        inter_t = dict(dd=e((cap, inter), torch.bfloat16), dc=e((cap, 2 * inter), torch.bfloat16),
                       dp_rows=e(cap, torch.float32), dx_rows=e((cap, H), torch.bfloat16))
        if dx_rows_f32:
            inter_t["dx_rows_f32"] = e((cap, H), torch.float32)
        dbg = BackwardIntermediates(**{n: t.data_ptr() for n, t in inter_t.items()})
    ev = timer.events if timer is not None else None
    check(L.moe_expert_backward(ptr(dy), ptr(x), T, H, inter, k, E, cap, ptr(fc1_out), ptr(d),
                                ptr(expert_offsets), ptr(row_src), ptr(row_prob), ptr(dst_row),
                                ptr(w1), ptr(w2), ptr(out["dx"]), ptr(out["dw1"]),
                                ptr(out["dw2"]), ptr(out["dprob"]), ptr(workspace),
                                workspace.numel(), C.byref(dbg) if dbg is not None else None,
                                C.cast(ev, C.c_void_p) if ev is not None else None,
                                stream_handle()), "moe_expert_backward")
    if debug:
        return out, inter_t
    return out


# ---- operators on unquantized tensors --------------------------------------
# Their tensors are float32, bfloat16 or float16; rows may be strided (a last
# dimension of stride 1), outputs are contiguous.  Calls run on the current
# stream of the operands' own device.

_DTYPE_CODE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _need_rows(t, name, width=None, dtype=None):
    """A [rows, width] tensor of an element type, its last dimension dense.
    Returns the distance of its rows in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise NvFp4Error(f"{name} must be a device tensor (got {t.device})")
    have = t.dtype
    if have not in _DTYPE_CODE or (dtype is not None and have != dtype):
        raise TypeError(f"{name}: dtype {have}, expected "
                        f"{dtype if dtype is not None else tuple(_DTYPE_CODE)}")
    if t.dim() != 2 or (width is not None and t.shape[1] != width):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected [rows, "
                         f"{'width' if width is None else width}]")
    n, w = t.shape
    if w < 1:
        raise ValueError(f"{name}: rows of no elements")
    s0, s1 = t.stride()
    ld = s0 if n > 1 else w
    if n > 0 and ((s1 != 1 and w > 1) or ld < w):
        raise ValueError(f"{name}: rows must be dense and must not overlap (strides {t.stride()})")
    return ld


def _dense(t, dtype, shape, dev, name):
    """A contiguous tensor of this dtype and shape on device number dev.  (The
    checks of a small call take as long as its kernel: one test where all is
    well, the reasons only where it is not.)"""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev
            and t.shape == shape and t.is_contiguous()):
        return
    _need(t, (dtype,), name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise NvFp4Error(f"{name} is on {t.device}, the call's first operand on cuda:{dev}")


def _same_device(t, dev, name):
    if t.get_device() != dev:
        raise NvFp4Error(f"{name} is on {t.device}, the call's first operand on cuda:{dev}")


def _addr(t):
    return None if t is None else t.data_ptr()


def _call(dev, what, *args):
    """The library call `what` on device number dev's current stream.  (A
    launch goes to the current device; switching, and a Stream object for the
    handle, cost as much as a small call, so neither is done without need.)"""
    stream = torch._C._cuda_getCurrentRawStream(dev)
    if dev == torch._C._cuda_getDevice():
        status = getattr(lib(), what)(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = getattr(lib(), what)(*args, stream)
    if status:
        check(status, what)


def moe_router(logits, topk: int, bias=None, score: int = 0, renormalize: bool = True,
               scale: float = 1.0, score_bias=None):
    """The top-k experts of every token and their weights, from router logits
    [T, E] (float32, bf16 or fp16).  Returns (topk_idx int32 [T, k], topk_prob
    float32 [T, k]), the arguments of moe_permute and the expert layers.
    score 0: softmax over all experts, 1: sigmoid; renormalize: divided by the
    picks' sum; scale multiplies the weights.  For the choice alone, bias
    float32 [E] is added to the logits, or score_bias float32 [E] to the scores
    (softmax or sigmoid over all experts, as a learned load-balancing correction
    is); not both.  Experts whose logit is -inf are never picked; a token with
    fewer than k left gets ids -1 with weight 0."""
    ld = _need_rows(logits, "logits")
    T, E = logits.shape
    dev = logits.get_device()
    if bias is not None:
        _dense(bias, torch.float32, (E,), dev, "bias")
    what = "moe_router"
    if score_bias is not None:
        if bias is not None:
            raise ValueError("moe_router: either bias or score_bias")
        _dense(score_bias, torch.float32, (E,), dev, "score_bias")
        what, bias = "moe_router_score_bias", score_bias
    if not 1 <= topk <= E:
        raise NvFp4Error(f"moe_router: topk {topk} of {E} experts")
    idx = logits.new_empty((T, topk), dtype=torch.int32)
    prob = logits.new_empty((T, topk), dtype=torch.float32)
    _call(dev, what, logits.data_ptr(), _DTYPE_CODE[logits.dtype], T, E, ld, _addr(bias),
          topk, score, int(bool(renormalize)), scale, idx.data_ptr(), prob.data_ptr())
    return idx, prob


def moe_router_backward(dprob, logits, topk_idx, score: int = 0, renormalize: bool = True,
                        scale: float = 1.0):
    """The logits' gradient [T, E] (their dtype) from the weights' gradient
    dprob [T, k], with moe_router's logits, ids and choices."""
    ld = _need_rows(logits, "logits")
    T, E = logits.shape
    dev = logits.get_device()
    k = _topk_of(topk_idx, T, dev)
    _dense(dprob, torch.float32, (T, k), dev, "dprob")
    out = logits.new_empty((T, E))
    _call(dev, "moe_router_backward", logits.data_ptr(), _DTYPE_CODE[logits.dtype], T, E, ld,
          topk_idx.data_ptr(), dprob.data_ptr(), k, score, int(bool(renormalize)), scale,
          out.data_ptr())
    return out


def _topk_of(ids, tokens, dev, name="topk_idx"):
    """The entries per token of an int32 [T, k] tensor."""
    if not (isinstance(ids, torch.Tensor) and ids.dim() == 2
            and (tokens is None or ids.shape[0] == tokens)):
        _need(ids, (torch.int32,), name)
        raise ValueError(f"{name}: shape {tuple(ids.shape)}, expected "
                         f"[{'T' if tokens is None else tokens}, k]")
    _dense(ids, torch.int32, ids.shape, dev, name)
    return ids.shape[1]


def _rows_out(out, like, dev, expert_offsets, row_src):
    """The routed rows' tensor, [cap, H] in like's dtype, and cap."""
    for t, n in ((expert_offsets, "expert_offsets"), (row_src, "row_src")):
        if not isinstance(t, torch.Tensor) or t.dim() != 1:
            _need(t, (torch.int32,), n)
            raise ValueError(f"{n}: shape {tuple(t.shape)}, expected one dimension")
        _dense(t, torch.int32, t.shape, dev, n)
    shape = (row_src.shape[0], like.shape[1])
    if out is None:
        return like.new_empty(shape), shape[0]
    _dense(out, like.dtype, shape, dev, "out")
    return out, shape[0]


def moe_sort_tokens(x, dst_row, row_src, expert_offsets, prob=None, out=None):
    """Tokens x [T, H] to routed rows [cap, H] in expert order, unquantized:
    rows[dst_row[t, j]] = prob[t, j] * x[t] (prob None: copies), zeros in the
    padding rows.  dst_row, row_src and expert_offsets are moe_permute's (its
    `offsets`).  Rows at or beyond the last offset are not written."""
    ld = _need_rows(x, "x")
    T, H = x.shape
    dev = x.get_device()
    k = _topk_of(dst_row, T, dev, "dst_row")
    if prob is not None:
        _dense(prob, torch.float32, (T, k), dev, "prob")
    rows, cap = _rows_out(out, x, dev, expert_offsets, row_src)
    _call(dev, "moe_sort_tokens", x.data_ptr(), _DTYPE_CODE[x.dtype], T, H, ld, dst_row.data_ptr(),
          _addr(prob), k, row_src.data_ptr(), expert_offsets.data_ptr(),
          expert_offsets.shape[0] - 1, cap, rows.data_ptr())
    return rows


def moe_sort_tokens_backward(drows, dst_row, x=None, prob=None):
    """Gradients of moe_sort_tokens from that of its rows: dx [T, H] and, with
    the forward's x given, dprob [T, k] (else None).  Returns (dx, dprob)."""
    ld = _need_rows(drows, "drows")
    cap, H = drows.shape
    dev = drows.get_device()
    k = _topk_of(dst_row, None, dev, "dst_row")
    T = dst_row.shape[0]
    if prob is not None:
        _dense(prob, torch.float32, (T, k), dev, "prob")
    ld_x, dprob = H, None
    if x is not None:
        ld_x = _need_rows(x, "x", H, drows.dtype)
        if x.shape[0] != T:
            raise ValueError(f"x: shape {tuple(x.shape)}, expected {(T, H)}")
        _same_device(x, dev, "x")
        dprob = drows.new_empty((T, k), dtype=torch.float32)
    dx = drows.new_empty((T, H))
    _call(dev, "moe_sort_tokens_backward", drows.data_ptr(), _DTYPE_CODE[drows.dtype], T, H, ld,
          cap, dst_row.data_ptr(), _addr(prob), k, _addr(x), ld_x, dx.data_ptr(), _addr(dprob))
    return dx, dprob


def moe_unsort_tokens(rows, dst_row, prob=None):
    """Routed rows [cap, H] back to tokens: y[t] = sum_j prob[t, j] *
    rows[dst_row[t, j]] (prob None: plain sums), in the rows' dtype.  Entries
    with dst_row < 0 add nothing."""
    ld = _need_rows(rows, "rows")
    cap, H = rows.shape
    dev = rows.get_device()
    k = _topk_of(dst_row, None, dev, "dst_row")
    T = dst_row.shape[0]
    if prob is not None:
        _dense(prob, torch.float32, (T, k), dev, "prob")
    y = rows.new_empty((T, H))
    _call(dev, "moe_unsort_tokens", rows.data_ptr(), _DTYPE_CODE[rows.dtype], T, H, ld, cap,
          dst_row.data_ptr(), _addr(prob), k, y.data_ptr())
    return y


def moe_unsort_tokens_backward(dy, dst_row, row_src, expert_offsets, rows=None, prob=None,
                               out=None):
    """Gradients of moe_unsort_tokens from dy [T, H]: drows [cap, H] (zeros in
    the padding rows, nothing written behind the last) and, with the forward's
    rows given, dprob [T, k] (else None).  Returns (drows, dprob)."""
    ld = _need_rows(dy, "dy")
    T, H = dy.shape
    dev = dy.get_device()
    k = _topk_of(dst_row, T, dev, "dst_row")
    if prob is not None:
        _dense(prob, torch.float32, (T, k), dev, "prob")
    drows, cap = _rows_out(out, dy, dev, expert_offsets, row_src)
    ld_rows, dprob = H, None
    if rows is not None:
        ld_rows = _need_rows(rows, "rows", H, dy.dtype)
        if rows.shape[0] != cap:
            raise ValueError(f"rows: shape {tuple(rows.shape)}, expected {(cap, H)}")
        _same_device(rows, dev, "rows")
        dprob = dy.new_empty((T, k), dtype=torch.float32)
    _call(dev, "moe_unsort_tokens_backward", dy.data_ptr(), _DTYPE_CODE[dy.dtype], T, H, ld,
          dst_row.data_ptr(), _addr(prob), k, row_src.data_ptr(), expert_offsets.data_ptr(),
          expert_offsets.shape[0] - 1, cap, _addr(rows), ld_rows, drows.data_ptr(), _addr(dprob))
    return drows, dprob


def _weights_type(*named):
    for w, name in named:
        if not isinstance(w, NvFp4Weights):
            raise TypeError(f"{name} must be NvFp4Weights")


def _need_weights(w, name, dev, groups=None, n=None, k=None):
    """NVFP4 weights whose three tensors fit each other (and the given sizes).
    Returns [G, N, K]."""
    codes = w.codes
    if not isinstance(codes, torch.Tensor) or codes.dim() != 3:
        _need(codes, (torch.uint8,), f"{name}.codes")
        raise ValueError(f"{name}.codes: shape {tuple(codes.shape)}, expected [G, N, K/2]")
    G, N, kh = codes.shape
    K = 2 * kh
    if (groups is not None and G != groups) or (n is not None and N != n) or (k is not None and K != k):
        raise ValueError(f"{name}: [G, N, K] is {(G, N, K)}, expected "
                         f"{tuple('any' if v is None else v for v in (groups, n, k))}")
    _dense(codes, torch.uint8, (G, N, kh), dev, "codes of " + name)
    _dense(w.scales, torch.uint8, (G, N, kh // 8), dev, "scales of " + name)
    _dense(w.gscale, torch.float32, (G,), dev, "gscale of " + name)
    return G, N, K


def _out_rows(out, shape, dtype, like, dev):
    if dtype not in _DTYPE_CODE:
        raise TypeError(f"out_dtype {dtype} not in {tuple(_DTYPE_CODE)}")
    if out is None:
        return like.new_empty(shape, dtype=dtype)
    _dense(out, dtype, shape, dev, "out")
    return out


def nvfp4_matvec(x, w: NvFp4Weights, out_dtype=None, out=None):
    """x [T, K] (float32, bf16 or fp16) times one NVFP4 matrix (w: [1, N, K],
    either layout): [T, N] in out_dtype (x's by default).  For the few rows of
    new tokens: the weights are read once, as they are."""
    _weights_type((w, "w"))
    ld = _need_rows(x, "x")
    T, K = x.shape
    dev = x.get_device()
    _, N, _ = _need_weights(w, "w", dev, 1, None, K)
    out = _out_rows(out, (T, N), out_dtype if out_dtype is not None else x.dtype, x, dev)
    _call(dev, "nvfp4_matvec", x.data_ptr(), _DTYPE_CODE[x.dtype], T, ld, C.byref(w.c_struct()), N,
          K, _DTYPE_CODE[out.dtype], out.data_ptr())
    return out


def nvfp4_expert_matvec(x, topk_idx, w: NvFp4Weights, out_dtype=None, out=None):
    """Every entry's row times its expert's NVFP4 matrix (w: [E, N, K]): x
    [T, K], or [T, k, K] with a row per entry, topk_idx int32 [T, k] -> out
    [T, k, N].  Entries with an id outside [0, E) give zeros."""
    _weights_type((w, "w"))
    by_entry = isinstance(x, torch.Tensor) and x.dim() == 3
    rows = x
    if by_entry:
        if not x.is_contiguous():
            raise ValueError("x must be contiguous")
        rows = x.view(x.shape[0] * x.shape[1], x.shape[2])
    ld = _need_rows(rows, "x")
    T, K = x.shape[0], x.shape[-1]
    dev = x.get_device()
    k = _topk_of(topk_idx, T, dev)
    if by_entry and x.shape[1] != k:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected {(T, k, K)}")
    E, N, _ = _need_weights(w, "w", dev, None, None, K)
    out = _out_rows(out, (T, k, N), out_dtype if out_dtype is not None else x.dtype, x, dev)
    _call(dev, "nvfp4_expert_matvec", x.data_ptr(), _DTYPE_CODE[x.dtype], T, ld, int(by_entry),
          topk_idx.data_ptr(), k, C.byref(w.c_struct()), E, N, K, _DTYPE_CODE[out.dtype],
          out.data_ptr())
    return out


def moe_expert_decode_workspace_size(tokens, hidden, inter, topk) -> int:
    return int(lib().moe_expert_decode_workspace_size(tokens, hidden, inter, topk))


def moe_expert_decode(x, topk_idx, topk_prob, num_experts: int, inter: int, w1: NvFp4Weights,
                      w2: NvFp4Weights, workspace=None, y=None):
    """The expert layer for a few tokens on unquantized activations: FC1,
    weighted SwiGLU, FC2 and the sum over a token's experts with
    moe_expert_forward's weights.  x [T, H] float32, bf16 or fp16, T * k <=
    4096; returns y [T, H] in x's dtype."""
    _weights_type((w1, "w1"), (w2, "w2"))
    ld = _need_rows(x, "x")
    T, H = x.shape
    dev = x.get_device()
    k = _topk_of(topk_idx, T, dev)
    _dense(topk_prob, torch.float32, (T, k), dev, "topk_prob")
    _need_weights(w1, "w1", dev, num_experts, 2 * inter, H)
    _need_weights(w2, "w2", dev, num_experts, H, inter)
    y = _out_rows(y, (T, H), x.dtype, x, dev)
    if workspace is None:
        size = lib().moe_expert_decode_workspace_size(T, H, inter, k)
        workspace = x.new_empty((max(size, 256),), dtype=torch.uint8)
    else:
        _need(workspace, (torch.uint8,), "workspace")
        _same_device(workspace, dev, "workspace")
    _call(dev, "moe_expert_decode", x.data_ptr(), _DTYPE_CODE[x.dtype], T, H, inter, ld,
          topk_idx.data_ptr(), topk_prob.data_ptr(), k, num_experts, C.byref(w1.c_struct()),
          C.byref(w2.c_struct()), y.data_ptr(), workspace.data_ptr(), workspace.numel())
    return y


# ---- low-rank adapters -------------------------------------------------------

def lora_forward_workspace_size(tokens, k, rank) -> int:
    return int(lib().lora_forward_workspace_size(tokens, k, rank))


def lora_backward_workspace_size(dtype, tokens, k, n, adapters, rank) -> int:
    return int(lib().lora_backward_workspace_size(_DTYPE_CODE[dtype], tokens, k, n, adapters, rank))


def nvfp4_lora_matvec_workspace_size(tokens, n, k, rank) -> int:
    return int(lib().nvfp4_lora_matvec_workspace_size(tokens, n, k, rank))


def _need_adapters(a, b, ids, scale, tokens, k, dtype, dev):
    """Adapters a [S, R, K] and b [S, N, R] of this dtype, a token's adapter and
    the scales.  Returns (S, R, N)."""
    for t, name in ((a, "a"), (b, "b")):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            _need(t, (dtype,), name)
            raise ValueError(f"{name}: shape {tuple(t.shape)}, expected three dimensions")
    S, R, _ = a.shape
    N = b.shape[1]
    _dense(a, dtype, (S, R, k), dev, "a")
    _dense(b, dtype, (S, N, R), dev, "b")
    _dense(ids, torch.int32, (tokens,), dev, "ids")
    if scale is not None:
        _dense(scale, torch.float32, (S,), dev, "scale")
    return S, R, N


def _base_rows(base, tokens, width, dtype, dev):
    """The distance of base's rows (its width where there is none)."""
    if base is None:
        return width
    ld = _need_rows(base, "base", width, dtype)
    if base.shape[0] != tokens:
        raise ValueError(f"base: shape {tuple(base.shape)}, expected {(tokens, width)}")
    _same_device(base, dev, "base")
    return ld


def _work_bytes(workspace, size, like, dev):
    if workspace is None:
        return like.new_empty((max(size, 256),), dtype=torch.uint8)
    _need(workspace, (torch.uint8,), "workspace")
    _same_device(workspace, dev, "workspace")
    return workspace


def lora_forward(x, a, b, ids, scale=None, base=None, out_dtype=None, out=None,
                 return_h: bool = False, workspace=None):
    """Low-rank adapters of many requests: y[t] = base[t] + scale[s] b[s] (a[s]
    x[t]) with s = ids[t].  x [T, K], a [S, R, K], b [S, N, R] of one type
    (float32, bf16 or fp16), ids int32 [T] (outside [0, S): no adapter), scale
    float32 [S], base [T, N] in the output's type (the projection's output; `out`
    may be base itself, but overlap nothing else).  Returns y [T, N] in out_dtype (x's by default), with
    return_h also h = a[s] x[t] float32 [T, R], lora_backward's argument."""
    ld = _need_rows(x, "x")
    T, K = x.shape
    dev = x.get_device()
    S, R, N = _need_adapters(a, b, ids, scale, T, K, x.dtype, dev)
    out = _out_rows(out, (T, N), out_dtype if out_dtype is not None else x.dtype, x, dev)
    ld_base = _base_rows(base, T, N, out.dtype, dev)
    h = x.new_empty((T, R), dtype=torch.float32) if return_h else None
    ws = _work_bytes(workspace, lib().lora_forward_workspace_size(T, K, R), x, dev)
    _call(dev, "lora_forward", x.data_ptr(), _DTYPE_CODE[x.dtype], T, K, ld, ids.data_ptr(),
          a.data_ptr(), b.data_ptr(), _addr(scale), S, R, N, _addr(base), ld_base,
          _DTYPE_CODE[out.dtype], out.data_ptr(), _addr(h), ws.data_ptr(), ws.numel())
    return (out, h) if return_h else out


def lora_backward(dy, x, a, b, ids, scale=None, h=None, base=None, out=None, workspace=None):
    """Gradients of lora_forward from dy [T, N] (x's type): dx [T, K] (x's type)
    = base[t] + a[s]^T g[t] with g[t] = scale[s] b[s]^T dy[t] (base: the rest of
    x's gradient; `out` may be base itself, but overlap nothing else), da float32 [S, R, K] and db float32
    [S, N, R].  h: the forward's (None: computed again).  Returns (dx, da, db)."""
    ld_dy = _need_rows(dy, "dy")
    T, N = dy.shape
    dev = dy.get_device()
    ld_x = _need_rows(x, "x", None, dy.dtype)
    K = x.shape[1]
    if x.shape[0] != T:
        raise ValueError(f"x: shape {tuple(x.shape)}, expected {(T, K)}")
    _same_device(x, dev, "x")
    S, R, n = _need_adapters(a, b, ids, scale, T, K, dy.dtype, dev)
    if n != N:
        raise ValueError(f"b: shape {tuple(b.shape)}, expected {(S, N, R)}")
    if h is not None:
        _dense(h, torch.float32, (T, R), dev, "h")
    ld_base = _base_rows(base, T, K, dy.dtype, dev)
    dx = _out_rows(out, (T, K), dy.dtype, dy, dev)
    da = dy.new_empty((S, R, K), dtype=torch.float32)
    db = dy.new_empty((S, N, R), dtype=torch.float32)
    code = _DTYPE_CODE[dy.dtype]
    ws = _work_bytes(workspace, lib().lora_backward_workspace_size(code, T, K, N, S, R), dy, dev)
    _call(dev, "lora_backward", dy.data_ptr(), code, T, N, ld_dy, x.data_ptr(), K, ld_x,
          ids.data_ptr(), a.data_ptr(), b.data_ptr(), _addr(scale), S, R, _addr(h), _addr(base),
          ld_base, dx.data_ptr(), da.data_ptr(), db.data_ptr(), ws.data_ptr(), ws.numel())
    return dx, da, db


def nvfp4_lora_matvec(x, w: NvFp4Weights, a, b, ids, scale=None, out_dtype=None, out=None,
                      workspace=None):
    """nvfp4_matvec with every row's low-rank adapter: x [T, K] times one NVFP4
    matrix (w: [1, N, K], either layout) plus scale[s] b[s] (a[s] x[t]), s =
    ids[t]; a, b, ids and scale as lora_forward's.  Returns [T, N] in out_dtype
    (x's by default), rounded once."""
    _weights_type((w, "w"))
    ld = _need_rows(x, "x")
    T, K = x.shape
    dev = x.get_device()
    S, R, N = _need_adapters(a, b, ids, scale, T, K, x.dtype, dev)
    _need_weights(w, "w", dev, 1, N, K)
    out = _out_rows(out, (T, N), out_dtype if out_dtype is not None else x.dtype, x, dev)
    ws = _work_bytes(workspace, lib().nvfp4_lora_matvec_workspace_size(T, N, K, R), x, dev)
    _call(dev, "nvfp4_lora_matvec", x.data_ptr(), _DTYPE_CODE[x.dtype], T, ld,
          C.byref(w.c_struct()), N, K, ids.data_ptr(), a.data_ptr(), b.data_ptr(), _addr(scale), S,
          R, _DTYPE_CODE[out.dtype], out.data_ptr(), ws.data_ptr(), ws.numel())
    return out


# ---- the orthogonalised update -------------------------------------------------

def newton_schulz_workspace_size(batch, rows, cols, out_dtype) -> int:
    return int(lib().newton_schulz_workspace_size(batch, rows, cols, _DTYPE_CODE[out_dtype]))


def newton_schulz(g, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315), eps: float = 1e-7,
                  scale: float = 1.0, out_dtype=None, out=None, workspace=None):
    """The orthogonalised update of a weight gradient g [rows, cols], or of a
    batch [E, rows, cols] of them (float32, bf16 or fp16; the last dimension
    dense): X = g / (|g|_F + eps), then `steps` times X = a X + (b A + c A A) X
    with A = X X^T (from the other side where rows > cols), times scale.
    Returns g's shape in out_dtype (g's by default; `out` may be g itself if that
    is dense and of the same type, and may not overlap it otherwise).
    bf16 results take faster products in the last steps, as many as stay near bf16's
    own rounding (the usual coefficients: five)."""
    if not isinstance(g, torch.Tensor):
        raise TypeError("g must be a torch.Tensor")
    if not g.is_cuda:
        raise NvFp4Error(f"g must be a device tensor (got {g.device})")
    if g.dtype not in _DTYPE_CODE:
        raise TypeError(f"g: dtype {g.dtype} not in {tuple(_DTYPE_CODE)}")
    if g.dim() not in (2, 3):
        raise ValueError(f"g: shape {tuple(g.shape)}, expected [rows, cols] or [E, rows, cols]")
    rows, cols = g.shape[-2:]
    E = g.shape[0] if g.dim() == 3 else 1
    if rows < 1 or cols < 1:
        raise ValueError(f"g: shape {tuple(g.shape)}, expected elements")
    ld_row = g.stride(-2) if rows > 1 else cols
    ld_batch = g.stride(0) if E > 1 else 0
    if (g.stride(-1) != 1 and cols > 1) or ld_row < cols:
        raise ValueError(f"g: rows must be dense and must not overlap (strides {g.stride()})")
    a, b, c = coefficients
    dev = g.get_device()
    out = _out_rows(out, g.shape, out_dtype if out_dtype is not None else g.dtype, g, dev)
    code = _DTYPE_CODE[out.dtype]
    ws = _work_bytes(workspace, lib().newton_schulz_workspace_size(E, rows, cols, code), g, dev)
    _call(dev, "newton_schulz", g.data_ptr(), _DTYPE_CODE[g.dtype], E, rows, cols, ld_row, ld_batch,
          steps, a, b, c, eps, scale, code, out.data_ptr(), ws.data_ptr(), ws.numel())
    return out
