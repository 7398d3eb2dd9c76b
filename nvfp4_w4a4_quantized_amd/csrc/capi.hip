// capi.hip -- the C ABI declared in include/nvfp4moe.h: host-side argument
// validation (before any HIP call), workspace carving and kernel launches.
#include "nvfp4moe.h"

#include <hip/hip_runtime.h>

#include "launch.h"

using namespace nvfp4;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int hip_status(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_HIP_ERROR; }

size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

bool valid_align(int32_t align) {
  return align >= 1 && align <= 256 && (align & (align - 1)) == 0;
}

constexpr int64_t kMaxK = 16384;
constexpr int32_t kMaxExperts = 1024;

// Sequential carve of 256-byte aligned regions out of one workspace.
struct Carver {
  char* base;
  size_t used = 0;
  explicit Carver(void* b) : base(static_cast<char*>(b)) {}
  template <typename T>
  T* take(size_t count) {
    T* p = base ? reinterpret_cast<T*>(base + used) : nullptr;
    used += round_up(count * sizeof(T), 256);
    return p;
  }
};

struct MoeLayout {
  int32_t* route_ws_i; int32_t* offsets; int32_t* dst_row; int32_t* row_src; float* row_prob;
  uint8_t* tokc; uint8_t* toks; float* tokg;   // token-major quantized activations
  uint8_t* rank;                               // routing entries' ranks inside their chunk
  uint16_t* d; float* amax_d;
  uint8_t* a2c; uint8_t* a2s; float* a2g;
  uint16_t* y_rows;
  int4* tab1; int4* tab2;   // FC1 / FC2 tile tables
  int32_t* bounds;          // per-tensor activation scale: the reduction's row range
  float* tamax;             // per-tensor activation scale: amax of x [0], of D [1]
  size_t bytes;
};

// The FC1 / FC2 launch arguments that fix the grids (sizes only).
GemmArgs moe_gemm_shape(int64_t cap, int64_t H, int64_t I, int32_t E, bool fc1) {
  GemmArgs g{};
  g.num_groups = E; g.rows_cap = cap;
  g.n = fc1 ? 2 * I : H; g.k = fc1 ? H : I; g.inter = fc1 ? I : 0;
  return g;
}

MoeLayout carve_moe(void* ws, int64_t T, int64_t H, int64_t I, int32_t k, int32_t E, int32_t align) {
  const int64_t cap = moe_rows_capacity(T, k, E, align);
  Carver c(ws);
  MoeLayout L;
  L.route_ws_i = c.take<int32_t>(route_workspace_bytes(T, E) / 4);
  L.offsets = c.take<int32_t>(E + 1);
  L.dst_row = c.take<int32_t>((size_t)(T * k));
  L.row_src = c.take<int32_t>((size_t)cap);
  L.row_prob = c.take<float>((size_t)cap);
  L.tokc = c.take<uint8_t>((size_t)((T + 1) * H / 2));   // + the zero row padding rows read
  L.toks = c.take<uint8_t>((size_t)((T + 1) * H / 16));
  L.tokg = c.take<float>((size_t)T);
  L.rank = c.take<uint8_t>((size_t)(T * k));
  L.d = c.take<uint16_t>((size_t)(cap * I));
  L.amax_d = c.take<float>((size_t)cap);
  L.a2c = c.take<uint8_t>((size_t)(cap * I / 2));
  L.a2s = c.take<uint8_t>((size_t)(cap * I / 16));
  L.a2g = c.take<float>((size_t)cap);
  L.y_rows = c.take<uint16_t>((size_t)(cap * H));
  L.tab1 = c.take<int4>((size_t)gemm_grid_blocks(moe_gemm_shape(cap, H, I, E, true), true));
  L.tab2 = c.take<int4>((size_t)gemm_grid_blocks(moe_gemm_shape(cap, H, I, E, false), false));
  L.bounds = c.take<int32_t>(2);
  L.tamax = c.take<float>(2);
  L.bytes = c.used;
  return L;
}

// Workspace of the single-pass layer: routing, token rows, per-row maps and
// scales, the FC2 rows and the fused kernel's tile table.
struct SpLayout {
  int32_t* route_ws_i; int32_t* offsets; int32_t* dst_row; int32_t* row_src; float* row_prob;
  uint8_t* tokc; uint8_t* toks; float* tokg; uint8_t* rank;
  uint16_t* y_rows;
  int4* tab;
  int64_t blocks;
  size_t bytes;
};

SpLayout carve_single_pass(void* ws, int64_t T, int64_t H, int64_t I, int32_t k, int32_t E,
                           int32_t align) {
  const int64_t cap = moe_rows_capacity(T, k, E, align);
  Carver c(ws);
  SpLayout L;
  L.route_ws_i = c.take<int32_t>(route_workspace_bytes(T, E) / 4);
  L.offsets = c.take<int32_t>(E + 1);
  L.dst_row = c.take<int32_t>((size_t)(T * k));
  L.row_src = c.take<int32_t>((size_t)cap);
  L.row_prob = c.take<float>((size_t)cap);
  L.tokc = c.take<uint8_t>((size_t)((T + 1) * H / 2));
  L.toks = c.take<uint8_t>((size_t)((T + 1) * H / 16));
  L.tokg = c.take<float>((size_t)T);
  L.rank = c.take<uint8_t>((size_t)(T * k));
  L.y_rows = c.take<uint16_t>((size_t)(cap * H));
  L.blocks = single_pass_table_spec(cap, E, H, nullptr).blocks;
  L.tab = c.take<int4>((size_t)L.blocks);
  L.bytes = c.used;
  return L;
}

// Workspace of the backward: the two dgrad tile tables, the wgrads' expert
// order, dD, dC, the rows' router-weight gradients and the FC1 dgrad rows.
struct BwdLayout {
  int4* tab2; int4* tab1;   // FC2 / FC1 dgrad tile tables
  int64_t blocks2, blocks1;
  int32_t* order;
  uint16_t* dd; uint16_t* dc; float* dp; uint16_t* dxr;
  size_t bytes;
};

BwdLayout carve_backward(void* ws, int64_t cap, int64_t H, int64_t I, int32_t E) {
  Carver c(ws);
  BwdLayout L;
  L.blocks2 = bwd_dgrad_table_spec(cap, E, H, I, nullptr).blocks;
  L.blocks1 = bwd_dgrad_table_spec(cap, E, 2 * I, H, nullptr).blocks;
  L.tab2 = c.take<int4>((size_t)L.blocks2);
  L.tab1 = c.take<int4>((size_t)L.blocks1);
  L.order = c.take<int32_t>((size_t)E);
  L.dd = c.take<uint16_t>((size_t)(cap * I));
  L.dc = c.take<uint16_t>((size_t)(cap * 2 * I));
  L.dp = c.take<float>((size_t)cap);
  L.dxr = c.take<uint16_t>((size_t)(cap * H));
  L.bytes = c.used;
  return L;
}

bool route_args_ok(int64_t tokens, int32_t topk, int32_t num_experts, int32_t align) {
  if (tokens < 0 || topk < 1 || num_experts < 1 || num_experts > kMaxExperts) return false;
  if (topk > num_experts || !valid_align(align)) return false;
  const int64_t cap = (int64_t)tokens * topk + (int64_t)num_experts * align;
  return cap < 0x7FFFFFFFLL;
}

}  // namespace

extern "C" {

const char* nvfp4_status_string(int status) {
  switch (status) {
    case NVFP4_OK: return "ok";
    case NVFP4_INVALID_ARGUMENT: return "invalid argument";
    case NVFP4_UNSUPPORTED: return "unsupported shape";
    case NVFP4_HIP_ERROR: return "HIP launch/runtime error";
    case NVFP4_WORKSPACE_TOO_SMALL: return "workspace too small";
    case NVFP4_SCRATCH_LIMIT: return "exceeds the static scratch of the no-allocation entry point";
    default: return "unknown status";
  }
}

int nvfp4_debug_checks(void) {
#ifdef NVFP4_DEBUG_CHECKS
  return 1;
#else
  return 0;
#endif
}

int nvfp4_quantize(const uint16_t* x, int64_t rows, int64_t k, int64_t ld_x, int scale_domain,
                   const int32_t* group_offsets, int32_t num_groups, const float* amax_in,
                   int block_rule, uint8_t* codes, uint8_t* block_scales, float* global_scales,
                   void* stream) {
  if (block_rule < 0 || block_rule > 2) return NVFP4_INVALID_ARGUMENT;
  if (rows < 0 || rows >= 0x7FFFFFFFLL || k < 16 || k % 16 != 0 || ld_x < k || ld_x % 8 != 0)
    return NVFP4_INVALID_ARGUMENT;
  if (k > kMaxK) return NVFP4_UNSUPPORTED;
  if (!x || !codes || !block_scales || !global_scales) return NVFP4_INVALID_ARGUMENT;
  if (!aligned(x, 16) || !aligned(codes, 8) || !aligned(global_scales, 4))
    return NVFP4_INVALID_ARGUMENT;
  hipStream_t s = static_cast<hipStream_t>(stream);
  QuantRowsArgs a{x, rows, k, ld_x, 0, amax_in, group_offsets, num_groups,
                  codes, block_scales, global_scales, block_rule};
  if (scale_domain == 0) {
    a.amax_kind = amax_in ? 1 : 0;
    return hip_status(launch_quantize_rows(a, s));
  }
  if (scale_domain != 1 && scale_domain != 2) return NVFP4_INVALID_ARGUMENT;
  if (!group_offsets || num_groups < 1 || num_groups >= 0x7FFFFFFF) return NVFP4_INVALID_ARGUMENT;
  if (scale_domain == 2 && (rows % 16 != 0 || block_rule != 0)) return NVFP4_UNSUPPORTED;
  // group amax: reduce into global_scales (as bits) unless given
  const float* amax_src = amax_in;
  if (!amax_src) {
    hipError_t e = launch_group_amax(x, rows, k, ld_x, group_offsets, num_groups,
                                     reinterpret_cast<uint32_t*>(global_scales), s);
    if (e != hipSuccess) return NVFP4_HIP_ERROR;
    amax_src = global_scales;
  }
  a.amax_kind = 2;
  a.amax_in = amax_src;
  hipError_t e = scale_domain == 2 ? launch_quantize_tiles2d(a, s) : launch_quantize_rows(a, s);
  if (e != hipSuccess) return NVFP4_HIP_ERROR;
  return hip_status(launch_group_finalize(amax_src, global_scales, num_groups, block_rule, s));
}

int64_t moe_rows_capacity(int64_t tokens, int32_t topk, int32_t num_experts, int32_t align) {
  if (tokens < 0 || topk < 1 || num_experts < 1 || align < 1) return 0;
  return tokens * (int64_t)topk + (int64_t)num_experts * (int64_t)(align - 1);
}

size_t moe_permute_workspace_size(int64_t tokens, int32_t topk, int32_t num_experts) {
  (void)topk;
  if (tokens < 0 || num_experts < 1) return 0;
  return route_workspace_bytes(tokens, num_experts);
}

}  // extern "C"

// moe_permute's host-side checks of everything but the workspace.
int nvfp4::permute_args_status(const uint16_t* x, int64_t tokens, int64_t hidden,
                               const int32_t* topk_idx, const float* topk_prob, int32_t topk,
                               int32_t num_experts, int32_t align, int32_t block_rule,
                               const int32_t* expert_offsets, const int32_t* dst_row,
                               const int32_t* row_src, const float* row_prob, const uint8_t* codes,
                               const uint8_t* block_scales, const float* global_scales) {
  if (!route_args_ok(tokens, topk, num_experts, align)) return NVFP4_INVALID_ARGUMENT;
  if (block_rule < 0 || block_rule > 2) return NVFP4_INVALID_ARGUMENT;
  if (!expert_offsets || !row_src || !row_prob) return NVFP4_INVALID_ARGUMENT;
  if (tokens > 0 && (!topk_idx || !topk_prob || !dst_row)) return NVFP4_INVALID_ARGUMENT;
  if (x) {
    if (hidden < 16 || hidden % 16 != 0) return NVFP4_INVALID_ARGUMENT;
    if (hidden > kMaxK) return NVFP4_UNSUPPORTED;
    if (!codes || !block_scales || !global_scales) return NVFP4_INVALID_ARGUMENT;
    if (!aligned(x, 16) || !aligned(codes, 8)) return NVFP4_INVALID_ARGUMENT;
  }
  return NVFP4_OK;
}

extern "C" {

int moe_permute(const uint16_t* x, int64_t tokens, int64_t hidden, const int32_t* topk_idx,
                const float* topk_prob, int32_t topk, int32_t num_experts, int32_t align,
                int32_t block_rule, int32_t* expert_offsets, int32_t* dst_row, int32_t* row_src, float* row_prob,
                uint8_t* codes, uint8_t* block_scales, float* global_scales, void* workspace,
                size_t workspace_bytes, void* stream) {
  const int st = permute_args_status(x, tokens, hidden, topk_idx, topk_prob, topk, num_experts,
                                     align, block_rule, expert_offsets, dst_row, row_src, row_prob,
                                     codes, block_scales, global_scales);
  if (st != NVFP4_OK) return st;
  if (!workspace || !aligned(workspace, 16)) return NVFP4_INVALID_ARGUMENT;
  if (workspace_bytes < route_workspace_bytes(tokens, num_experts)) return NVFP4_WORKSPACE_TOO_SMALL;
  RouteArgs a{};
  a.x = x; a.tokens = tokens; a.hidden = x ? hidden : 0;
  a.topk_idx = topk_idx; a.topk_prob = topk_prob; a.topk = topk;
  a.num_experts = num_experts; a.align = align;
  a.offsets = expert_offsets; a.dst_row = dst_row; a.row_src = row_src; a.row_prob = row_prob;
  a.codes = codes; a.scales = block_scales; a.gscale = global_scales;
  a.workspace = workspace; a.block_rule = block_rule;
  return hip_status(launch_route(a, static_cast<hipStream_t>(stream)));
}

static int gemm_args_ok(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_gscale,
                        int64_t rows_cap, const uint8_t* b_codes, const uint8_t* b_scales,
                        const float* b_gscale, const int32_t* group_offsets, int32_t num_groups,
                        int64_t k) {
  if (!a_codes || !a_scales || !a_gscale || !b_codes || !b_scales || !b_gscale || !group_offsets)
    return NVFP4_INVALID_ARGUMENT;
  if (rows_cap < 0 || rows_cap >= 0x7FFFFFFFLL || num_groups < 1 || num_groups > kMaxExperts)
    return NVFP4_INVALID_ARGUMENT;
  if (k < 16 || k % 16 != 0) return NVFP4_INVALID_ARGUMENT;
  if (k % 128 != 0 || k > kMaxK) return NVFP4_UNSUPPORTED;
  if (!aligned(a_codes, 16) || !aligned(b_codes, 16) || !aligned(a_scales, 4) ||
      !aligned(b_scales, 4))
    return NVFP4_INVALID_ARGUMENT;
  return NVFP4_OK;
}

int w4a4_grouped_gemm(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_gscale,
                      int64_t rows_cap, const uint8_t* b_codes, const uint8_t* b_scales,
                      const float* b_gscale, const int32_t* group_offsets, int32_t num_groups,
                      int64_t n, int64_t k, int b_layout, int out_dtype, void* out,
                      void* stream) {
  int st = gemm_args_ok(a_codes, a_scales, a_gscale, rows_cap, b_codes, b_scales, b_gscale,
                        group_offsets, num_groups, k);
  if (st != NVFP4_OK) return st;
  if (!out || (out_dtype != 0 && out_dtype != 1) || !aligned(out, 16)) return NVFP4_INVALID_ARGUMENT;
  if (b_layout != 0 && b_layout != 1) return NVFP4_INVALID_ARGUMENT;
  if (n < 32 || n % 32 != 0) return NVFP4_UNSUPPORTED;
  if ((int64_t)num_groups * n >= 0x7FFFFFFFLL) return NVFP4_INVALID_ARGUMENT;
  if (n * (k / 2) > 0xFFFFFFFFLL) return NVFP4_UNSUPPORTED;   // 32-bit offsets inside a group
  GemmArgs a{};
  a.a_codes = a_codes; a.a_scales = a_scales; a.a_gscale = a_gscale;
  a.b_codes = b_codes; a.b_scales = b_scales; a.b_gscale = b_gscale;
  a.offsets = group_offsets; a.num_groups = num_groups; a.rows_cap = rows_cap;
  a.n = n; a.k = k; a.b_layout = b_layout; a.out_dtype = out_dtype; a.out = out;
  return hip_status(launch_gemm_plain(a, static_cast<hipStream_t>(stream)));
}

int w4a4_grouped_gemm_swiglu(const uint8_t* a_codes, const uint8_t* a_scales, const float* a_gscale,
                             int64_t rows_cap, const uint8_t* b_codes, const uint8_t* b_scales,
                             const float* b_gscale, const int32_t* group_offsets,
                             int32_t num_groups, int64_t inter, int64_t k, int b_layout,
                             const float* row_prob,
                             uint16_t* d_out, float* amax, float* c_out, void* stream) {
  int st = gemm_args_ok(a_codes, a_scales, a_gscale, rows_cap, b_codes, b_scales, b_gscale,
                        group_offsets, num_groups, k);
  if (st != NVFP4_OK) return st;
  if (!row_prob || !d_out || !amax) return NVFP4_INVALID_ARGUMENT;
  if (b_layout != 0 && b_layout != 1) return NVFP4_INVALID_ARGUMENT;
  if (inter < 64 || inter % 64 != 0) return NVFP4_UNSUPPORTED;
  if ((int64_t)num_groups * 2 * inter >= 0x7FFFFFFFLL) return NVFP4_INVALID_ARGUMENT;
  if (2 * inter * (k / 2) > 0xFFFFFFFFLL) return NVFP4_UNSUPPORTED;   // 32-bit offsets inside a group
  GemmArgs a{};
  a.a_codes = a_codes; a.a_scales = a_scales; a.a_gscale = a_gscale;
  a.b_codes = b_codes; a.b_scales = b_scales; a.b_gscale = b_gscale;
  a.offsets = group_offsets; a.num_groups = num_groups; a.rows_cap = rows_cap;
  a.n = 2 * inter; a.k = k; a.inter = inter; a.b_layout = b_layout;
  a.row_prob = row_prob; a.d_out = d_out; a.amax = amax; a.c_out = c_out;
  return hip_status(launch_gemm_swiglu(a, static_cast<hipStream_t>(stream)));
}

int moe_combine(const void* y_rows, int y_rows_dtype, const int32_t* dst_row, int64_t tokens,
                int32_t topk, int64_t hidden, uint16_t* y, void* stream) {
  if (tokens < 0 || topk < 1 || hidden < 8 || hidden % 8 != 0) return NVFP4_INVALID_ARGUMENT;
  if (y_rows_dtype != 0 && y_rows_dtype != 1) return NVFP4_INVALID_ARGUMENT;
  if (tokens > 0 && (!y_rows || !dst_row || !y)) return NVFP4_INVALID_ARGUMENT;
  if (!aligned(y_rows, 16) || !aligned(y, 16)) return NVFP4_INVALID_ARGUMENT;
  return hip_status(launch_combine(y_rows, y_rows_dtype, dst_row, tokens, topk, hidden, y,
                                   static_cast<hipStream_t>(stream)));
}

size_t moe_expert_forward_workspace_size(int64_t tokens, int64_t hidden, int64_t inter,
                                         int32_t topk, int32_t num_experts, int32_t align) {
  if (!route_args_ok(tokens, topk, num_experts, align) || hidden < 0 || inter < 0) return 0;
  return carve_moe(nullptr, tokens, hidden, inter, topk, num_experts, align).bytes;
}

int moe_expert_forward(const uint16_t* x, int64_t tokens, int64_t hidden, int64_t inter,
                       const int32_t* topk_idx, const float* topk_prob, int32_t topk,
                       int32_t num_experts, int32_t align, int32_t act_block_rule,
                       int32_t act_scale_domain, const nvfp4_weights* w1,
                       const nvfp4_weights* w2, uint16_t* y, void* workspace,
                       size_t workspace_bytes, const nvfp4_moe_intermediates* debug,
                       void* const* stage_events, void* stream) {
  if (!route_args_ok(tokens, topk, num_experts, align)) return NVFP4_INVALID_ARGUMENT;
  if (act_block_rule < 0 || act_block_rule > 2) return NVFP4_INVALID_ARGUMENT;
  if (act_scale_domain != 0 && act_scale_domain != 1) return NVFP4_INVALID_ARGUMENT;
  if (hidden < 128 || hidden % 128 != 0 || inter < 128 || inter % 128 != 0)
    return NVFP4_UNSUPPORTED;
  if (hidden > kMaxK || inter > kMaxK) return NVFP4_UNSUPPORTED;
  if (!w1 || !w2 || !w1->codes || !w1->scales || !w1->gscale || !w2->codes || !w2->scales ||
      !w2->gscale || !workspace)
    return NVFP4_INVALID_ARGUMENT;
  if ((w1->layout != 0 && w1->layout != 1) || (w2->layout != 0 && w2->layout != 1))
    return NVFP4_INVALID_ARGUMENT;
  if (tokens > 0 && (!x || !y || !topk_idx || !topk_prob)) return NVFP4_INVALID_ARGUMENT;
  if (!aligned(workspace, 256) || (x && !aligned(x, 16)) || (y && !aligned(y, 16)) ||
      !aligned(w1->codes, 16) || !aligned(w2->codes, 16) || !aligned(w1->scales, 4) ||
      !aligned(w2->scales, 4))
    return NVFP4_INVALID_ARGUMENT;
  if ((int64_t)num_experts * 2 * inter >= 0x7FFFFFFFLL ||
      (int64_t)num_experts * hidden >= 0x7FFFFFFFLL)
    return NVFP4_INVALID_ARGUMENT;
  if ((tokens + 1) * (hidden / 2) > 0xFFFFFFFFLL) return NVFP4_UNSUPPORTED;   // 32-bit row offsets
  MoeLayout L = carve_moe(workspace, tokens, hidden, inter, topk, num_experts, align);
  if (workspace_bytes < L.bytes) return NVFP4_WORKSPACE_TOO_SMALL;
  float* c_out = nullptr;
  float* y_f32 = nullptr;
  if (debug) {
    if (debug->expert_offsets) L.offsets = debug->expert_offsets;
    if (debug->dst_row) L.dst_row = debug->dst_row;
    if (debug->row_src) L.row_src = debug->row_src;
    if (debug->row_prob) L.row_prob = debug->row_prob;
    if ((debug->a1_codes != nullptr) != (debug->a1_scales != nullptr)) return NVFP4_INVALID_ARGUMENT;
    if (debug->d) L.d = debug->d;
    if (debug->amax_d) L.amax_d = debug->amax_d;
    if (debug->a2_codes) L.a2c = debug->a2_codes;
    if (debug->a2_scales) L.a2s = debug->a2_scales;
    if (debug->a2_gscale) L.a2g = debug->a2_gscale;
    if (debug->y_rows) L.y_rows = debug->y_rows;
    c_out = debug->fc1_out;
    y_f32 = debug->y_rows_f32;
    const void* ptrs16[] = {debug->a1_codes, L.a2c, L.d, L.y_rows, y_f32};
    for (const void* p : ptrs16)
      if (p && !aligned(p, 16)) return NVFP4_INVALID_ARGUMENT;
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t cap = moe_rows_capacity(tokens, topk, num_experts, align);
  auto mark = [&](int i) -> hipError_t {
    if (!stage_events || !stage_events[i]) return hipSuccess;
    return hipEventRecord(static_cast<hipEvent_t>(stage_events[i]), s);
  };
  hipError_t e;
  if ((e = mark(0)) != hipSuccess) return NVFP4_HIP_ERROR;
  GemmArgs g1{};
  g1.a_codes = L.tokc; g1.a_scales = L.toks; g1.a_gscale = L.tokg; g1.a_row_src = L.row_src;
  g1.a_pad_row = tokens;
  g1.b_codes = w1->codes; g1.b_scales = w1->scales; g1.b_gscale = w1->gscale;
  g1.offsets = L.offsets; g1.num_groups = num_experts; g1.rows_cap = cap;
  g1.n = 2 * inter; g1.k = hidden; g1.inter = inter; g1.b_layout = w1->layout;
  g1.row_prob = L.row_prob; g1.d_out = L.d; g1.amax = L.amax_d; g1.c_out = c_out;
  g1.tile_table = L.tab1;
  GemmArgs g2{};
  g2.a_codes = L.a2c; g2.a_scales = L.a2s; g2.a_gscale = L.a2g;
  g2.b_codes = w2->codes; g2.b_scales = w2->scales; g2.b_gscale = w2->gscale;
  g2.offsets = L.offsets; g2.num_groups = num_experts; g2.rows_cap = cap;
  g2.n = hidden; g2.k = inter; g2.b_layout = w2->layout;
  g2.out_dtype = y_f32 ? 0 : 1;
  g2.out = y_f32 ? static_cast<void*>(y_f32) : static_cast<void*>(L.y_rows);
  g2.tile_table = L.tab2;
  // a1 + a2: routing metadata and per-token quantization.  Each token is
  // quantized once into a token-major row; FC1 reads routed row r from token
  // row_src[r] (the permutation is applied by the GEMM's A loads, so no
  // routed copies are written).  The same launches clear amax_d over the
  // whole capacity (FC1 takes atomic maxima into it) and, while they hold
  // the offsets, write both GEMMs' tile tables.
  RouteArgs ra{};
  ra.x = x; ra.tokens = tokens; ra.hidden = hidden;
  ra.topk_idx = topk_idx; ra.topk_prob = topk_prob; ra.topk = topk;
  ra.num_experts = num_experts; ra.align = align;
  ra.offsets = L.offsets; ra.dst_row = L.dst_row;
  ra.row_src = L.row_src;
  ra.row_prob = L.row_prob; ra.gscale = nullptr;   // the GEMMs read tok_gscale through row_src
  ra.tok_codes = L.tokc; ra.tok_scales = L.toks; ra.tok_gscale = L.tokg; ra.entry_rank = L.rank;
  ra.zero_per_row = L.amax_d; ra.zero_rows = cap;
  ra.tables[0] = gemm_tile_table_spec(g1, true, L.tab1);
  ra.tables[1] = gemm_tile_table_spec(g2, false, L.tab2);
  ra.num_tables = 2;
  ra.workspace = L.route_ws_i; ra.block_rule = act_block_rule;
  if (act_scale_domain == 1 && tokens > 0) {
    // one outer scale for the whole x ([miniTE] §2.3 per-tensor scaling)
    if ((e = launch_tensor_amax(x, tokens, hidden, hidden, L.bounds,
                                reinterpret_cast<uint32_t*>(L.tamax), s)) != hipSuccess)
      return NVFP4_HIP_ERROR;
    ra.tok_amax = L.tamax;
  }
  if ((e = launch_route(ra, s)) != hipSuccess) return NVFP4_HIP_ERROR;
  if (debug) {   // the permuted rows and their outer scales, for inspection
    if ((e = launch_gather_rows(L.tokc, L.toks, L.tokg, L.row_src, L.offsets + num_experts, cap,
                                hidden, debug->a1_codes, debug->a1_scales, debug->a1_gscale,
                                s)) != hipSuccess)
      return NVFP4_HIP_ERROR;
  }
  if ((e = mark(1)) != hipSuccess) return NVFP4_HIP_ERROR;
  // a3 + a4: FC1 with the weighted SwiGLU epilogue and D's row amax
  if ((e = launch_gemm_swiglu(g1, s)) != hipSuccess) return NVFP4_HIP_ERROR;
  if ((e = mark(2)) != hipSuccess) return NVFP4_HIP_ERROR;
  // a5: requantize D reusing its amax (rows up to offsets[E] live on device:
  // quantize the whole capacity; rows past the end are ignored downstream)
  QuantRowsArgs q{L.d, cap, inter, inter, 1, L.amax_d, nullptr, 0, L.a2c, L.a2s, L.a2g,
                  act_block_rule};
  if (act_scale_domain == 1) {
    // one outer scale for all routed rows of D: the maximum of their amax
    if ((e = launch_rows_amax(L.amax_d, L.offsets + num_experts, cap, L.tamax + 1, s)) !=
        hipSuccess)
      return NVFP4_HIP_ERROR;
    q.amax_kind = 3;
    q.amax_in = L.tamax + 1;
  }
  if ((e = launch_quantize_rows(q, s)) != hipSuccess) return NVFP4_HIP_ERROR;
  if ((e = mark(3)) != hipSuccess) return NVFP4_HIP_ERROR;
  // a6: FC2
  if ((e = launch_gemm_plain(g2, s)) != hipSuccess) return NVFP4_HIP_ERROR;
  if ((e = mark(4)) != hipSuccess) return NVFP4_HIP_ERROR;
  // a7: combine
  if ((e = launch_combine(y_f32 ? static_cast<const void*>(y_f32) : L.y_rows, y_f32 ? 0 : 1,
                          L.dst_row, tokens, topk, hidden, y, s)) != hipSuccess)
    return NVFP4_HIP_ERROR;
  if ((e = mark(5)) != hipSuccess) return NVFP4_HIP_ERROR;
  return NVFP4_OK;
}

size_t moe_expert_backward_workspace_size(int64_t rows_cap, int64_t hidden, int64_t inter,
                                          int32_t num_experts) {
  if (rows_cap < 0 || rows_cap >= 0x7FFFFFFFLL || hidden < 0 || inter < 0 || num_experts < 1 ||
      num_experts > kMaxExperts)
    return 0;
  return carve_backward(nullptr, rows_cap, hidden, inter, num_experts).bytes;
}

int moe_expert_backward(const uint16_t* dy, const uint16_t* x, int64_t tokens, int64_t hidden,
                        int64_t inter, int32_t topk, int32_t num_experts, int64_t rows_cap,
                        const float* fc1_out, const uint16_t* d, const int32_t* expert_offsets,
                        const int32_t* row_src, const float* row_prob, const int32_t* dst_row,
                        const uint16_t* w1, const uint16_t* w2, uint16_t* dx, float* dw1,
                        float* dw2, float* dprob, void* workspace, size_t workspace_bytes,
                        const nvfp4_moe_backward_intermediates* debug,
                        void* const* stage_events, void* stream) {
  if (tokens < 0 || topk < 1 || num_experts < 1 || num_experts > kMaxExperts || topk > num_experts)
    return NVFP4_INVALID_ARGUMENT;
  if (rows_cap < 0 || rows_cap >= 0x7FFFFFFFLL || tokens * topk >= 0x7FFFFFFFLL)
    return NVFP4_INVALID_ARGUMENT;
  if (hidden < 128 || hidden % 128 != 0 || inter < 128 || inter % 128 != 0)
    return NVFP4_UNSUPPORTED;
  if (hidden > kMaxK || inter > kMaxK) return NVFP4_UNSUPPORTED;
  if (!w1 || !w2 || !dw1 || !dw2 || !expert_offsets || !workspace) return NVFP4_INVALID_ARGUMENT;
  if (rows_cap > 0 && (!fc1_out || !d || !row_src || !row_prob)) return NVFP4_INVALID_ARGUMENT;
  if (tokens > 0 && (!dy || !x || !dx || !dprob || !dst_row)) return NVFP4_INVALID_ARGUMENT;
  const void* a16[] = {dy, x, fc1_out, d, w1, w2, dx, dw1, dw2, workspace};
  for (const void* p : a16)
    if (p && !aligned(p, 16)) return NVFP4_INVALID_ARGUMENT;
  const void* a4[] = {dprob, row_src, row_prob, dst_row, expert_offsets};
  for (const void* p : a4)
    if (p && !aligned(p, 4)) return NVFP4_INVALID_ARGUMENT;
  if (!aligned(workspace, 256)) return NVFP4_INVALID_ARGUMENT;
  // every operand the GEMMs read is addressed with 32-bit byte offsets
  const int64_t tok_bytes = tokens * hidden * 2, c_bytes = rows_cap * 2 * inter * 4;
  const int64_t dc_bytes = rows_cap * 2 * inter * 2, w_bytes = 2 * inter * hidden * 2;
  if (tok_bytes >= 0x80000000LL || c_bytes >= 0x80000000LL || dc_bytes >= 0x80000000LL ||
      w_bytes >= 0x80000000LL)
    return NVFP4_UNSUPPORTED;
  BwdLayout L = carve_backward(workspace, rows_cap, hidden, inter, num_experts);
  if (workspace_bytes < L.bytes) return NVFP4_WORKSPACE_TOO_SMALL;
  float* dxr_f32 = nullptr;
  if (debug) {
    if (debug->dd) L.dd = debug->dd;
    if (debug->dc) L.dc = debug->dc;
    if (debug->dp_rows) L.dp = debug->dp_rows;
    if (debug->dx_rows) L.dxr = debug->dx_rows;
    dxr_f32 = debug->dx_rows_f32;
    const void* p16[] = {L.dd, L.dc, L.dxr};
    for (const void* p : p16)
      if (!aligned(p, 16)) return NVFP4_INVALID_ARGUMENT;
    if (dxr_f32 && !aligned(dxr_f32, 16)) return NVFP4_INVALID_ARGUMENT;
    const void* p4[] = {L.dp};
    for (const void* p : p4)
      if (p && !aligned(p, 4)) return NVFP4_INVALID_ARGUMENT;
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto mark = [&](int i) -> hipError_t {
    if (!stage_events || !stage_events[i]) return hipSuccess;
    return hipEventRecord(static_cast<hipEvent_t>(stage_events[i]), s);
  };
  if (mark(0) != hipSuccess) return NVFP4_HIP_ERROR;
  // the dgrads' tile tables from the device offsets
  const TileTableSpec t2 = bwd_dgrad_table_spec(rows_cap, num_experts, hidden, inter, L.tab2);
  const TileTableSpec t1 = bwd_dgrad_table_spec(rows_cap, num_experts, 2 * inter, hidden, L.tab1);
  if (launch_bwd_tables(expert_offsets, num_experts, t2, t1, L.order, s) != hipSuccess)
    return NVFP4_HIP_ERROR;
  if (mark(1) != hipSuccess) return NVFP4_HIP_ERROR;
  // FC2 dgrad: dD = dYr W2[e] (bf16 rows), then the SwiGLU backward
  BwdGemmArgs f2{};
  f2.a = BwdOperand{dy, hidden, 0, row_src, 1, (uint32_t)tok_bytes};
  f2.b = BwdOperand{w2, inter, hidden * inter, nullptr, 0, (uint32_t)(hidden * inter * 2)};
  f2.offsets = expert_offsets; f2.num_groups = num_experts;
  f2.m = rows_cap; f2.n = inter; f2.k = hidden; f2.tiles = L.tab2;
  f2.out_bf16 = L.dd;
  if (launch_bwd_gemm(BWD_DGRAD_ROWS, f2, L.blocks2, s) != hipSuccess) return NVFP4_HIP_ERROR;
  if (mark(2) != hipSuccess) return NVFP4_HIP_ERROR;
  if (launch_swiglu_bwd(L.dd, fc1_out, row_src, row_prob, expert_offsets + num_experts, rows_cap,
                        inter, L.dc, L.dp, s) != hipSuccess)
    return NVFP4_HIP_ERROR;
  if (mark(3) != hipSuccess) return NVFP4_HIP_ERROR;
  // The dgrads and the reductions first, the wgrads last: the FC1 dgrad and
  // the dx sum then read dC and dXr right after they were written, while
  // they are still in the last-level cache, rather than behind the wgrads'
  // 2.4 GB of weight-gradient stores (the dx sum ran at half speed there).
  // FC1 dgrad: dXr = dC W1[e] (bf16 rows)
  BwdGemmArgs f1{};
  f1.a = BwdOperand{L.dc, 2 * inter, 0, nullptr, 0, (uint32_t)dc_bytes};
  f1.b = BwdOperand{w1, hidden, 2 * inter * hidden, nullptr, 0, (uint32_t)w_bytes};
  f1.offsets = expert_offsets; f1.num_groups = num_experts;
  f1.m = rows_cap; f1.n = hidden; f1.k = 2 * inter; f1.tiles = L.tab1;
  f1.out_bf16 = L.dxr; f1.out_f32 = dxr_f32;
  if (launch_bwd_gemm(BWD_DGRAD_ROWS, f1, L.blocks1, s) != hipSuccess) return NVFP4_HIP_ERROR;
  if (mark(4) != hipSuccess) return NVFP4_HIP_ERROR;
  // dx: the sum of each token's rows; dprob: each entry's row sum
  if (launch_combine(L.dxr, 1, dst_row, tokens, topk, hidden, dx, s) != hipSuccess)
    return NVFP4_HIP_ERROR;
  if (launch_bwd_entry_grad(L.dp, dst_row, tokens * topk, dprob, s) != hipSuccess)
    return NVFP4_HIP_ERROR;
  if (mark(5) != hipSuccess) return NVFP4_HIP_ERROR;
  // FC2 wgrad: dW2[e] = dYr^T D over the expert's rows
  BwdGemmArgs w2g{};
  w2g.a = BwdOperand{dy, hidden, 0, row_src, 1, (uint32_t)tok_bytes};
  w2g.b = BwdOperand{d, inter, 0, nullptr, 0, (uint32_t)(dc_bytes / 2)};
  w2g.offsets = expert_offsets; w2g.num_groups = num_experts; w2g.order = L.order;
  w2g.m = hidden; w2g.n = inter; w2g.out_f32 = dw2;
  if (launch_bwd_gemm(BWD_WGRAD, w2g, bwd_wgrad_blocks(num_experts, hidden, inter), s) !=
      hipSuccess)
    return NVFP4_HIP_ERROR;
  if (mark(6) != hipSuccess) return NVFP4_HIP_ERROR;
  // FC1 wgrad: dW1[e] = dC^T X over the expert's rows
  BwdGemmArgs w1g{};
  w1g.a = BwdOperand{L.dc, 2 * inter, 0, nullptr, 0, (uint32_t)dc_bytes};
  w1g.b = BwdOperand{x, hidden, 0, row_src, 1, (uint32_t)tok_bytes};
  w1g.offsets = expert_offsets; w1g.num_groups = num_experts; w1g.order = L.order;
  w1g.m = 2 * inter; w1g.n = hidden; w1g.out_f32 = dw1;
  if (launch_bwd_gemm(BWD_WGRAD, w1g, bwd_wgrad_blocks(num_experts, 2 * inter, hidden), s) !=
      hipSuccess)
    return NVFP4_HIP_ERROR;
  if (mark(7) != hipSuccess) return NVFP4_HIP_ERROR;
  return NVFP4_OK;
}

int nvfp4_pack_weights(const uint8_t* codes, const uint8_t* scales, int32_t num_groups,
                       int64_t n, int64_t k, uint8_t* packed_codes, uint8_t* packed_scales,
                       void* stream) {
  if (!codes || !scales || !packed_codes || !packed_scales) return NVFP4_INVALID_ARGUMENT;
  if (num_groups < 1 || n < 0 || k < 0) return NVFP4_INVALID_ARGUMENT;
  if (n % 32 != 0 || k % 128 != 0 || k > kMaxK) return NVFP4_UNSUPPORTED;
  if ((int64_t)num_groups * n >= 0x7FFFFFFFLL) return NVFP4_INVALID_ARGUMENT;
  if (!aligned(codes, 16) || !aligned(packed_codes, 16) || !aligned(scales, 4) ||
      !aligned(packed_scales, 4))
    return NVFP4_INVALID_ARGUMENT;
  return hip_status(launch_pack_b(codes, scales, (int64_t)num_groups * n, k, packed_codes,
                                  packed_scales, static_cast<hipStream_t>(stream)));
}

// ---- operators on unquantized tensors ----

static bool valid_dtype(int d) { return d >= 0 && d <= 2; }
static size_t dtype_size(int d) { return d == 0 ? 4 : 2; }

static int router_args_status(const void* logits, int dtype, int64_t tokens, int32_t num_experts,
                              int64_t ld, int32_t topk, int score, int renormalize, float scale) {
  if (!valid_dtype(dtype) || tokens < 0 || num_experts < 1 || num_experts > kMaxExperts ||
      topk < 1 || topk > num_experts || ld < num_experts)
    return NVFP4_INVALID_ARGUMENT;
  if (score != 0 && score != 1) return NVFP4_INVALID_ARGUMENT;
  if (renormalize != 0 && renormalize != 1) return NVFP4_INVALID_ARGUMENT;
  if (!(scale - scale == 0.0f)) return NVFP4_INVALID_ARGUMENT;   // Inf or NaN
  if (tokens > 0x7FFFFFFELL / topk) return NVFP4_INVALID_ARGUMENT;
  if (tokens > 0 && !logits) return NVFP4_INVALID_ARGUMENT;
  if (!aligned(logits, dtype_size(dtype))) return NVFP4_INVALID_ARGUMENT;
  return NVFP4_OK;
}

static int router_call(const void* logits, int dtype, int64_t tokens, int32_t num_experts,
                       int64_t ld_logits, const float* bias, int bias_on_score, int32_t topk,
                       int score, int renormalize, float scale, int32_t* topk_idx,
                       float* topk_prob, void* stream) {
  const int st = router_args_status(logits, dtype, tokens, num_experts, ld_logits, topk, score,
                                    renormalize, scale);
  if (st != NVFP4_OK) return st;
  if (tokens > 0 && (!topk_idx || !topk_prob)) return NVFP4_INVALID_ARGUMENT;
  if (!aligned(bias, 4) || !aligned(topk_idx, 4) || !aligned(topk_prob, 4))
    return NVFP4_INVALID_ARGUMENT;
  RouterArgs a{logits, dtype, tokens, num_experts, ld_logits, bias, bias_on_score,
               topk,   score, renormalize, scale, topk_idx, topk_prob};
  return hip_status(launch_router(a, static_cast<hipStream_t>(stream)));
}

int moe_router(const void* logits, int dtype, int64_t tokens, int32_t num_experts,
               int64_t ld_logits, const float* bias, int32_t topk, int score, int renormalize,
               float scale, int32_t* topk_idx, float* topk_prob, void* stream) {
  return router_call(logits, dtype, tokens, num_experts, ld_logits, bias, 0, topk, score,
                     renormalize, scale, topk_idx, topk_prob, stream);
}

int moe_router_score_bias(const void* logits, int dtype, int64_t tokens, int32_t num_experts,
                          int64_t ld_logits, const float* score_bias, int32_t topk, int score,
                          int renormalize, float scale, int32_t* topk_idx, float* topk_prob,
                          void* stream) {
  if (!score_bias) return NVFP4_INVALID_ARGUMENT;
  return router_call(logits, dtype, tokens, num_experts, ld_logits, score_bias, 1, topk, score,
                     renormalize, scale, topk_idx, topk_prob, stream);
}

int moe_router_backward(const void* logits, int dtype, int64_t tokens, int32_t num_experts,
                        int64_t ld_logits, const int32_t* topk_idx, const float* dprob,
                        int32_t topk, int score, int renormalize, float scale, void* dlogits,
                        void* stream) {
  const int st = router_args_status(logits, dtype, tokens, num_experts, ld_logits, topk, score,
                                    renormalize, scale);
  if (st != NVFP4_OK) return st;
  if (tokens > 0 && (!topk_idx || !dprob || !dlogits)) return NVFP4_INVALID_ARGUMENT;
  if (!aligned(topk_idx, 4) || !aligned(dprob, 4) || !aligned(dlogits, dtype_size(dtype)))
    return NVFP4_INVALID_ARGUMENT;
  RouterBackwardArgs a{logits, dtype, tokens, num_experts, ld_logits, topk_idx, dprob,
                       topk,   score, renormalize, scale, dlogits};
  return hip_status(launch_router_backward(a, static_cast<hipStream_t>(stream)));
}

// Checks shared by the four token movements: `tok` / `rows` are the token
// and row tensors the call reads or writes (with their row distances).
static int token_rows_status(int dtype, int64_t tokens, int64_t hidden, int32_t topk,
                             int64_t rows_cap, const int32_t* dst_row, const float* prob,
                             const float* dprob, const void* tok, int64_t ld_tok,
                             const void* rows, int64_t ld_rows) {
  if (!valid_dtype(dtype) || tokens < 0 || hidden < 1 || topk < 1 || rows_cap < 0 ||
      rows_cap >= 0x7FFFFFFFLL || tokens > 0x7FFFFFFELL / topk)
    return NVFP4_INVALID_ARGUMENT;
  if (hidden > 0x7FFFFFFFLL) return NVFP4_UNSUPPORTED;
  if (ld_tok < hidden || ld_rows < hidden) return NVFP4_INVALID_ARGUMENT;
  if (tokens > 0 && (!tok || !dst_row)) return NVFP4_INVALID_ARGUMENT;
  if (rows_cap > 0 && !rows) return NVFP4_INVALID_ARGUMENT;
  const size_t es = dtype_size(dtype);
  if (!aligned(tok, es) || !aligned(rows, es) || !aligned(dst_row, 4) || !aligned(prob, 4) ||
      !aligned(dprob, 4))
    return NVFP4_INVALID_ARGUMENT;
  return NVFP4_OK;
}

static int spread_status(const int32_t* row_src, const int32_t* expert_offsets,
                         int32_t num_experts, int64_t rows_cap) {
  if (num_experts < 1 || num_experts > kMaxExperts || !expert_offsets ||
      (rows_cap > 0 && !row_src) || !aligned(row_src, 4) || !aligned(expert_offsets, 4))
    return NVFP4_INVALID_ARGUMENT;
  return NVFP4_OK;
}

int moe_sort_tokens(const void* x, int dtype, int64_t tokens, int64_t hidden, int64_t ld_x,
                    const int32_t* dst_row, const float* prob, int32_t topk,
                    const int32_t* row_src, const int32_t* expert_offsets, int32_t num_experts,
                    int64_t rows_cap, void* rows, void* stream) {
  int st = token_rows_status(dtype, tokens, hidden, topk, rows_cap, dst_row, prob, nullptr, x,
                             ld_x, rows, hidden);
  if (st == NVFP4_OK) st = spread_status(row_src, expert_offsets, num_experts, rows_cap);
  if (st != NVFP4_OK) return st;
  TokenRowsArgs a{};
  a.dtype = dtype; a.tokens = tokens; a.hidden = hidden; a.topk = topk; a.rows_cap = rows_cap;
  a.dst_row = dst_row; a.prob = prob; a.tok = x; a.ld_tok = ld_x;
  a.row_src = row_src; a.rows_end = expert_offsets + num_experts; a.rows_out = rows;
  return hip_status(launch_spread(a, static_cast<hipStream_t>(stream)));
}

int moe_sort_tokens_backward(const void* drows, int dtype, int64_t tokens, int64_t hidden,
                             int64_t ld_rows, int64_t rows_cap, const int32_t* dst_row,
                             const float* prob, int32_t topk, const void* x, int64_t ld_x,
                             void* dx, float* dprob, void* stream) {
  const int st = token_rows_status(dtype, tokens, hidden, topk, rows_cap, dst_row, prob, dprob, dx,
                                   hidden, drows, ld_rows);
  if (st != NVFP4_OK) return st;
  if (dprob && tokens > 0 && (!x || ld_x < hidden || !aligned(x, dtype_size(dtype))))
    return NVFP4_INVALID_ARGUMENT;
  TokenRowsArgs a{};
  a.dtype = dtype; a.tokens = tokens; a.hidden = hidden; a.topk = topk; a.rows_cap = rows_cap;
  a.dst_row = dst_row; a.prob = prob; a.dprob = dprob; a.given = x; a.ld_given = ld_x;
  a.rows = drows; a.ld_rows = ld_rows; a.tok_out = dx;
  return hip_status(launch_collect(a, static_cast<hipStream_t>(stream)));
}

int moe_unsort_tokens(const void* rows, int dtype, int64_t tokens, int64_t hidden, int64_t ld_rows,
                      int64_t rows_cap, const int32_t* dst_row, const float* prob, int32_t topk,
                      void* y, void* stream) {
  const int st = token_rows_status(dtype, tokens, hidden, topk, rows_cap, dst_row, prob, nullptr,
                                   y, hidden, rows, ld_rows);
  if (st != NVFP4_OK) return st;
  TokenRowsArgs a{};
  a.dtype = dtype; a.tokens = tokens; a.hidden = hidden; a.topk = topk; a.rows_cap = rows_cap;
  a.dst_row = dst_row; a.prob = prob; a.rows = rows; a.ld_rows = ld_rows; a.tok_out = y;
  return hip_status(launch_collect(a, static_cast<hipStream_t>(stream)));
}

int moe_unsort_tokens_backward(const void* dy, int dtype, int64_t tokens, int64_t hidden,
                               int64_t ld_dy, const int32_t* dst_row, const float* prob,
                               int32_t topk, const int32_t* row_src,
                               const int32_t* expert_offsets, int32_t num_experts,
                               int64_t rows_cap, const void* rows, int64_t ld_rows, void* drows,
                               float* dprob, void* stream) {
  int st = token_rows_status(dtype, tokens, hidden, topk, rows_cap, dst_row, prob, dprob, dy,
                             ld_dy, drows, hidden);
  if (st == NVFP4_OK) st = spread_status(row_src, expert_offsets, num_experts, rows_cap);
  if (st != NVFP4_OK) return st;
  if (dprob && rows_cap > 0 && (!rows || ld_rows < hidden || !aligned(rows, dtype_size(dtype))))
    return NVFP4_INVALID_ARGUMENT;
  TokenRowsArgs a{};
  a.dtype = dtype; a.tokens = tokens; a.hidden = hidden; a.topk = topk; a.rows_cap = rows_cap;
  a.dst_row = dst_row; a.prob = prob; a.dprob = dprob; a.given = rows; a.ld_given = ld_rows;
  a.tok = dy; a.ld_tok = ld_dy;
  a.row_src = row_src; a.rows_end = expert_offsets + num_experts; a.rows_out = drows;
  return hip_status(launch_spread(a, static_cast<hipStream_t>(stream)));
}

// Most entries (tokens * topk) of an expert call: their list lies in LDS.
constexpr int64_t kMaxEntries = 4096;

static int matvec_weights_status(const nvfp4_weights* w, int64_t n, int64_t k) {
  if (!w || !w->codes || !w->scales || !w->gscale || (w->layout != 0 && w->layout != 1) ||
      !aligned(w->gscale, 4))
    return NVFP4_INVALID_ARGUMENT;
  if (n < 1 || k < 16 || k % 16 != 0) return NVFP4_INVALID_ARGUMENT;
  if (k > kMaxK || n > 0x7FFFFFFFLL / (k / 2)) return NVFP4_UNSUPPORTED;
  if (w->layout == 1) {
    if (n % 32 != 0 || k % 128 != 0) return NVFP4_UNSUPPORTED;
    if (!aligned(w->codes, 16) || !aligned(w->scales, 4)) return NVFP4_INVALID_ARGUMENT;
  }
  return NVFP4_OK;
}

static MatvecArgs matvec_args(const void* x, int x_dtype, int64_t ld_x, int64_t tokens,
                              const nvfp4_weights* w, int32_t groups, int64_t n, int64_t k) {
  MatvecArgs a{};
  a.x = x; a.x_dtype = x_dtype; a.ld_x = ld_x; a.tokens = tokens;
  a.codes = w->codes; a.scales = w->scales; a.gscale = w->gscale; a.layout = w->layout;
  a.num_groups = groups; a.n = n; a.k = k; a.topk = 1;
  return a;
}

int nvfp4_matvec(const void* x, int x_dtype, int64_t tokens, int64_t ld_x, const nvfp4_weights* w,
                 int64_t n, int64_t k, int out_dtype, void* out, void* stream) {
  const int st = matvec_weights_status(w, n, k);
  if (st != NVFP4_OK) return st;
  if (!valid_dtype(x_dtype) || !valid_dtype(out_dtype) || tokens < 0 || ld_x < k)
    return NVFP4_INVALID_ARGUMENT;
  if (tokens > 65536) return NVFP4_UNSUPPORTED;
  if (tokens > 0 && (!x || !out)) return NVFP4_INVALID_ARGUMENT;
  if (!aligned(x, dtype_size(x_dtype)) || !aligned(out, dtype_size(out_dtype)))
    return NVFP4_INVALID_ARGUMENT;
  MatvecArgs a = matvec_args(x, x_dtype, ld_x, tokens, w, 1, n, k);
  a.out = out; a.out_dtype = out_dtype;
  return hip_status(launch_matvec(a, static_cast<hipStream_t>(stream)));
}

int nvfp4_expert_matvec(const void* x, int x_dtype, int64_t tokens, int64_t ld_x, int x_by_entry,
                        const int32_t* topk_idx, int32_t topk, const nvfp4_weights* w,
                        int32_t num_experts, int64_t n, int64_t k, int out_dtype, void* out,
                        void* stream) {
  const int st = matvec_weights_status(w, n, k);
  if (st != NVFP4_OK) return st;
  if (!valid_dtype(x_dtype) || !valid_dtype(out_dtype) || tokens < 0 || ld_x < k || topk < 1 ||
      num_experts < 1 || num_experts > kMaxExperts || (x_by_entry != 0 && x_by_entry != 1))
    return NVFP4_INVALID_ARGUMENT;
  if (tokens > kMaxEntries / topk) return NVFP4_UNSUPPORTED;
  if (tokens > 0 && (!x || !out || !topk_idx)) return NVFP4_INVALID_ARGUMENT;
  if (!aligned(x, dtype_size(x_dtype)) || !aligned(out, dtype_size(out_dtype)) ||
      !aligned(topk_idx, 4))
    return NVFP4_INVALID_ARGUMENT;
  MatvecArgs a = matvec_args(x, x_dtype, ld_x, tokens, w, num_experts, n, k);
  a.x_by_entry = x_by_entry; a.topk_idx = topk_idx; a.topk = topk;
  a.out = out; a.out_dtype = out_dtype;
  return hip_status(launch_matvec(a, static_cast<hipStream_t>(stream)));
}

struct DecodeLayout {
  uint16_t* d;      // FC2's input, binary32 as three bf16 parts: [3, entries, inter]
  float* y_rows;    // FC2's output [entries, hidden]
  size_t bytes;
};

static DecodeLayout carve_decode(void* ws, int64_t entries, int64_t hidden, int64_t inter) {
  Carver c(ws);
  DecodeLayout L;
  L.d = c.take<uint16_t>((size_t)(3 * entries * inter));
  L.y_rows = c.take<float>((size_t)(entries * hidden));
  L.bytes = c.used;
  return L;
}

size_t moe_expert_decode_workspace_size(int64_t tokens, int64_t hidden, int64_t inter,
                                        int32_t topk) {
  if (tokens < 0 || topk < 1 || tokens > kMaxEntries / topk || hidden < 0 || inter < 0 ||
      hidden > kMaxK || inter > kMaxK)
    return 0;
  return carve_decode(nullptr, tokens * topk, hidden, inter).bytes;
}

int moe_expert_decode(const void* x, int x_dtype, int64_t tokens, int64_t hidden, int64_t inter,
                      int64_t ld_x, const int32_t* topk_idx, const float* topk_prob, int32_t topk,
                      int32_t num_experts, const nvfp4_weights* w1, const nvfp4_weights* w2,
                      void* y, void* workspace, size_t workspace_bytes, void* stream) {
  if (!valid_dtype(x_dtype) || tokens < 0 || ld_x < hidden || topk < 1 || num_experts < 1 ||
      num_experts > kMaxExperts || topk > num_experts)
    return NVFP4_INVALID_ARGUMENT;
  if (hidden < 16 || hidden % 16 != 0 || inter < 16 || inter % 16 != 0 || hidden > kMaxK ||
      inter > kMaxK)
    return NVFP4_UNSUPPORTED;
  int st = matvec_weights_status(w1, 2 * inter, hidden);
  if (st == NVFP4_OK) st = matvec_weights_status(w2, hidden, inter);
  if (st != NVFP4_OK) return st;
  if (w1->layout == 1 && inter % 32 != 0) return NVFP4_UNSUPPORTED;
  if (tokens > kMaxEntries / topk) return NVFP4_UNSUPPORTED;
  if (tokens == 0) return NVFP4_OK;
  if (!x || !y || !topk_idx || !topk_prob || !workspace) return NVFP4_INVALID_ARGUMENT;
  if (!aligned(x, dtype_size(x_dtype)) || !aligned(y, dtype_size(x_dtype)) ||
      !aligned(topk_idx, 4) || !aligned(topk_prob, 4) || !aligned(workspace, 16))
    return NVFP4_INVALID_ARGUMENT;
  const DecodeLayout L = carve_decode(workspace, tokens * topk, hidden, inter);
  if (workspace_bytes < L.bytes) return NVFP4_WORKSPACE_TOO_SMALL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  MatvecArgs f1 = matvec_args(x, x_dtype, ld_x, tokens, w1, num_experts, 2 * inter, hidden);
  f1.topk_idx = topk_idx; f1.topk = topk; f1.prob = topk_prob;
  f1.d = L.d; f1.d_plane = tokens * topk * inter; f1.inter = inter;
  if (launch_matvec(f1, s) != hipSuccess) return NVFP4_HIP_ERROR;
  MatvecArgs f2 = matvec_args(L.d, 1, inter, tokens, w2, num_experts, hidden, inter);
  f2.x_plane = f1.d_plane; f2.x_by_entry = 1; f2.topk_idx = topk_idx; f2.topk = topk;
  if (decode_down_fits(tokens, topk, num_experts)) {
    f2.out = y; f2.out_dtype = x_dtype;
    return hip_status(launch_decode_down(f2, s));
  }
  f2.out = L.y_rows; f2.out_dtype = 0; f2.skip_unrouted = 1;
  if (launch_matvec(f2, s) != hipSuccess) return NVFP4_HIP_ERROR;
  return hip_status(launch_decode_combine(L.y_rows, topk_idx, tokens, topk, num_experts, hidden,
                                          x_dtype, y, s));
}

// ---- low-rank adapters ----

constexpr int64_t kMaxLoraTokens = 1 << 24, kMaxLoraWidth = 1 << 18;
constexpr int32_t kMaxRank = 256;

// What every adapter call asks of its sizes and adapters.
static int lora_status(int dtype, int64_t tokens, int64_t k, int64_t n, const int32_t* ids,
                       const void* a, const void* b, const float* scale, int32_t adapters,
                       int32_t rank) {
  if (!valid_dtype(dtype) || tokens < 0 || k < 1 || n < 1 || adapters < 1 || rank < 1)
    return NVFP4_INVALID_ARGUMENT;
  if (tokens > kMaxLoraTokens || k > kMaxLoraWidth || n > kMaxLoraWidth ||
      adapters > kMaxAdapters || rank > kMaxRank)
    return NVFP4_UNSUPPORTED;
  const size_t e = dtype_size(dtype);
  if (!a || !b || !aligned(a, e) || !aligned(b, e) || !aligned(scale, 4) || !aligned(ids, 4) ||
      (tokens > 0 && !ids))
    return NVFP4_INVALID_ARGUMENT;
  return NVFP4_OK;
}

static bool rows_ok(const void* p, int64_t tokens, int64_t width, int64_t ld, int dtype) {
  return ld >= width && (p || tokens == 0) && aligned(p, dtype_size(dtype));
}

static LoraDownArgs lora_down(const void* x, int dtype, int64_t tokens, int64_t k, int64_t ld_x,
                              const int32_t* ids, const void* a, int32_t adapters, int32_t rank,
                              float* h) {
  LoraDownArgs d{};
  d.x = x; d.dtype = dtype; d.tokens = tokens; d.k = k; d.ld_x = ld_x;
  d.ids = ids; d.adapters = adapters; d.rank = rank; d.a = a; d.h = h;
  return d;
}

static LoraUpArgs lora_up(const float* h, int shares, int64_t tokens, int64_t n, const int32_t* ids,
                          const void* b, int dtype, const float* scale, int32_t adapters,
                          int32_t rank, const void* base, int base_dtype, int64_t ld_base, void* out,
                          int out_dtype) {
  LoraUpArgs u{};
  u.h = h; u.shares = shares; u.tokens = tokens; u.n = n;
  u.ids = ids; u.adapters = adapters; u.rank = rank; u.b = b; u.dtype = dtype; u.scale = scale;
  u.base = base; u.base_dtype = base_dtype; u.ld_base = ld_base; u.out = out; u.out_dtype = out_dtype;
  return u;
}

size_t lora_forward_workspace_size(int64_t tokens, int64_t k, int32_t rank) {
  if (tokens < 0 || tokens > kMaxLoraTokens || k < 1 || k > kMaxLoraWidth || rank < 1 ||
      rank > kMaxRank)
    return 0;
  Carver c(nullptr);
  c.take<float>((size_t)(lora_shares(tokens, k) * tokens * rank));
  return c.used;
}

int lora_forward(const void* x, int dtype, int64_t tokens, int64_t k, int64_t ld_x,
                 const int32_t* ids, const void* a, const void* b, const float* scale,
                 int32_t adapters, int32_t rank, int64_t n, const void* base, int64_t ld_base,
                 int out_dtype, void* out, float* h, void* workspace, size_t workspace_bytes,
                 void* stream) {
  const int st = lora_status(dtype, tokens, k, n, ids, a, b, scale, adapters, rank);
  if (st != NVFP4_OK) return st;
  if (!valid_dtype(out_dtype) || !rows_ok(x, tokens, k, ld_x, dtype) ||
      !rows_ok(out, tokens, n, n, out_dtype) || !aligned(h, 4) ||
      (base && !rows_ok(base, tokens, n, ld_base, out_dtype)))
    return NVFP4_INVALID_ARGUMENT;
  if (tokens == 0) return NVFP4_OK;
  if (!workspace || !aligned(workspace, 16)) return NVFP4_INVALID_ARGUMENT;
  if (workspace_bytes < lora_forward_workspace_size(tokens, k, rank)) return NVFP4_WORKSPACE_TOO_SMALL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  float* shares = static_cast<float*>(workspace);
  const bool direct = lora_direct(dtype, tokens, k, n, rank);
  if (!direct &&
      launch_lora_down(lora_down(x, dtype, tokens, k, ld_x, ids, a, adapters, rank, shares), s) !=
          hipSuccess)
    return NVFP4_HIP_ERROR;
  LoraUpArgs u = lora_up(shares, lora_shares(tokens, k), tokens, n, ids, b, dtype, scale, adapters,
                         rank, base, out_dtype, ld_base, out, out_dtype);
  u.h_out = h;
  if (direct) { u.x = x; u.a = a; u.k = k; u.ld_x = ld_x; }
  return hip_status(launch_lora_up(u, s));
}

struct LoraMatvecLayout {
  float* shares;    // [shares, tokens, rank]
  float* y;         // [tokens, n]: the projection's sums before the adapters'
  size_t bytes;
};

static LoraMatvecLayout carve_lora_matvec(void* ws, int64_t tokens, int64_t n, int64_t k, int32_t rank) {
  Carver c(ws);
  LoraMatvecLayout L;
  L.shares = c.take<float>((size_t)(lora_shares(tokens, k) * tokens * rank));
  L.y = c.take<float>((size_t)(tokens * n));
  L.bytes = c.used;
  return L;
}

size_t nvfp4_lora_matvec_workspace_size(int64_t tokens, int64_t n, int64_t k, int32_t rank) {
  if (tokens < 0 || tokens > 65536 || n < 1 || n > kMaxLoraWidth || k < 1 || k > kMaxK || rank < 1 ||
      rank > kMaxRank)
    return 0;
  return carve_lora_matvec(nullptr, tokens, n, k, rank).bytes;
}

int nvfp4_lora_matvec(const void* x, int x_dtype, int64_t tokens, int64_t ld_x,
                      const nvfp4_weights* w, int64_t n, int64_t k, const int32_t* ids,
                      const void* a, const void* b, const float* scale, int32_t adapters,
                      int32_t rank, int out_dtype, void* out, void* workspace,
                      size_t workspace_bytes, void* stream) {
  int st = matvec_weights_status(w, n, k);
  if (st == NVFP4_OK) st = lora_status(x_dtype, tokens, k, n, ids, a, b, scale, adapters, rank);
  if (st != NVFP4_OK) return st;
  if (tokens > 65536) return NVFP4_UNSUPPORTED;
  if (!valid_dtype(out_dtype) || !rows_ok(x, tokens, k, ld_x, x_dtype) ||
      !rows_ok(out, tokens, n, n, out_dtype))
    return NVFP4_INVALID_ARGUMENT;
  if (tokens == 0) return NVFP4_OK;
  if (!workspace || !aligned(workspace, 16)) return NVFP4_INVALID_ARGUMENT;
  const LoraMatvecLayout L = carve_lora_matvec(workspace, tokens, n, k, rank);
  if (workspace_bytes < L.bytes) return NVFP4_WORKSPACE_TOO_SMALL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool direct = lora_direct(x_dtype, tokens, k, n, rank);
  if (!direct &&
      launch_lora_down(lora_down(x, x_dtype, tokens, k, ld_x, ids, a, adapters, rank, L.shares), s) !=
          hipSuccess)
    return NVFP4_HIP_ERROR;
  MatvecArgs m = matvec_args(x, x_dtype, ld_x, tokens, w, 1, n, k);
  m.out = L.y; m.out_dtype = 0;
  if (launch_matvec(m, s) != hipSuccess) return NVFP4_HIP_ERROR;
  LoraUpArgs u = lora_up(L.shares, lora_shares(tokens, k), tokens, n, ids, b, x_dtype, scale,
                         adapters, rank, L.y, 0, n, out, out_dtype);
  if (direct) { u.x = x; u.a = a; u.k = k; u.ld_x = ld_x; }
  return hip_status(launch_lora_up(u, s));
}

struct LoraBackwardLayout {
  void* at; void* bt;         // A and B transposed: [S, K, R], [S, R, N]
  float* shares;              // of g, then (without the forward's h) of h
  float* g; float* h;         // [tokens, rank]
  int32_t* rows; int4* entries; int32_t* part0;
  float* parts;
  int32_t chunk, max_entries;
  size_t bytes;
};

static LoraBackwardLayout carve_lora_backward(void* ws, int dtype, int64_t T, int64_t k, int64_t n,
                                              int32_t S, int32_t rank) {
  Carver c(ws);
  LoraBackwardLayout L;
  const size_t e = dtype_size(dtype), wide = (size_t)rank * (size_t)(k + n);
  L.at = c.take<char>(e * S * rank * k);
  L.bt = c.take<char>(e * S * rank * n);
  const int sk = lora_shares(T, k), sn = lora_shares(T, n);
  L.shares = c.take<float>((size_t)((sk > sn ? sk : sn) * T * rank));
  L.g = c.take<float>((size_t)(T * rank));
  L.h = c.take<float>((size_t)(T * rank));
  L.rows = c.take<int32_t>((size_t)T + kRowsBehind);
  L.chunk = lora_chunk(dtype, T, k, n, rank);
  L.max_entries = (int32_t)(T / L.chunk) + S;
  L.entries = c.take<int4>((size_t)L.max_entries);
  L.part0 = c.take<int32_t>((size_t)S + 1);
  // an adapter of more than a chunk's tokens has at most twice their quotient of chunks
  L.parts = c.take<float>((size_t)(2 * T / L.chunk) * wide);
  L.bytes = c.used;
  return L;
}

// A launch takes fewer than 2^32 threads: one per value of h where it is computed
// again, and 1024 per 64 x 64 tile of A and B, which the transposes take, and the sort.
static bool lora_backward_fits(int64_t tokens, int64_t k, int64_t n, int32_t adapters, int32_t rank) {
  const int64_t tiles = (int64_t)adapters * ((rank + 63) / 64) * ((k + 63) / 64 + (n + 63) / 64);
  return tokens * rank < (1LL << 32) && tiles < (1 << 22) - 1;
}

size_t lora_backward_workspace_size(int dtype, int64_t tokens, int64_t k, int64_t n,
                                    int32_t adapters, int32_t rank) {
  if (!valid_dtype(dtype) || tokens < 0 || tokens > kMaxLoraTokens || k < 1 || n < 1 ||
      k > kMaxLoraWidth || n > kMaxLoraWidth || adapters < 1 || adapters > kMaxAdapters || rank < 1 ||
      rank > kMaxRank || !lora_backward_fits(tokens, k, n, adapters, rank))
    return 0;
  return carve_lora_backward(nullptr, dtype, tokens, k, n, adapters, rank).bytes;
}

int lora_backward(const void* dy, int dtype, int64_t tokens, int64_t n, int64_t ld_dy,
                  const void* x, int64_t k, int64_t ld_x, const int32_t* ids, const void* a,
                  const void* b, const float* scale, int32_t adapters, int32_t rank, const float* h,
                  const void* base, int64_t ld_base, void* dx, float* da, float* db,
                  void* workspace, size_t workspace_bytes, void* stream) {
  const int st = lora_status(dtype, tokens, k, n, ids, a, b, scale, adapters, rank);
  if (st != NVFP4_OK) return st;
  if (!lora_backward_fits(tokens, k, n, adapters, rank)) return NVFP4_UNSUPPORTED;
  if (!rows_ok(dy, tokens, n, ld_dy, dtype) || !rows_ok(x, tokens, k, ld_x, dtype) ||
      (base && !rows_ok(base, tokens, k, ld_base, dtype)) || !rows_ok(dx, tokens, k, k, dtype) ||
      !da || !db || !aligned(da, 4) || !aligned(db, 4) || !aligned(h, 4) || !workspace ||
      !aligned(workspace, 16))
    return NVFP4_INVALID_ARGUMENT;
  const LoraBackwardLayout L = carve_lora_backward(workspace, dtype, tokens, k, n, adapters, rank);
  if (workspace_bytes < L.bytes) return NVFP4_WORKSPACE_TOO_SMALL;
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = hipSuccess;
  if (!h) {
    e = launch_lora_down(lora_down(x, dtype, tokens, k, ld_x, ids, a, adapters, rank, L.shares), s);
    if (e == hipSuccess)
      e = launch_lora_join_shares(L.shares, lora_shares(tokens, k), tokens * rank, L.h, s);
  }
  LoraPrepareArgs pr{};
  pr.sort.ids = ids; pr.sort.tokens = tokens; pr.sort.adapters = adapters; pr.sort.chunk = L.chunk;
  pr.sort.max_entries = L.max_entries; pr.sort.rows = L.rows; pr.sort.entries = L.entries;
  pr.sort.part0 = L.part0;
  pr.a = a; pr.b = b; pr.dtype = dtype; pr.k = k; pr.n = n; pr.rank = rank; pr.at = L.at; pr.bt = L.bt;
  if (e == hipSuccess) e = launch_lora_prepare(pr, s);
  if (e == hipSuccess)
    e = launch_lora_down(lora_down(dy, dtype, tokens, n, ld_dy, ids, L.bt, adapters, rank, L.shares), s);
  if (e == hipSuccess) {
    LoraUpArgs u = lora_up(L.shares, lora_shares(tokens, n), tokens, k, ids, L.at, dtype, scale,
                           adapters, rank, base, dtype, ld_base, dx, dtype);
    u.h_out = L.g; u.h_scaled = 1;
    e = launch_lora_up(u, s);
  }
  LoraGradArgs gr{};
  gr.x = x; gr.dy = dy; gr.dtype = dtype; gr.k = k; gr.n = n; gr.ld_x = ld_x; gr.ld_dy = ld_dy;
  gr.g = L.g; gr.h = h ? h : L.h; gr.scale = scale; gr.adapters = adapters; gr.rank = rank;
  gr.rows = L.rows; gr.entries = L.entries; gr.da = da; gr.db = db; gr.parts = L.parts;
  if (e == hipSuccess) e = launch_lora_grad(gr, L.max_entries, L.part0, s);
  return hip_status(e);
}

// ---- the orthogonalised update ----

constexpr int64_t kMaxSide = 16384, kMaxMatrices = 1 << 20;

struct NsLayout {
  double* norms; int32_t* k0;
  _Float16* x[4]; _Float16* sq[4];
  double* parts; double* q;   // of a short side alone
  size_t bytes;
};

static NsLayout carve_ns(void* ws, int64_t batch, int64_t rows, int64_t cols) {
  Carver c(ws);
  NsLayout L{};
  const int64_t m = ns_batch(batch, rows, cols), n = rows < cols ? rows : cols;
  const size_t xs = (size_t)(m * rows) * round_up((size_t)cols, 64);
  const size_t ns = (size_t)(m * n) * round_up((size_t)n, 64);
  L.norms = c.take<double>((size_t)(m * ns_norm_parts(m, rows)));
  L.k0 = c.take<int32_t>((size_t)m);
  for (int i = 0; i < 4; ++i) L.x[i] = c.take<_Float16>(xs);
  for (int i = 0; i < 4; ++i) L.sq[i] = c.take<_Float16>(ns);
  L.bytes = c.used;
  if (n <= 64) {              // (whichever of the two the coefficients choose)
    Carver d(ws);
    const int64_t most = ns_small_batch(batch), side = ns_small_side(n), tiles = side / 16 * (side / 16 + 1) / 2;
    L.parts = d.take<double>((size_t)(most * ns_small_shares(most, rows < cols ? cols : rows) * tiles * 256));
    L.q = d.take<double>((size_t)(most * side * side));
    if (d.used > L.bytes) L.bytes = d.used;
  }
  return L;
}

static int ns_status(int64_t batch, int64_t rows, int64_t cols, int out_dtype) {
  if (batch < 0 || rows < 1 || cols < 1 || !valid_dtype(out_dtype)) return NVFP4_INVALID_ARGUMENT;
  if (rows > kMaxSide || cols > kMaxSide || batch > kMaxMatrices) return NVFP4_UNSUPPORTED;
  return NVFP4_OK;
}

size_t newton_schulz_workspace_size(int64_t batch, int64_t rows, int64_t cols, int out_dtype) {
  if (ns_status(batch, rows, cols, out_dtype) != NVFP4_OK || batch == 0) return 0;
  return carve_ns(nullptr, batch, rows, cols).bytes;
}

int newton_schulz(const void* g, int dtype, int64_t batch, int64_t rows, int64_t cols,
                  int64_t ld_row, int64_t ld_batch, int steps, float a, float b, float c, float eps,
                  float scale, int out_dtype, void* out, void* workspace, size_t workspace_bytes,
                  void* stream) {
  const int st = ns_status(batch, rows, cols, out_dtype);
  if (st != NVFP4_OK) return st;
  const float big = 3.4e38f;
  if (!valid_dtype(dtype) || ld_row < cols || ld_batch < 0 || steps < 1 || !(eps >= 0.0f) ||
      !(eps <= big) || !(scale >= -big && scale <= big) || !(a >= -big && a <= big) ||
      !(b >= -big && b <= big) || !(c >= -big && c <= big))
    return NVFP4_INVALID_ARGUMENT;
  if (batch > 0 && (!g || !out || !workspace)) return NVFP4_INVALID_ARGUMENT;
  if (!aligned(g, dtype_size(dtype)) || !aligned(out, dtype_size(out_dtype)) || !aligned(workspace, 16))
    return NVFP4_INVALID_ARGUMENT;
  NsArgs n{};
  if (steps > kMaxNsSteps || !ns_bounds(steps, a, b, c, &n.scales)) return NVFP4_UNSUPPORTED;
  const bool small = ns_is_small(rows, cols, steps, a, b, c);
  if (!small && !ns_keeps_small(steps, a)) return NVFP4_UNSUPPORTED;
  if (batch == 0) return NVFP4_OK;
  const NsLayout L = carve_ns(workspace, batch, rows, cols);
  if (workspace_bytes < L.bytes) return NVFP4_WORKSPACE_TOO_SMALL;
  n.src.g = g; n.src.dtype = dtype; n.src.rows = rows; n.src.cols = cols;
  n.src.ld_row = ld_row; n.src.ld_batch = ld_batch; n.batch = batch;
  n.steps = steps; n.a = a; n.b = b; n.c = c; n.eps = eps; n.out_scale = scale;
  n.exact = out_dtype != 1 ? steps : steps - n.scales.fast;
  n.out = out; n.out_dtype = out_dtype; n.norms = L.norms; n.k0 = L.k0;
  for (int i = 0; i < 4; ++i) {
    n.x[i] = L.x[i];
    n.sq[i] = L.sq[i];
  }
  n.small_parts = L.parts; n.small_q = L.q;
  if (small)
    return hip_status(launch_newton_schulz_small(n, static_cast<hipStream_t>(stream)));
  return hip_status(launch_newton_schulz(n, static_cast<hipStream_t>(stream)));
}

int nvfp4_event_create(void** event) {
  if (!event) return NVFP4_INVALID_ARGUMENT;
  hipEvent_t ev;
  if (hipEventCreate(&ev) != hipSuccess) return NVFP4_HIP_ERROR;
  *event = ev;
  return NVFP4_OK;
}

int nvfp4_event_record(void* event, void* stream) {
  if (!event) return NVFP4_INVALID_ARGUMENT;
  return hip_status(hipEventRecord(static_cast<hipEvent_t>(event), static_cast<hipStream_t>(stream)));
}

int nvfp4_event_elapsed_ms(void* start, void* stop, float* ms) {
  if (!start || !stop || !ms) return NVFP4_INVALID_ARGUMENT;
  return hip_status(hipEventElapsedTime(ms, static_cast<hipEvent_t>(start), static_cast<hipEvent_t>(stop)));
}

int nvfp4_event_destroy(void* event) {
  if (!event) return NVFP4_INVALID_ARGUMENT;
  return hip_status(hipEventDestroy(static_cast<hipEvent_t>(event)));
}

size_t moe_expert_forward_single_pass_workspace_size(int64_t tokens, int64_t hidden,
                                                     int64_t inter, int32_t topk,
                                                     int32_t num_experts, int32_t align) {
  if (!route_args_ok(tokens, topk, num_experts, align) || hidden < 0 || inter < 0) return 0;
  return carve_single_pass(nullptr, tokens, hidden, inter, topk, num_experts, align).bytes;
}

int moe_expert_forward_single_pass(const uint16_t* x, int64_t tokens, int64_t hidden,
                                   int64_t inter, const int32_t* topk_idx,
                                   const float* topk_prob, int32_t topk, int32_t num_experts,
                                   int32_t align, const nvfp4_weights* w1,
                                   const nvfp4_weights* w2, uint16_t* y, void* workspace,
                                   size_t workspace_bytes,
                                   const nvfp4_single_pass_intermediates* debug,
                                   void* const* stage_events, void* stream) {
  if (!route_args_ok(tokens, topk, num_experts, align)) return NVFP4_INVALID_ARGUMENT;
  if (hidden < 128 || hidden % 128 != 0 || inter < 128 || inter % 128 != 0)
    return NVFP4_UNSUPPORTED;
  if (hidden > kMaxK || inter > 1152) return NVFP4_UNSUPPORTED;   // on-chip FC2 input (LDS)
  if (!w1 || !w2 || !w1->codes || !w1->scales || !w1->gscale || !w2->codes || !w2->scales ||
      !w2->gscale || !workspace)
    return NVFP4_INVALID_ARGUMENT;
  if ((w1->layout != 0 && w1->layout != 1) || (w2->layout != 0 && w2->layout != 1))
    return NVFP4_INVALID_ARGUMENT;
  if (tokens > 0 && (!x || !y || !topk_idx || !topk_prob)) return NVFP4_INVALID_ARGUMENT;
  if (!aligned(workspace, 256) || (x && !aligned(x, 16)) || (y && !aligned(y, 16)) ||
      !aligned(w1->codes, 16) || !aligned(w2->codes, 16) || !aligned(w1->scales, 4) ||
      !aligned(w2->scales, 4))
    return NVFP4_INVALID_ARGUMENT;
  if ((int64_t)num_experts * 2 * inter >= 0x7FFFFFFFLL ||
      (int64_t)num_experts * hidden >= 0x7FFFFFFFLL)
    return NVFP4_INVALID_ARGUMENT;
  if ((tokens + 1) * (hidden / 2) > 0xFFFFFFFFLL) return NVFP4_UNSUPPORTED;
  if (2 * inter * (hidden / 2) > 0xFFFFFFFFLL || hidden * (inter / 2) > 0xFFFFFFFFLL)
    return NVFP4_UNSUPPORTED;
  SpLayout L = carve_single_pass(workspace, tokens, hidden, inter, topk, num_experts, align);
  if (workspace_bytes < L.bytes) return NVFP4_WORKSPACE_TOO_SMALL;
  const int64_t cap = moe_rows_capacity(tokens, topk, num_experts, align);
  float* y_f32 = nullptr;
  SinglePassArgs sp{};
  if (debug) {
    if ((debug->a1_codes != nullptr) != (debug->a1_scales != nullptr)) return NVFP4_INVALID_ARGUMENT;
    if (debug->expert_offsets) L.offsets = debug->expert_offsets;
    if (debug->dst_row) L.dst_row = debug->dst_row;
    if (debug->row_src) L.row_src = debug->row_src;
    if (debug->row_prob) L.row_prob = debug->row_prob;
    if (debug->y_rows) L.y_rows = debug->y_rows;
    y_f32 = debug->y_rows_f32;
    sp.c_out = debug->fc1_out; sp.p_out = debug->p;
    sp.a2c_out = debug->a2_codes; sp.a2s_out = debug->a2_scales; sp.gs_out = debug->gs_tiles;
    const void* ptrs16[] = {debug->a1_codes, L.y_rows, y_f32};
    for (const void* q : ptrs16)
      if (q && !aligned(q, 16)) return NVFP4_INVALID_ARGUMENT;
    if (debug->a2_codes && !aligned(debug->a2_codes, 8)) return NVFP4_INVALID_ARGUMENT;
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  auto mark = [&](int i) -> hipError_t {
    if (!stage_events || !stage_events[i]) return hipSuccess;
    return hipEventRecord(static_cast<hipEvent_t>(stage_events[i]), s);
  };
  hipError_t e;
  if ((e = mark(0)) != hipSuccess) return NVFP4_HIP_ERROR;
  RouteArgs ra{};
  ra.x = x; ra.tokens = tokens; ra.hidden = hidden;
  ra.topk_idx = topk_idx; ra.topk_prob = topk_prob; ra.topk = topk;
  ra.num_experts = num_experts; ra.align = align;
  ra.offsets = L.offsets; ra.dst_row = L.dst_row; ra.row_src = L.row_src;
  ra.row_prob = L.row_prob; ra.gscale = nullptr;   // the kernel reads tok_gscale through row_src
  ra.tok_codes = L.tokc; ra.tok_scales = L.toks; ra.tok_gscale = L.tokg; ra.entry_rank = L.rank;
  ra.tables[0] = single_pass_table_spec(cap, num_experts, hidden, L.tab);
  ra.num_tables = 1;
  ra.workspace = L.route_ws_i; ra.block_rule = 0;
  if ((e = launch_route(ra, s)) != hipSuccess) return NVFP4_HIP_ERROR;
  if (debug) {
    if ((e = launch_gather_rows(L.tokc, L.toks, L.tokg, L.row_src, L.offsets + num_experts, cap,
                                hidden, debug->a1_codes, debug->a1_scales, debug->a1_gscale,
                                s)) != hipSuccess)
      return NVFP4_HIP_ERROR;
  }
  if ((e = mark(1)) != hipSuccess) return NVFP4_HIP_ERROR;
  sp.a_codes = L.tokc; sp.a_scales = L.toks; sp.a_gscale = L.tokg;
  sp.a_row_src = L.row_src; sp.a_pad_row = tokens; sp.row_prob = L.row_prob;
  sp.w1_codes = w1->codes; sp.w1_scales = w1->scales; sp.w1_gscale = w1->gscale;
  sp.w1_layout = w1->layout;
  sp.w2_codes = w2->codes; sp.w2_scales = w2->scales; sp.w2_gscale = w2->gscale;
  sp.w2_layout = w2->layout;
  sp.hidden = hidden; sp.inter = inter; sp.tile_table = L.tab;
  sp.y_bf16 = L.y_rows; sp.y_f32 = y_f32;
  if ((e = launch_single_pass(sp, L.blocks, s)) != hipSuccess) return NVFP4_HIP_ERROR;
  if ((e = mark(2)) != hipSuccess) return NVFP4_HIP_ERROR;
  if ((e = launch_combine(y_f32 ? static_cast<const void*>(y_f32) : L.y_rows, y_f32 ? 0 : 1,
                          L.dst_row, tokens, topk, hidden, y, s)) != hipSuccess)
    return NVFP4_HIP_ERROR;
  if ((e = mark(3)) != hipSuccess) return NVFP4_HIP_ERROR;
  return NVFP4_OK;
}

}  // extern "C"
