// matvec.hip -- products of a few unquantized rows with NVFP4 weights, and
// the expert layer's projections for a few tokens:
//   y[t, n] = s_g sum_k (q s_b)[n, k] x[t, k]
// with W one [n, k] matrix, or matrix e of a group for the entry (t, j) whose
// expert id is e.
//
// Arithmetic: a weight's q s_b has at most 6 significant bits and lies in
// [2^-10, 2688], so it is exact in bf16 and in fp16 and goes to the matrix
// cores in the type of x; products are exact in the binary32 accumulator and
// s_g multiplies the sum.  binary32 x is split into three bf16 parts by
// truncation (8 + 8 + 8 significant bits, an exact sum) and takes three
// products.  The layer's intermediate D is a binary32 value whatever the type of
// x; FC1 writes it as its three parts, one plane each, so that FC2 multiplies
// them without splitting again (FC2 splitting a binary32 D cost one token of the
// layer 3 us of 16, 256 tokens 7 of 109).
//
// Mapping: a wave multiplies 16 weight rows (32 with SwiGLU: 16 gate and the
// 16 up rows) with 16 columns, a column being a row of x: v_mfma 16x16x32
// with the weights as its A operand.  A lane owns 32 consecutive k of one
// weight row per 128-element stage -- 16 bytes of codes, two block scales and
// the same 32 elements of its column -- and feeds them to four products, 8 k
// each; the order of k inside a sum is free as both operands share it.  The
// waves of a workgroup take the stages in turn and their sums are added in
// LDS in wave order, so results do not depend on timing.
//
// Bound: the weights' bytes (9/16 per weight); x comes from the caches.
// Two kernels: matvec_kernel gives every 16 rows a workgroup whose waves split
// k, for little work and few columns; matvec_rows_kernel gives a workgroup 64
// or 128 rows and shares x through LDS.  Measured kernel times: one bf16 row
// by [5120, 2048] 4.9 us (one round of loads, a reduction and two launches'
// latency: 1.2 TB/s), by [16384, 4096] 3.3 TB/s (both the direct kernel); by
// [32768, 8192] 1 to 16 rows 4.1 TB/s, 64 rows 2.8 TB/s (the LDS kernel).
#include "elem.h"
#include "gemm_common.h"
#include "launch.h"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// How x travels: 0 binary32, 1 bf16, 2 fp16, 3 a binary32 value as three planes of
// bf16 parts, a.x_plane elements apart (the layer's D)
constexpr int kPlanes = 3;
constexpr int parts_of(int xt) { return xt == 0 || xt == kPlanes ? 3 : 1; }
constexpr int kStage = 128;   // k elements of a stage
constexpr int kTile = 16;     // weight rows of a tile, columns of a product

// 32 elements of a column: one stage of a lane.
template <int XT>
struct XStage {
  static constexpr int kWords = XT == 0 ? 8 : (XT == kPlanes ? 12 : 4);
  uint4 w[kWords];
};

// `plane`: bytes from one part's plane to the next.
template <int XT>
__device__ __forceinline__ XStage<XT> load_x(const char* p, int64_t plane) {
  XStage<XT> x;
  if (XT == kPlanes) {
#pragma unroll
    for (int i = 0; i < 3; ++i) __builtin_memcpy(&x.w[4 * i % XStage<XT>::kWords], p + i * plane, 64);
  } else {
    __builtin_memcpy(&x.w[0], p, XT == 0 ? 128 : 64);
  }
  return x;
}

// Part `part` of elements [8s, 8s + 8) of the stage as an operand.
template <int XT>
__device__ __forceinline__ uint4 x_operand(const XStage<XT>& x, int s, int part) {
  if (XT == kPlanes) return x.w[(part * 4 + s) % XStage<XT>::kWords];
  if (XT != 0) return x.w[s];
  // Upper halves of the value (a quiet NaN stays one), of what is left of it, and
  // of the rest.  The lower parts are the largest finite value's for an
  // infinity, whose difference would be NaN: they add to it with its sign.
  const uint4 a = x.w[(2 * s) % XStage<XT>::kWords], b = x.w[(2 * s + 1) % XStage<XT>::kWords];
  uint32_t f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (part > 0)
      f[i] = __float_as_uint(__builtin_amdgcn_fmed3f(__uint_as_float(f[i]), -__FLT_MAX__, __FLT_MAX__));
    for (int p = 0; p < part; ++p)
      f[i] = __float_as_uint(__uint_as_float(f[i]) - __uint_as_float(f[i] & 0xFFFF0000u));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    o[i] = __builtin_amdgcn_perm(f[2 * i + 1], f[2 * i], 0x07060302u);
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// 8 codes times their block scale (binary32) as bf16, exactly.
__device__ __forceinline__ bf16x8_t decode8_bf16(uint32_t c, float sb) {
  const f32x2_t h0 = fp4_pair_value<0>(c), h1 = fp4_pair_value<1>(c);
  const f32x2_t h2 = fp4_pair_value<2>(c), h3 = fp4_pair_value<3>(c);
  uint32_t w[4] = {pack_bf16x2(h0[0] * sb, h0[1] * sb), pack_bf16x2(h1[0] * sb, h1[1] * sb),
                   pack_bf16x2(h2[0] * sb, h2[1] * sb), pack_bf16x2(h3[0] * sb, h3[1] * sb)};
  bf16x8_t r;
  __builtin_memcpy(&r, w, 16);
  return r;
}

// Two E4M3 bytes (bits 0-7 and 8-15) as binary32, exactly: the hardware
// conversion reads the OCP format, subnormals included (the NaN byte 0x7F is
// no scale).
__device__ __forceinline__ f32x2_t block_scales(uint32_t s) {
  return __builtin_amdgcn_cvt_pk_f32_fp8((int)s, false);
}

// One stage of one 16-row tile: c = the lane's 32 codes, sb = its two E4M3
// bytes (the second block's in bits 8-15).
template <int XT>
__device__ __forceinline__ void stage_product(f32x4_t& acc, const uint4& c, uint32_t sb,
                                              const XStage<XT>& x) {
  const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
  const f32x2_t s2 = block_scales(sb);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if (XT == 2) {
      const _Float16 h = (_Float16)s2[s / 2];
      const half8_t a = decode8(cw[s], (half2_t){h, h});
      const uint4 xo = x_operand<XT>(x, s, 0);
      half8_t b;
      __builtin_memcpy(&b, &xo, 16);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, acc, 0, 0, 0);
    } else {
      const bf16x8_t a = decode8_bf16(cw[s], s2[s / 2]);
#pragma unroll
      for (int p = 0; p < parts_of(XT); ++p) {
        const uint4 xo = x_operand<XT>(x, s, p);
        bf16x8_t b;
        __builtin_memcpy(&b, &xo, 16);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
      }
    }
  }
}

// A lane's place in one matrix: address of its codes and scales of stage 0
// and what a stage advances them by.
struct LanePlace {
  const uint8_t* codes;
  const uint8_t* scales;
};

__device__ __forceinline__ LanePlace lane_place(const MatvecArgs& a, int e, int64_t row, int q) {
  const uint8_t* c = a.codes + (int64_t)e * a.n * (a.k / 2);
  const uint8_t* s = a.scales + (int64_t)e * a.n * (a.k / 16);
  if (a.layout == 0) return {c + row * (a.k / 2) + 16 * q, s + row * (a.k / 16) + 2 * q};
  const int64_t tile = (row / 32) * (a.k / kStage);
  const int in = (int)(row % 32) + 32 * (q / 2);
  return {c + tile * 2048 + (q % 2) * 1024 + 16 * in, s + tile * 256 + 4 * in + 2 * (q % 2)};
}

__device__ __forceinline__ uint32_t load_u16(const uint8_t* p) {
  uint16_t v;
  __builtin_memcpy(&v, p, 2);
  return v;
}
__device__ __forceinline__ uint4 load_u128(const uint8_t* p) {
  uint4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// The entries whose expert is e (e == num_groups: of no expert) into `list`,
// returning their number.  The order is the same in every workgroup that lists
// e (several may share its columns): by wave, each wave's in ascending order.
// `ids` holds topk_idx[threadIdx.x + i * blockDim.x], loaded by the caller
// ahead of other work; more entries are read in rounds of as many loads.
// `counts` is a word of LDS per wave.
constexpr int kIds = 8;
__device__ __forceinline__ void load_ids(const MatvecArgs& a, int at, int entries, int (&ids)[kIds]) {
#pragma unroll
  for (int i = 0; i < kIds; ++i) {
    const int j = at + i * (int)blockDim.x;
    // (no load where no thread of the workgroup has an entry left)
    if (at - (int)threadIdx.x + i * (int)blockDim.x < entries)
      ids[i] = a.topk_idx[j < entries ? j : 0];
  }
}
template <int WAVES>
__device__ __forceinline__ int collect_entries(const MatvecArgs& a, int e, int (&ids)[kIds],
                                               int entries, uint16_t* list, int* counts) {
  constexpr int kThreads = WAVES * kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  int m = 0;
  for (int base = 0; base < entries; base += kIds * kThreads) {
    if (base != 0) load_ids(a, base + threadIdx.x, entries, ids);
    uint64_t mask[kIds];
    int n = 0;
#pragma unroll
    for (int i = 0; i < kIds; ++i) {
      const int first = base + i * kThreads;
      mask[i] = 0;
      if (first >= entries) continue;   // (the whole workgroup's)
      const int of = ids[i] >= 0 && ids[i] < a.num_groups ? ids[i] : a.num_groups;
      mask[i] = __ballot(first + (int)threadIdx.x < entries && of == e);
      n += __popcll(mask[i]);
    }
    if (threadIdx.x % kWave == 0) counts[wave] = n;
    __syncthreads();
    int c[WAVES], at = m;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) c[w] = counts[w];
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      at += w < wave ? c[w] : 0;
      m += c[w];
    }
#pragma unroll
    for (int i = 0; i < kIds; ++i) {
      if (mask[i] == 0) continue;
      const int before = __builtin_amdgcn_mbcnt_hi(
          (uint32_t)(mask[i] >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask[i], 0));
      if ((mask[i] >> (threadIdx.x % kWave)) & 1)
        list[at + before] = (uint16_t)(base + i * kThreads + threadIdx.x);
      at += __popcll(mask[i]);
    }
    __syncthreads();
  }
  return m;
}

// Stores the values of rows [row, row + 4) of one column (those below n): one
// store where n is a multiple of 4, as row is.
template <int DT>
__device__ __forceinline__ void store4_as(void* out, int64_t at, int count, bool four, f32x4_t v) {
  typename Elem<DT>::type o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = Elem<DT>::from_float(v[i]);
  typename Elem<DT>::type* p = static_cast<typename Elem<DT>::type*>(out) + at;
  if (four) {
    if (count > 0) __builtin_memcpy(p, o, sizeof(o));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < count) p[i] = o[i];
  }
}
__device__ __forceinline__ void store4(const MatvecArgs& a, int64_t out_row, int64_t row, f32x4_t v) {
  const int64_t at = out_row * a.n + row, left = a.n - row;
  const int count = left < 4 ? (int)left : 4;
  const bool four = a.n % 4 == 0;
  if (a.out_dtype == 0) store4_as<0>(a.out, at, count, four, v);
  else if (a.out_dtype == 1) store4_as<1>(a.out, at, count, four, v);
  else store4_as<2>(a.out, at, count, four, v);
}

// Zero results for the listed entries' rows [row, row + count).
__device__ __forceinline__ void store_zeros(const MatvecArgs& a, const uint16_t* list, int m,
                                            int64_t row, int count) {
  for (int i = threadIdx.x; i < m * (count / 4); i += blockDim.x)
    store4(a, list[i / (count / 4)], row + 4 * (i % (count / 4)), (f32x4_t){0.f, 0.f, 0.f, 0.f});
}

// silu(g) u p; the product is binary64 and rounded once, so no part of it leaves
// binary32's range before the whole does.  Below g = -80, where binary32 exp(-g)
// overflows and e^g leaves the normal range, silu(g) = g e^g (1 + e^g is one) with
// e^g = 2^n e^f, |f| <= ln 2 / 2, the power of two applied in binary64.  Below -700
// g counts as -700, where D is zero for any finite u and p and an infinity for an
// infinite u.  Both branches share the exponential: a binary64 exp in a branch of
// its own took 20 to 50 registers and a wave per SIMD from the kernels.
__device__ __forceinline__ float weighted_swiglu(float g, float u, float p) {
  constexpr double kLn2 = 0.69314718055994530942;
  constexpr float kHigh = (float)kLn2, kLow = (float)(kLn2 - kHigh);
  const bool tail = g < -80.0f && g >= -__FLT_MAX__;
  const float gt = __builtin_amdgcn_fmed3f(g, -700.0f, 0.0f), n = rintf(gt * (float)(1.0 / kLn2));
  const float f = fmaf(-n, kLow, fmaf(-n, kHigh, gt));
  const float e = expf(tail ? f : -g);
  const double s = tail ? ldexp((double)gt * e, (int)n) : (double)(g / (1.0f + e));
  return (float)(s * u * p);
}

// The layer's D of one entry, silu(g) u p in binary32, as its three bf16 parts:
// the upper half of its bits, of what is left of it, and the rest -- an exact
// sum.  The lower parts of an infinity are zero (inf - inf would be NaN).
__device__ __forceinline__ void store_d4(const MatvecArgs& a, int64_t entry, int64_t col, f32x4_t g,
                                         f32x4_t u, float p) {
  uint16_t part[3][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float d = weighted_swiglu(g[i], u[i], p);
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      const uint32_t top = __float_as_uint(d) & 0xFFFF0000u;
      part[q][i] = (uint16_t)(top >> 16);
      d = fabsf(d) < __builtin_huge_valf() ? d - __uint_as_float(top) : 0.0f;
    }
  }
#pragma unroll
  for (int q = 0; q < 3; ++q)
    __builtin_memcpy(a.d + q * a.d_plane + entry * a.inter + col, part[q], 8);
}

}  // namespace

// The n-th set bit of a mask (n below its population).
__device__ __forceinline__ int nth_bit(uint64_t mask, int n) {
  for (int i = 0; i < n; ++i) mask &= mask - 1;
  return __builtin_ctzll(mask);
}

// The entries of expert e, found by every wave on its own (one ballot per 64
// ids, no LDS and no barrier).  *entry is that of column c0 + r, or some other
// entry of e where the column is past the last; returns their number, or 0 if
// an entry before `slot` is among them.
__device__ __forceinline__ int find_entries(const MatvecArgs& a, int e, int entries, int slot, int c0,
                                            int r, int* entry) {
  const int lane = threadIdx.x % kWave;
  int m = 0;
  for (int base = 0; base < entries; base += kWave) {
    const int i = base + lane;
    const int id = a.topk_idx[i < entries ? i : 0];
    const uint64_t mask = __ballot(i < entries && id == e);
    if (mask == 0) continue;
    if (base + __builtin_ctzll(mask) < slot) return 0;
    const int n = __popcll(mask), want = c0 + r - m;
    if (m == 0) *entry = base + __builtin_ctzll(mask);
    if (want > 0 && want < n) *entry = base + nth_bit(mask, want);
    if (want == 0) *entry = base + __builtin_ctzll(mask);
    m += n;
  }
  return m;
}

// acc += the products of stages st, st + step, ... of the lane's rows, two
// stages in flight.  With k no multiple of 128 (row-major weights) the stage
// behind the last whole one, a multiple of 16, is taken too: a lane has none,
// half or all of its 32 elements there.
template <int XT, int RT>
__device__ __forceinline__ void stage_loop(const MatvecArgs& a, f32x4_t (&acc)[RT],
                                           const LanePlace (&place)[RT], const char* xp, int q,
                                           int st, int step) {
  constexpr int xsize = XT == 0 ? 4 : 2;
  const int64_t plane = a.x_plane * 2;
  const int64_t cstep = a.layout == 0 ? kStage / 2 : 2048, sstep = a.layout == 0 ? kStage / 16 : 256;
  const int stages = (int)(a.k / kStage);
  for (; st < stages; st += 2 * step) {
    const int st2 = st + step < stages ? st + step : st;
    uint4 c[2][RT];
    uint32_t sb[2][RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      c[0][rt] = load_u128(place[rt].codes + st * cstep);
      sb[0][rt] = load_u16(place[rt].scales + st * sstep);
    }
    const XStage<XT> x0 = load_x<XT>(xp + (int64_t)st * kStage * xsize, plane);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      c[1][rt] = load_u128(place[rt].codes + st2 * cstep);
      sb[1][rt] = load_u16(place[rt].scales + st2 * sstep);
    }
    const XStage<XT> x1 = load_x<XT>(xp + (int64_t)st2 * kStage * xsize, plane);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) stage_product<XT>(acc[rt], c[0][rt], sb[0][rt], x0);
    if (st2 != st) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) stage_product<XT>(acc[rt], c[1][rt], sb[1][rt], x1);
    }
  }
  if (a.k % kStage != 0 && st % step == stages % step) {
    const int left = (int)(a.k - (int64_t)stages * kStage) - 32 * q;
    XStage<XT> x = {};
    uint4 c[RT] = {};
    uint32_t sb[RT] = {};
    if (left >= 16) {
      xp += (int64_t)stages * kStage * xsize;
      if (left >= 32) {
        x = load_x<XT>(xp, plane);
      } else {
#pragma unroll
        for (int i = 0; i < (XT == kPlanes ? 3 : 1); ++i)
          __builtin_memcpy(&x.w[4 * i % XStage<XT>::kWords], xp + i * plane, 16 * xsize);
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const uint8_t* pc = place[rt].codes + stages * cstep;
        const uint8_t* ps = place[rt].scales + stages * sstep;
        if (left >= 32) {
          c[rt] = load_u128(pc);
          sb[rt] = load_u16(ps);
        } else {
          __builtin_memcpy(&c[rt], pc, 8);
          sb[rt] = *ps;
        }
      }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) stage_product<XT>(acc[rt], c[rt], sb[rt], x);
  }
}

// The value N lanes further on in the lane's row of 16 (zero past its end).
template <int N>
__device__ __forceinline__ float row_ahead(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x100 + N, 0xf, 0xf, true));   // row_shl:N
}

// Grid: x = 16-row tiles of the output, y = slots (EXPERT) or chunks of 16
// columns.  A slot is an entry when there are no more entries than experts
// (the first entry of an expert does the work of all of its entries), else an
// expert, with one more slot for the entries of no expert.
template <int XT, bool SWIGLU, bool EXPERT>
__global__ __launch_bounds__(512) void matvec_kernel(MatvecArgs a) {
  constexpr int RT = SWIGLU ? 2 : 1;
  extern __shared__ char lds[];
  const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int waves = blockDim.x / kWave;
  const int r = lane % kTile, q = lane / kTile;
  const int64_t row0 = (int64_t)blockIdx.x * kTile;
  f32x4_t* red = reinterpret_cast<f32x4_t*>(lds);
  const int entries = EXPERT ? (int)a.tokens * a.topk : 0, slot = blockIdx.y;
  const bool by_entry = EXPERT && entries <= a.num_groups;
  int e = 0, m = (int)a.tokens, first = 0, entry = 0;
  if (EXPERT) {
    e = by_entry ? a.topk_idx[slot] : slot;
    if (e < 0 || e >= a.num_groups) {
      // entries of no expert: zero results, this one's or all of them
      if (SWIGLU || a.skip_unrouted) return;
      for (int i = by_entry ? slot : threadIdx.x; i < (by_entry ? slot + 1 : entries); i += blockDim.x) {
        const int id = a.topk_idx[i];
        if ((id >= 0 && id < a.num_groups) || (by_entry && threadIdx.x != 0)) continue;
        for (int c = 0; c < kTile; c += 4) store4(a, i, row0 + c, (f32x4_t){0.f, 0.f, 0.f, 0.f});
      }
      return;
    }
    m = find_entries(a, e, entries, by_entry ? slot : 0, 0, r, &entry);
    if (m == 0) return;
  } else {
    first = blockIdx.y * kTile;
    m = m < first + kTile ? m : first + kTile;
  }
  LanePlace place[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    // rows past the last read the last one (and are not stored)
    int64_t row = row0 + r + (SWIGLU ? rt * a.inter : 0);
    if (!SWIGLU && row >= a.n) row = a.n - 1;
    place[rt] = lane_place(a, e, row, q);
  }
  constexpr int xsize = XT == 0 ? 4 : 2;
  const float sg = a.gscale[e];
  for (int c0 = first; c0 < m; c0 += kTile) {
    // columns past the last read another's row (and are not stored)
    if (!EXPERT) entry = c0 + r < m ? c0 + r : m - 1;
    else if (c0 != 0) find_entries(a, e, entries, 0, c0, r, &entry);
    const int64_t xrow = EXPERT && !a.x_by_entry ? entry / a.topk : entry;
    const char* xp = static_cast<const char*>(a.x) + (xrow * a.ld_x + 32 * q) * xsize;
    const float p = SWIGLU ? a.prob[entry] : 1.0f;
    f32x4_t acc[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) acc[rt] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
    stage_loop<XT, RT>(a, acc, place, xp, q, wave, waves);
    if (c0 != first) __syncthreads();   // the last chunk's sums have been read
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) red[(wave * RT + rt) * kWave + lane] = acc[rt];
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        f32x4_t s = red[rt * kWave + lane];
        for (int w = 1; w < waves; ++w) s += red[(w * RT + rt) * kWave + lane];
        acc[rt] = s * sg;
      }
      if (c0 + r < m) {
        if (SWIGLU) store_d4(a, entry, row0 + 4 * q, acc[0], acc[RT - 1], p);
        else store4(a, entry, row0 + 4 * q, acc[0]);
      }
    }
  }
}

// The layer's FC2 and the sum over a token's experts in one: grid x = 16-row
// tiles, y = tokens; `parts` waves share the stages of one of the token's
// entries and the workgroup's wave sets take the entries in turn.  D's three
// parts are three columns of one product (the others repeat the first and are
// not used).  An entry's sums meet in LDS, so that it is whole, and rounded,
// before the entries are added in ascending order, as in the separate kernels.
__global__ __launch_bounds__(1024) void decode_down_kernel(MatvecArgs a, int parts) {
  extern __shared__ char lds[];
  const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int waves = blockDim.x / kWave, sets = waves / parts;
  const int r = lane % kTile, q = lane / kTile;
  const int64_t row0 = (int64_t)blockIdx.x * kTile, t = blockIdx.y;
  f32x4_t* red = reinterpret_cast<f32x4_t*>(lds);               // [topk, parts, 4]
  float* outer = reinterpret_cast<float*>(red + a.topk * parts * 4);   // [topk]
  for (int j = wave / parts; j < a.topk; j += sets) {
    const int64_t entry = t * a.topk + j;
    const int e = a.topk_idx[entry];
    float sg = 0.0f;                                            // an entry of no expert adds zero
    f32x4_t acc[1] = {(f32x4_t){0.f, 0.f, 0.f, 0.f}};
    if (e >= 0 && e < a.num_groups) {
      sg = a.gscale[e];
      const int64_t row = row0 + r;
      const LanePlace place[1] = {lane_place(a, e, row < a.n ? row : a.n - 1, q)};
      const int64_t at = (r < 3 ? r : 0) * a.x_plane + entry * a.ld_x + 32 * q;
      stage_loop<1, 1>(a, acc, place, static_cast<const char*>(a.x) + at * 2, q, wave % parts, parts);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[0][i] = acc[0][i] + row_ahead<1>(acc[0][i]) + row_ahead<2>(acc[0][i]);
    }
    if (r == 0) red[(j * parts + wave % parts) * 4 + q] = acc[0];
    if (lane == 0) outer[j] = sg;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.topk * 4; i += blockDim.x) {
    f32x4_t* own = red + i / 4 * parts * 4 + i % 4;
    f32x4_t y = own[0];
    for (int p = 1; p < parts; ++p) y += own[4 * p];
    own[0] = y * outer[i / 4];
  }
  __syncthreads();
  if (threadIdx.x < 4) {
    f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < a.topk; ++j) sum += red[j * parts * 4 + threadIdx.x];
    store4(a, t, row0 + 4 * threadIdx.x, sum);
  }
}

// ---- more columns: x staged in LDS --------------------------------------
//
// From a handful of columns on, a wave's own reads of x cost more than its
// weights (a 16-column operand is 4 KiB a stage beside 1.1 KiB of weights).
// Here a workgroup's waves take 32 rows each (16 gate and 16 up rows with
// SwiGLU), in one, two or four groups that take the stages in turn, and share 16
// NC columns of x, brought into LDS once per workgroup as the parts' bf16 /
// fp16 values, double buffered.  Each wave keeps kDepth stages of its weights
// in flight in registers; loads past the last stage are out of the buffer's
// range and cost nothing, and what they return, zeros, adds nothing.
//
// Shapes (waves of a group x groups), by measurement: experts 4 x 1, as many
// small workgroups that overlap each other's prologue (entries listed, x
// brought in) with streaming -- two groups ran the layer of 256 tokens in 141
// us, two waves a group in 131, against 108 -- and 2 x 2 where that makes no more
// than two workgroups a CU, so that latency counts (k 4096, 8 columns: 8 experts
// of 2048 rows 15.5 against 22 us, 16 of 512 14.6 against 21.8; 32 of 2048, 1024
// workgroups, 37 against 35).  One matrix: 64 rows a workgroup (n 16384, k 4096,
// 16 rows: 14.4 us, 17.3 with 128 rows) and as many columns as leave a workgroup
// for every CU (k 8192, 64 rows: n 4096, 16 columns 18 us, 32 22.6, 64 32; n 8192
// 27, 24, 33); four groups while there is no second workgroup for a CU, else two
// (k 8192, 16 rows: n 8192 17.5 / 22.7 us; n 24576, k 4096, 64 rows 39 / 33); and
// 4 x 2 where 64 columns of x make 128 rows worth a workgroup (55 against 66 us).
// More stages in flight cost occupancy (four: 127 against 109 us), and do not
// help the small grids either (8 to 15% slower).
//
// What bounds it: with 1-2 columns of 16, the weights' stream (FC1 of 256
// tokens 54 us, 226 MB at 4.2 TB/s; FC2 47 us, where D's three planes, which
// eight row blocks read each, and the rows come on top of 113 MB).  With 64
// columns the compute side shows: a copy without any global traffic took 40 of
// the 56-65 us (decode, products and LDS reads at two waves a SIMD), and
// row-major weights add the block scales' scattered 2-byte loads (54 us without
// them); the tiled layout is the faster one.
//
// The last stage of a k that is no multiple of 128 (row-major weights):
// lanes take the window [min(k0, k - 32), + 32) instead of [k0, + 32), and x
// is zero wherever the window leaves [k0, k), so the loads need no branch.

namespace {

constexpr int kWide = 2;               // 16-row tiles of a wave
// The workgroup's shape: waves of a group (32 rows each), and groups, taking
// the stages in turn.
template <int XT, int NC, int ROW_WAVES, int GROUPS>
struct RowsShape {
  static constexpr int kThreads = GROUPS * ROW_WAVES * kWave;
  // an LDS buffer: one stage of every group
  static constexpr int kBuffer = GROUPS * parts_of(XT) * NC * kTile * kStage * 2;
};
constexpr int kDepth = 2;              // stages of weights and of x on their way

// A wave's weights of one stage.
struct WStage {
  u32x4_t c[kWide];
  uint32_t s[kWide];
};

// 8 elements of a column on their way to LDS.
template <int XT>
struct XPiece {
  static constexpr int kWords = XT == 0 ? 2 : (XT == kPlanes ? 3 : 1);
  u32x4_t w[kWords];
};

// A column's stage is 16 pieces of 8 elements, piece 4q + s in slot
// slot_of(q, s) ^ (column % 16).  A 16-byte LDS read serves lanes 0-3, 12-15, 20-23 and 24-27 of
// each half wave together; with the quarters in this order those lanes, eight
// columns of quarter q and the eight others of q + 1, meet different banks
// (in the plain order they met in pairs, 4 extra cycles a read).
__device__ __forceinline__ int slot_of(int q, int s) { return 4 * ((q >> 1) ^ (q & 1 ? 3 : 0)) + s; }

template <int XT>
__device__ __forceinline__ uint4 piece_part(const XPiece<XT>& v, int part) {
  const u32x4_t& a = v.w[XT == kPlanes ? part % XPiece<XT>::kWords : 0];
  if (XT != 0) return make_uint4(a[0], a[1], a[2], a[3]);
  const u32x4_t& b = v.w[1 % XPiece<XT>::kWords];
  XStage<0> x;
  x.w[0] = make_uint4(a[0], a[1], a[2], a[3]);
  x.w[1] = make_uint4(b[0], b[1], b[2], b[3]);
  return x_operand<0>(x, 0, part);
}

}  // namespace

template <int XT, int NC, int ROW_WAVES, int GROUPS, bool SWIGLU, bool EXPERT>
__global__ __launch_bounds__(ROW_WAVES* GROUPS* kWave) void matvec_rows_kernel(MatvecArgs a) {
  typedef RowsShape<XT, NC, ROW_WAVES, GROUPS> Shape;
  constexpr int kRowWaves = ROW_WAVES, kGroups = GROUPS, kSets = kDepth;
  constexpr int kThreads = Shape::kThreads, kLines = kThreads / 16;
  constexpr int kCols = NC * kTile, kParts = parts_of(XT);
  constexpr int XS = kGroups;                             // stages of a buffer
  constexpr int kColBytes = kStage * 2;                   // one part of a column's stage
  constexpr int kPlane = kCols * kColBytes;
  constexpr int kBuffer = Shape::kBuffer;
  constexpr int kOwn = XS * NC * 256 / kThreads;          // pieces a thread brings per buffer
  constexpr int xsize = XT == 0 ? 4 : 2;
  static_assert(kDepth % 2 == 0 && kDepth % kSets == 0, "buffers and sets turn in the loop");
  // No static LDS in this kernel: the dynamic part would begin behind it, and
  // at an address that is no multiple of 16 the buffers' 16-byte accesses run
  // at half their rate (the layer of 256 tokens took 240 us instead of 110).
  extern __shared__ __align__(16) char lds[];
  int* counts = reinterpret_cast<int*>(lds + 2 * kBuffer);
  uint16_t* list = reinterpret_cast<uint16_t*>(counts + kThreads / kWave);
  const int lane = threadIdx.x % kWave, wid = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wave = wid % kRowWaves, group = kGroups == 1 ? 0 : wid / kRowWaves;
  const int r = lane % kTile, q = lane / kTile;
  int e = 0, m = (int)a.tokens, first = 0;
  // first row of the wave: of the output, or of the gate half
  const int64_t row0 = ((int64_t)blockIdx.x * kRowWaves + wave) * (SWIGLU ? kTile : kWide * kTile);
  const int64_t rows = SWIGLU ? a.inter : a.n;
  int ids[kIds];
  const int entries = EXPERT ? (int)a.tokens * a.topk : 0;
  if (EXPERT) {
    e = blockIdx.y;
    first = blockIdx.z * kCols;
    if (e == a.num_groups && (SWIGLU || a.skip_unrouted || first != 0)) return;
    load_ids(a, threadIdx.x, entries, ids);
  } else {
    first = blockIdx.y * kCols;
    m = m < first + kCols ? m : first + kCols;
  }
  const int em = EXPERT && e == a.num_groups ? 0 : e;     // a matrix whose addresses are valid
  const int k = (int)a.k, stages = (k + kStage - 1) / kStage;
  const bool ragged = k % kStage != 0;                    // the last stage is a partial one
  const int64_t matrix = a.n * (a.k / 2);                 // bytes of its codes, below 2^31
  const __amdgpu_buffer_rsrc_t codes = buffer_rsrc(a.codes + em * matrix, (uint32_t)matrix);
  const uint8_t* scales = a.scales + em * (matrix / 8);
  uint32_t wc[kWide], ws[kWide], wc_last[kWide], ws_last[kWide];
#pragma unroll
  for (int rt = 0; rt < kWide; ++rt) {
    // rows past the last read the last one (and are not stored)
    int64_t row = row0 + r + (SWIGLU ? 0 : rt * kTile);
    if (row >= rows) row = rows - 1;
    row += SWIGLU ? rt * a.inter : 0;
    const LanePlace p = lane_place(a, em, row, q);
    wc[rt] = (uint32_t)(p.codes - (a.codes + em * matrix));
    ws[rt] = (uint32_t)(p.scales - scales);
    const int k0 = (stages - 1) * kStage + 32 * q, at = k0 < k - 32 ? k0 : k - 32;
    wc_last[rt] = (uint32_t)(row * (k / 2) + at / 2);
    ws_last[rt] = (uint32_t)(row * (k / 16) + at / 16);
  }
  const int cstep = a.layout == 0 ? kStage / 2 : 2048, sstep = a.layout == 0 ? kStage / 16 : 256;
  // the wave's turn-th stage
  auto load_w = [&](int turn) {
    WStage w;
    const int i = turn * kGroups + group;
    const bool none = i >= stages;
    const int at = none ? 0 : i;
    const bool last = ragged && at == stages - 1;
#pragma unroll
    for (int rt = 0; rt < kWide; ++rt) {
      w.c[rt] = __builtin_amdgcn_raw_buffer_load_b128(
          codes, none ? kNone : (last ? wc_last[rt] : wc[rt]), last ? 0 : at * cstep, 0);
      w.s[rt] = load_u16(scales + (last ? 0 : at * sstep) + (last ? ws_last[rt] : ws[rt]));
    }
    return w;
  };
  const float sg = a.gscale[em];
  // the first weights are on their way while the entries are listed
  WStage w[kDepth];
#pragma unroll
  for (int d = 0; d < kDepth; ++d) w[d] = load_w(d);
  if (EXPERT) {
    m = collect_entries<kThreads / kWave>(a, e, ids, entries, list, counts);
    if (first >= m) return;
    if (e == a.num_groups) {   // entries of no expert
      store_zeros(a, list, m, row0 - wave * kWide * kTile, kRowWaves * kWide * kTile);
      return;
    }
  }
  // A thread brings slot threadIdx.x % 16 of every kLines-th line, a line being
  // a column's stage (line = stage * kCols + column; a wave's four lines are of
  // one stage).  Columns past the last and stages past the last are out of the
  // buffer's range: zeros, and no traffic.
  const int64_t xrows = EXPERT && a.x_by_entry ? entries : a.tokens;
  // (the planes one behind the other are one buffer; below 2^31)
  const uint32_t plane = XT == kPlanes ? (uint32_t)(a.x_plane * 2) : 0;
  const uint32_t xbytes = (uint32_t)(((xrows - 1) * a.ld_x + a.k) * xsize) + 2 * plane;
  const __amdgpu_buffer_rsrc_t xres = buffer_rsrc(a.x, xbytes);
  const int slot = threadIdx.x % 16, own = threadIdx.x / 16;
  const int pi = slot ^ (own % 16), pm = pi / 4;
  const int piece = 4 * ((((pm ^ (pm >> 1)) & 1) << 1) | (pm >> 1)) + pi % 4;   // slot_of's inverse
  const int turns = (stages + kGroups - 1) / kGroups;
  for (int c0 = first; c0 < m; c0 += kCols * (EXPERT ? (int)gridDim.z : 1)) {
    uint32_t xo[kOwn], xo_last[kOwn];
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int col = c0 + (i * kLines + own) % kCols;
      uint32_t at = kNone;
      if (col < m) {
        const int entry = EXPERT ? list[col] : col;
        const int64_t xrow = EXPERT && !a.x_by_entry ? entry / a.topk : entry;
        at = (uint32_t)(xrow * a.ld_x * xsize);
      }
      xo[i] = at + 8 * piece * xsize;
      // the window of the last, partial stage (see above)
      const int k0 = (stages - 1) * kStage + 32 * (piece / 4);
      const int kw = (k0 < k - 32 ? k0 : k - 32) + 8 * (piece % 4);
      xo_last[i] = kw >= k0 && kw < k ? at + kw * xsize : kNone;
    }
    // pieces on their way to the next kSets buffers
    XPiece<XT> xr[kSets][kOwn];
    auto load_xs = [&](int set, int st0) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int nth = st0 + (i * kLines + wid * 4) / kCols;
        const bool none = nth >= stages;
        const int st = none ? 0 : nth;
        const bool last = ragged && st == stages - 1;
        const uint32_t lo = none ? kNone : (last ? xo_last[i] : xo[i]);
        const int un = none || last ? 0 : st * kStage * xsize;
#pragma unroll
        for (int w = 0; w < XPiece<XT>::kWords; ++w)
          xr[set][i].w[w] = __builtin_amdgcn_raw_buffer_load_b128(xres, lo + (XT == 0 ? 16 * w : 0),
                                                                  un + w * plane, 0);
      }
    };
    auto store_xs = [&](int set, int buf) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int line = i * kLines + own;
#pragma unroll
        for (int p = 0; p < kParts; ++p)
          *reinterpret_cast<uint4*>(lds + buf * kBuffer + ((line / kCols) * kParts + p) * kPlane +
                                    (line % kCols) * kColBytes + slot * 16) = piece_part<XT>(xr[set][i], p);
      }
    };
    f32x4_t acc[kWide][NC];
#pragma unroll
    for (int rt = 0; rt < kWide; ++rt)
#pragma unroll
      for (int b = 0; b < NC; ++b) acc[rt][b] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kSets; ++i) load_xs(i, i * XS);
    if (c0 != first) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) w[d] = load_w(d);
      __syncthreads();                                    // the last columns' sums have been read
    }
    store_xs(0, 0);
    __syncthreads();
    for (int t0 = 0; t0 < turns; t0 += kDepth) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        const int turn = t0 + d, buf = d % 2;
        load_xs(d % kSets, (turn + kSets) * kGroups);
        {
          const char* xb0 = lds + buf * kBuffer + group * kParts * kPlane;
          f32x2_t s2[kWide];
#pragma unroll
          for (int rt = 0; rt < kWide; ++rt) s2[rt] = block_scales(w[d].s[rt]);
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            uint4 xv[kParts][NC];
#pragma unroll
            for (int p = 0; p < kParts; ++p)
#pragma unroll
              for (int b = 0; b < NC; ++b)
                xv[p][b] = *reinterpret_cast<const uint4*>(
                    xb0 + p * kPlane + (b * 16 + r) * kColBytes + (slot_of(q, s) ^ r) * 16);
#pragma unroll
            for (int rt = 0; rt < kWide; ++rt) {
              if (XT == 2) {
                const _Float16 h = (_Float16)s2[rt][s / 2];
                const half8_t wa = decode8(w[d].c[rt][s], (half2_t){h, h});
#pragma unroll
                for (int b = 0; b < NC; ++b) {
                  half8_t xb;
                  __builtin_memcpy(&xb, &xv[0][b], 16);
                  acc[rt][b] = __builtin_amdgcn_mfma_f32_16x16x32_f16(wa, xb, acc[rt][b], 0, 0, 0);
                }
              } else {
                const bf16x8_t wa = decode8_bf16(w[d].c[rt][s], s2[rt][s / 2]);
#pragma unroll
                for (int p = 0; p < kParts; ++p)
#pragma unroll
                  for (int b = 0; b < NC; ++b) {
                    bf16x8_t xb;
                    __builtin_memcpy(&xb, &xv[p][b], 16);
                    acc[rt][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wa, xb, acc[rt][b], 0, 0, 0);
                  }
              }
            }
          }
        }
        w[d] = load_w(turn + kDepth);
        store_xs((d + 1) % kSets, 1 - buf);
        __syncthreads();
      }
    }
    // the other groups' sums join the first's (the buffers are free now)
    f32x4_t* red = reinterpret_cast<f32x4_t*>(lds);
    constexpr int kSums = kRowWaves * kWide * NC * kWave;
    static_assert((kGroups - 1) * kSums * 16 <= 2 * kBuffer, "the sums fit the buffers");
    if (kGroups > 1) {
      if (group > 0) {
#pragma unroll
        for (int rt = 0; rt < kWide; ++rt)
#pragma unroll
          for (int b = 0; b < NC; ++b)
            red[(group - 1) * kSums + ((wave * kWide + rt) * NC + b) * kWave + lane] = acc[rt][b];
      }
      __syncthreads();
      if (group > 0) continue;
    }
#pragma unroll
    for (int b = 0; b < NC; ++b) {
#pragma unroll
      for (int rt = 0; rt < kWide; ++rt) {
#pragma unroll
        for (int g = 1; g < kGroups; ++g)
          acc[rt][b] += red[(g - 1) * kSums + ((wave * kWide + rt) * NC + b) * kWave + lane];
        acc[rt][b] *= sg;
      }
      const int ci = c0 + b * 16 + r;
      if (ci >= m) continue;
      const int entry = EXPERT ? list[ci] : ci;
      if (SWIGLU) {
        if (row0 < rows) store_d4(a, entry, row0 + 4 * q, acc[0][b], acc[1][b], a.prob[entry]);
      } else {
#pragma unroll
        for (int rt = 0; rt < kWide; ++rt) store4(a, entry, row0 + rt * kTile + 4 * q, acc[rt][b]);
      }
    }
  }
}

namespace {

// Experts that can have entries.
int64_t experts_met(const MatvecArgs& a) {
  const int64_t entries = a.tokens * a.topk;
  return entries < a.num_groups ? entries : a.num_groups;
}

// Whether the kernel with x in LDS is the faster one.  It reads the weights at
// a higher rate and does not pay for more columns, but needs many workgroups.
// Measured (GPU time, bf16, tiled; direct kernel / LDS kernel), one matrix:
//   k 512: n 8192, 16 rows 4.5 / 5.2 us, 32 rows 5.4 / 5.3; n 16384, 4 rows 4.5 /
//   5.3, 16 rows 5.3 / 5.3; n 32768, 1 row 5.1 / 6.0, 16 rows 8.1 / 6.2;
//   k 2048: n 4096, 16 rows 5.8 / 7.5, 32 rows 7.8 / 7.6, 64 rows 11.8 / 8.0; n
//   8192, 4 rows 6.0 / 7.9, 16 rows 8.3 / 7.9, 64 rows 20.9 / 10.3; n 16384, 1 row
//   7.6 / 8.8, 4 rows 8.6 / 8.8, 16 rows 12.7 / 8.9;
//   k 8192: n 1024, 64 rows 12.2 / 17.3; n 4096, 16 rows 13.0 / 17.2, 32 rows
//   21.7 / 17.3; n 16384, 1 row 18.0 / 18.4; n 32768, 1 row 45.6 / 35.
// Experts, by 128-row blocks of the experts met and columns each (tiled bf16;
// direct / LDS kernel): k 1024: 32 blocks, 16 columns 7.3 / 8.9 us; 128 blocks,
// 4 columns 6.8 / 7.3, 8 columns 7.6 / 7.6, 16 columns 11.1 / 9.4; 256 blocks, 1
// column 8.3 / 9.5, 2 columns 9.3-10.2 / 9.6, 8 columns 12.3 / 9.7; 512 blocks, 1
// column 12.7 / 11.9, 16 columns 39.9 / 14.9; k 4096: 64 blocks, 8 columns 11.7 /
// 14.6; 128 blocks, 2 columns 14.0 / 15.4, 16 columns 29.3 / 19.2; 256 blocks, 1
// column 18.2 / 18.9, 2 columns 22.5 / 19.3; 1024 blocks, 1 column 71 / 51.
bool rows_kernel_pays(const MatvecArgs& a, bool expert) {
  if (!expert) {
    const int64_t t = a.tokens;
    const int64_t from = t <= 2 ? 32768 : (t <= 8 ? 16384 : (t <= 16 ? 8192 : 4096));
    return a.n >= (a.k < 1024 ? 2 * from : from);
  }
  const int64_t entries = a.tokens * a.topk, blocks = (a.n + 127) / 128;
  // (No more entries than experts: the direct kernel has a slot per entry, the
  // LDS kernel one per expert, most of them empty.  The layer's FC1 and FC2,
  // top-8 of 128, 2048 and 768: 4 tokens, 384 and 512 blocks, 33.5 / 42.7 us; 6
  // tokens 52.3 / 54.2; 8 tokens 64.2 / 58.6.)
  return entries <= a.num_groups ? blocks * entries >= 512
                                 : blocks * (a.num_groups + entries) >= 768;
}

// Workgroups that share an expert's columns: what its mean number of entries
// fills, and one (an expert with more has its workgroups take several turns).
// Against one workgroup for all columns: 128 tokens, top-4 of 16, hidden 1024,
// intermediate 512: 25 against 35 us; 256 tokens, top-2 of 8, 2048 and 768: 38
// against 65.
int64_t column_blocks(const MatvecArgs& a, int64_t cols) {
  return 1 + a.tokens * a.topk / (a.num_groups * cols);
}

int matvec_waves(int64_t k) {
  const int64_t stages = (k + kStage - 1) / kStage;
  // two stages a wave: one round of loads
  return (int)(stages < 2 ? 1 : (stages < 16 ? (stages + 1) / 2 : 8));
}

}  // namespace

template <int XT, int NC, int ROW_WAVES, int GROUPS, bool SWIGLU, bool EXPERT>
static void launch_rows(const MatvecArgs& a, hipStream_t s) {
  typedef RowsShape<XT, NC, ROW_WAVES, GROUPS> Shape;
  // behind the buffers: a word per wave and the list of an expert's entries
  const size_t list = EXPERT ? Shape::kThreads / kWave * 4 + (size_t)(a.tokens * a.topk) * 2 : 0;
  const int64_t per = ROW_WAVES * kTile * (SWIGLU ? 1 : kWide);
  const int64_t rows = SWIGLU ? a.inter : a.n, cols = NC * kTile;
  // the columns of an expert with more than `cols` go to several workgroups
  const dim3 grid((unsigned)((rows + per - 1) / per),
                  (unsigned)(EXPERT ? a.num_groups + 1 : (a.tokens + cols - 1) / cols),
                  (unsigned)(EXPERT ? column_blocks(a, cols) : 1));
  matvec_rows_kernel<XT, NC, ROW_WAVES, GROUPS, SWIGLU, EXPERT>
      <<<grid, Shape::kThreads, 2 * Shape::kBuffer + list, s>>>(a);
}

// One matrix, 64-row workgroups: four groups of waves share k while the
// workgroups are no more than the CUs and k is long enough, else two (binary32
// x with 32 columns: the LDS holds no more).
template <int XT, int NC>
static void launch_groups(const MatvecArgs& a, hipStream_t s) {
  constexpr int kMost = XT == 0 && NC > 1 ? 2 : 4;
  const int64_t cols = NC * kTile;
  const bool few = (a.n + 63) / 64 * ((a.tokens + cols - 1) / cols) <= 256;
  if (few && a.k >= 1024) launch_rows<XT, NC, 2, kMost, false, false>(a, s);
  else launch_rows<XT, NC, 2, 2, false, false>(a, s);
}

template <int XT, bool SWIGLU, bool EXPERT>
static void launch_matvec_one(const MatvecArgs& a, hipStream_t s) {
  const int64_t entries = a.tokens * a.topk;
  const int64_t xrows = EXPERT && a.x_by_entry ? entries : a.tokens;
  const int64_t xbytes = ((xrows - 1) * a.ld_x + a.k) * (XT == 0 ? 4 : 2) + 2 * (a.x_plane * 2);
  if (a.k >= 32 && xbytes < kNone && rows_kernel_pays(a, EXPERT)) {
    if constexpr (EXPERT) {
      const auto workgroups = [&](int64_t per, int64_t cols) {
        return experts_met(a) * ((a.n + per - 1) / per) * column_blocks(a, cols);
      };
      // the entries of an expert scatter about their mean: room for twice as many.
      // D's planes take less room and time with 16 columns, which costs more where
      // the experts with more of them, whose weights are read twice, are many
      // (FC2 in three parts, whole layer, 16 / 32 columns: hidden 1024, intermediate
      // 512, top-4 of 16: 96 tokens 27.5 / 30.2 us, 256 tokens 33.0 / 34.1; 2048 and
      // 768: top-2 of 8, 256 tokens 39.4 / 41.4; top-8 of 64, 128 tokens, 2048
      // workgroups, 71.9 / 66.8)
      const bool one = 2 * entries <= 16 * a.num_groups ||
                       (XT == kPlanes && workgroups(128, 16) <= 1024);
      // 64-row workgroups whose groups share k while those are at most two a CU,
      // or one where the LDS holds no second (three parts of 32 columns: 128 tokens,
      // top-4 of 16 experts of [1024, 1024], binary32, 512 of them 24.3 us, half as
      // many 128-row workgroups 17.0)
      const int64_t most = !one && parts_of(XT) == 3 ? 256 : 512;
      const bool few = workgroups(64, one ? 16 : 32) <= most;
      static_assert(parts_of(XT) != 3 || 4 * RowsShape<XT, 2, 2, 2>::kBuffer > 160 * 1024, "see `most`");
      if (one && few) return launch_rows<XT, 1, 2, 2, SWIGLU, true>(a, s);
      if (one) return launch_rows<XT, 1, 4, 1, SWIGLU, true>(a, s);
      if (few) return launch_rows<XT, 2, 2, 2, SWIGLU, true>(a, s);
      // 32 columns of D's planes leave the LDS room for three workgroups a CU: eight
      // waves that share them instead of four where two of those fill every CU
      // (whole layer, 8 / 4 waves: 256 tokens, top-8 of 128, 2048 and 768, 1024
      // workgroups, 111 / 116 us; 512 tokens 186 / 209; 128 tokens, top-8 of 32, 512
      // workgroups, 58.3 / 61.8; 200 tokens, top-4 of 60, 1040 and 400, 300
      // workgroups, 39.4 / 38.0)
      if constexpr (XT == kPlanes) {
        if (workgroups(256, 32) >= 512) return launch_rows<XT, 2, 8, 1, SWIGLU, true>(a, s);
      }
      return launch_rows<XT, 2, 4, 1, SWIGLU, true>(a, s);
    } else {
      // as many columns a workgroup as leave one for every CU
      const auto fills = [&](int64_t cols) {
        return (a.n + 63) / 64 * ((a.tokens + cols - 1) / cols) >= 256;
      };
      if (XT != 0 && a.tokens > 32 && a.n >= 128 * 256) launch_rows<XT, XT == 0 ? 2 : 4, 4, 2, false, false>(a, s);
      else if (XT != 0 && a.tokens > 32 && fills(64)) launch_groups<XT, XT == 0 ? 2 : 4>(a, s);
      else if (a.tokens > 16 && fills(32)) launch_groups<XT, 2>(a, s);
      else launch_groups<XT, 1>(a, s);
    }
    return;
  }
  const int waves = matvec_waves(a.k);
  const int64_t tiles = SWIGLU ? a.inter / kTile : (a.n + kTile - 1) / kTile;
  const int64_t slots = !EXPERT ? (a.tokens + kTile - 1) / kTile
                                : (entries <= a.num_groups ? entries : a.num_groups + 1);
  matvec_kernel<XT, SWIGLU, EXPERT>
      <<<dim3((unsigned)tiles, (unsigned)slots), waves * kWave,
         (size_t)waves * (SWIGLU ? 2 : 1) * kWave * sizeof(f32x4_t), s>>>(a);
}

hipError_t launch_matvec(const MatvecArgs& a, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
  const bool swiglu = a.d != nullptr, expert = a.topk_idx != nullptr;
  const int xt = a.x_plane ? kPlanes : a.x_dtype;
  switch (xt * 4 + (swiglu ? 2 : 0) + (expert ? 1 : 0)) {
    case 0: launch_matvec_one<0, false, false>(a, s); break;
    case 1: launch_matvec_one<0, false, true>(a, s); break;
    case 3: launch_matvec_one<0, true, true>(a, s); break;
    case 4: launch_matvec_one<1, false, false>(a, s); break;
    case 5: launch_matvec_one<1, false, true>(a, s); break;
    case 7: launch_matvec_one<1, true, true>(a, s); break;
    case 8: launch_matvec_one<2, false, false>(a, s); break;
    case 9: launch_matvec_one<2, false, true>(a, s); break;
    case 11: launch_matvec_one<2, true, true>(a, s); break;
    default: launch_matvec_one<kPlanes, false, true>(a, s); break;
  }
  return hipGetLastError();
}

// It reads an expert's weights for every entry, so beyond four tokens it needs
// entries that seldom share one.  Measured (the whole layer, separate / fused sum,
// hidden 2048, intermediate 768 but where said): top-8 of 128: 5 tokens 48.2 / 41.2
// us, 8 tokens 61.4 / 58.9, 12 tokens 66.2 / 70.9; top-4 of 32: 5 tokens 27.1 / 25.2,
// 8 tokens 30.4 / 31.0, 12 tokens 32.2 / 38.5; top-4 of 16, 1024 and 512: 8 tokens
// 15.4 / 12.7, 12 tokens 15.8 / 15.3; top-2 of 8: 8 tokens 17.4 / 16.9, 12 tokens
// 18.4 / 20.1; top-8 of 16 (2.5 entries an expert): 5 tokens 26.7 / 27.6, 8 tokens
// 28.2 / 33.7.
bool decode_down_fits(int64_t tokens, int32_t topk, int32_t num_experts) {
  return tokens <= 4 || (tokens <= 8 && tokens * topk <= 2 * (int64_t)num_experts);
}

hipError_t launch_decode_down(const MatvecArgs& a, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
  const int64_t stages = (a.k + kStage - 1) / kStage;
  const int sets = a.topk < 16 ? a.topk : 16;
  int parts = 16 / sets;
  if (parts > (stages + 1) / 2) parts = (int)((stages + 1) / 2);
  const int waves = sets * parts;
  const dim3 grid((unsigned)((a.n + kTile - 1) / kTile), (unsigned)a.tokens);
  const size_t lds = (size_t)a.topk * (parts * 4 * sizeof(f32x4_t) + 4);
  decode_down_kernel<<<grid, waves * kWave, lds, s>>>(a, parts);
  return hipGetLastError();
}

// y[t] = sum over the routed entries (t, j), j ascending, of y_rows[t*k + j].
template <int DT>
__global__ __launch_bounds__(256) void decode_combine_kernel(const float* y_rows, const int32_t* idx,
                                                             int32_t topk, int32_t num_experts,
                                                             int64_t hidden, void* y) {
  const int64_t t = blockIdx.y;
  const int64_t c = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 4;
  if (c >= hidden) return;
  f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < topk; ++j) {
    const int e = idx[t * topk + j];
    if (e < 0 || e >= num_experts) continue;
    f32x4_t v;
    __builtin_memcpy(&v, y_rows + (t * topk + j) * hidden + c, 16);
    sum += v;
  }
  typename Elem<DT>::type o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = Elem<DT>::from_float(sum[i]);
  __builtin_memcpy(static_cast<typename Elem<DT>::type*>(y) + t * hidden + c, o, sizeof(o));
}

hipError_t launch_decode_combine(const float* y_rows, const int32_t* idx, int64_t tokens,
                                 int32_t topk, int32_t num_experts, int64_t hidden, int y_dtype,
                                 void* y, hipStream_t s) {
  if (tokens == 0) return hipSuccess;
  const int threads = hidden >= 1024 ? 256 : 64;
  const dim3 grid((unsigned)((hidden / 4 + threads - 1) / threads), (unsigned)tokens);
  if (y_dtype == 0)
    decode_combine_kernel<0><<<grid, threads, 0, s>>>(y_rows, idx, topk, num_experts, hidden, y);
  else if (y_dtype == 1)
    decode_combine_kernel<1><<<grid, threads, 0, s>>>(y_rows, idx, topk, num_experts, hidden, y);
  else
    decode_combine_kernel<2><<<grid, threads, 0, s>>>(y_rows, idx, topk, num_experts, hidden, y);
  return hipGetLastError();
}

}  // namespace nvfp4
