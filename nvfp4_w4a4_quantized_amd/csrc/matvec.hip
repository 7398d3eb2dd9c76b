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
// products.  The layer's intermediate D is kept as the sum of two bf16 parts,
// high = bf16(D) and low = bf16(D - high), within 2^-17 of the binary32 D, so
// FC2 adds no rounding that shows in a 16-bit result.
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
#include "elem.h"
#include "gemm_common.h"
#include "launch.h"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// How x travels: 0 binary32, 1 bf16, 2 fp16, 3 two bf16 parts (the layer's D)
constexpr int kPair = 3;
constexpr int parts_of(int xt) { return xt == 0 ? 3 : (xt == kPair ? 2 : 1); }
constexpr int kStage = 128;   // k elements of a stage
constexpr int kTile = 16;     // weight rows of a tile, columns of a product

// 32 elements of a column: one stage of a lane.
template <int XT>
struct XStage {
  uint4 w[XT == 0 || XT == kPair ? 8 : 4];
};

template <int XT>
__device__ __forceinline__ XStage<XT> load_x(const char* p, const char* p_lo) {
  XStage<XT> x;
  __builtin_memcpy(&x.w[0], p, XT == 0 ? 128 : 64);
  if (XT == kPair) __builtin_memcpy(&x.w[4 % (sizeof(x.w) / 16)], p_lo, 64);
  return x;
}

// Part `part` of elements [8s, 8s + 8) of the stage as an operand.
template <int XT>
__device__ __forceinline__ uint4 x_operand(const XStage<XT>& x, int s, int part) {
  if (XT == kPair) return x.w[(part * 4 + s) % (sizeof(x.w) / 16)];
  if (XT != 0) return x.w[s];
  // upper halves of the value, of what is left of it, and of the rest
  const uint4 a = x.w[(2 * s) % (sizeof(x.w) / 16)], b = x.w[(2 * s + 1) % (sizeof(x.w) / 16)];
  uint32_t f[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
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

// One stage of one 16-row tile: c = the lane's 32 codes, sb = its two E4M3
// bytes (the second block's in bits 8-15).
template <int XT>
__device__ __forceinline__ void stage_product(f32x4_t& acc, const uint4& c, uint32_t sb,
                                              const XStage<XT>& x) {
  const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
  const half2_t s2 = e4m3x2_to_half2(sb);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if (XT == 2) {
      const _Float16 h = s2[s / 2];
      const half8_t a = decode8(cw[s], (half2_t){h, h});
      const uint4 xo = x_operand<XT>(x, s, 0);
      half8_t b;
      __builtin_memcpy(&b, &xo, 16);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, acc, 0, 0, 0);
    } else {
      const bf16x8_t a = decode8_bf16(cw[s], (float)s2[s / 2]);
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

// Stores the values of rows [row, row + 4) of one column (those below n).
__device__ __forceinline__ void store4(const MatvecArgs& a, int64_t out_row, int64_t row, f32x4_t v) {
  const int64_t at = out_row * a.n + row;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (row + i >= a.n) continue;
    if (a.out_dtype == 0) static_cast<float*>(a.out)[at + i] = v[i];
    else if (a.out_dtype == 1) static_cast<uint16_t*>(a.out)[at + i] = Elem<1>::from_float(v[i]);
    else static_cast<_Float16*>(a.out)[at + i] = (_Float16)v[i];
  }
}

// The layer's D of one entry: silu(g) u p, as its two bf16 parts.
__device__ __forceinline__ void store_d4(const MatvecArgs& a, int64_t entry, int64_t col, f32x4_t g,
                                         f32x4_t u, float p) {
  uint16_t hi[4], lo[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float d = g[i] / (1.0f + expf(-g[i])) * u[i] * p;
    hi[i] = Elem<1>::from_float(d);
    const float h = Elem<1>::to_float(hi[i]);
    // an infinite D keeps a zero low part (inf - inf would be NaN)
    lo[i] = Elem<1>::from_float(fabsf(h) < __builtin_huge_valf() ? d - h : 0.0f);
  }
  __builtin_memcpy(a.d_hi + entry * a.inter + col, hi, 8);
  __builtin_memcpy(a.d_lo + entry * a.inter + col, lo, 8);
}

}  // namespace

// Grid: x = 16-row tiles of the output, y = slots (EXPERT) or chunks of 16
// columns.  A slot is an entry when there are no more entries than experts
// (the first entry of an expert does the work of all of its entries), else an
// expert, with one more slot for the entries of no expert.
template <int XT, bool SWIGLU, bool EXPERT>
__global__ __launch_bounds__(512) void matvec_kernel(MatvecArgs a) {
  constexpr int RT = SWIGLU ? 2 : 1;
  extern __shared__ char lds[];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int waves = blockDim.x / kWave;
  const int r = lane % kTile, q = lane / kTile;
  const int64_t row0 = (int64_t)blockIdx.x * kTile;
  f32x4_t* red = reinterpret_cast<f32x4_t*>(lds);
  uint16_t* list = reinterpret_cast<uint16_t*>(lds + waves * RT * kWave * sizeof(f32x4_t));
  __shared__ int found;
  int e = 0, m = (int)a.tokens, first = 0;
  if (EXPERT) {
    const int entries = (int)a.tokens * a.topk;
    const bool by_entry = entries <= a.num_groups;
    const int slot = blockIdx.y;
    e = by_entry ? a.topk_idx[slot] : slot;
    if (e < 0 || e >= a.num_groups) {
      if (SWIGLU) return;
      // entries of no expert: zero results
      for (int i = by_entry ? slot : 0; i < (by_entry ? slot + 1 : entries); ++i) {
        const int id = a.topk_idx[i];
        if ((id < 0 || id >= a.num_groups) && threadIdx.x < 4)
          store4(a, i, row0 + 4 * threadIdx.x, (f32x4_t){0.f, 0.f, 0.f, 0.f});
      }
      return;
    }
    if (threadIdx.x == 0) found = 0;
    __syncthreads();
    bool earlier = false;
    for (int i = threadIdx.x; i < entries; i += blockDim.x) {
      if (a.topk_idx[i] == e) {
        earlier = earlier || (by_entry && i < slot);
        // (a column's place does not change its result, so any order will do)
        list[atomicAdd(&found, 1)] = (uint16_t)i;
      }
    }
    if (__syncthreads_or(earlier)) return;
    m = found;
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
  const int64_t cstep = a.layout == 0 ? kStage / 2 : 2048, sstep = a.layout == 0 ? kStage / 16 : 256;
  const int stages = (int)(a.k / kStage);
  const int xsize = XT == 0 ? 4 : 2;
  const float sg = a.gscale[e];
  for (int c0 = first; c0 < m; c0 += kTile) {
    // columns past the last repeat it (and are not stored)
    const int ci = c0 + r < m ? c0 + r : m - 1;
    const int entry = EXPERT ? list[ci] : ci;
    const int64_t xrow = EXPERT && !a.x_by_entry ? entry / a.topk : entry;
    const char* xp = static_cast<const char*>(a.x) + (xrow * a.ld_x + 32 * q) * xsize;
    const char* xl = XT == kPair ? reinterpret_cast<const char*>(a.x_lo) + (xrow * a.ld_x + 32 * q) * 2
                                 : nullptr;
    f32x4_t acc[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) acc[rt] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
    for (int st = wave; st < stages; st += waves) {
      const XStage<XT> x = load_x<XT>(xp + (int64_t)st * kStage * xsize, XT == kPair ? xl + st * kStage * 2 : nullptr);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        stage_product<XT>(acc[rt], load_u128(place[rt].codes + st * cstep),
                          load_u16(place[rt].scales + st * sstep), x);
    }
    // the k behind the last whole stage (row-major weights only): a multiple
    // of 16, so a lane has none, half or all of its 32
    const int left = (int)(a.k - (int64_t)stages * kStage) - 32 * q;
    if (a.k % kStage != 0 && wave == stages % waves) {
      XStage<XT> x = {};
      uint4 c[RT] = {};
      uint32_t sb[RT] = {};
      const int64_t xo = (int64_t)stages * kStage * xsize;
      if (left >= 16) {
        const int bytes = left >= 32 ? 32 : 16;
        if (bytes == 32) {
          x = load_x<XT>(xp + xo, XT == kPair ? xl + stages * kStage * 2 : nullptr);
        } else {
          __builtin_memcpy(&x.w[0], xp + xo, 16 * xsize);
          if (XT == kPair) __builtin_memcpy(&x.w[4 % (sizeof(x.w) / 16)], xl + stages * kStage * 2, 32);
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const uint8_t* pc = place[rt].codes + stages * cstep;
          const uint8_t* ps = place[rt].scales + stages * sstep;
          if (bytes == 32) {
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
        if (SWIGLU) store_d4(a, entry, row0 + 4 * q, acc[0], acc[RT - 1], a.prob[entry]);
        else store4(a, entry, row0 + 4 * q, acc[0]);
      }
    }
  }
}

namespace {

int matvec_waves(int64_t k) {
  const int64_t stages = (k + kStage - 1) / kStage;
  return (int)(stages < 8 ? stages : 8);
}

}  // namespace

hipError_t launch_matvec(const MatvecArgs& a, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
  const bool swiglu = a.d_hi != nullptr, expert = a.topk_idx != nullptr;
  const int waves = matvec_waves(a.k);
  const int64_t entries = a.tokens * a.topk;
  const int64_t tiles = swiglu ? a.inter / kTile : (a.n + kTile - 1) / kTile;
  const int64_t slots = !expert ? (a.tokens + kTile - 1) / kTile
                                : (entries <= a.num_groups ? entries : a.num_groups + 1);
  const size_t lds = (size_t)waves * (swiglu ? 2 : 1) * kWave * sizeof(f32x4_t) +
                     (expert ? (size_t)entries * 2 : 0);
  const dim3 grid((unsigned)tiles, (unsigned)slots);
#define NVFP4_MATVEC(XT, SW, EX) \
  matvec_kernel<XT, SW, EX><<<grid, waves * kWave, lds, s>>>(a)
  if (swiglu) {
    if (a.x_dtype == 0) NVFP4_MATVEC(0, true, true);
    else if (a.x_dtype == 1) NVFP4_MATVEC(1, true, true);
    else NVFP4_MATVEC(2, true, true);
  } else if (expert) {
    if (a.x_lo) NVFP4_MATVEC(kPair, false, true);
    else if (a.x_dtype == 0) NVFP4_MATVEC(0, false, true);
    else if (a.x_dtype == 1) NVFP4_MATVEC(1, false, true);
    else NVFP4_MATVEC(2, false, true);
  } else {
    if (a.x_dtype == 0) NVFP4_MATVEC(0, false, false);
    else if (a.x_dtype == 1) NVFP4_MATVEC(1, false, false);
    else NVFP4_MATVEC(2, false, false);
  }
#undef NVFP4_MATVEC
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
