// newton_schulz.hip -- the orthogonalised update of a weight's gradient:
//   X0 = G / (|G|_F + eps),   X <- a X + P X,   P = b A + c A A,   A = X X^T
// for wide G (rows <= cols), and from the other side, A = X^T X, X <- a X + X P,
// for tall G, so that nothing is transposed and A is as small as it can be.
//
// Arithmetic.  X is kept as two binary16 parts (hi, and lo the rest: 22 bits)
// times a power of two that brings its largest possible element near the top of
// the range.  The products run on the matrix cores in binary16 with binary32 sums:
//   - 16-bit "fast" products, of bf16 results in as many of the last steps as the
//     coefficients let them (ns_bounds), take hi alone, of X and of P + a I, and a lo is added
//     to them: the small singular values, which the iteration multiplies by a per
//     step, keep X's 22 bits.  (Taking a hi from memory instead of the products
//     reads X once more: an update of 128 matrices of 2048 x 768 takes 524 us
//     instead of 502.)  Against binary64 the result of 768 x 2048 gradients is
//     1e-3 off (bf16's own rounding: 1.7e-3; X in 11 bits: 3e-3 to 5e-2; bf16
//     products: 2e-2).
//   - "exact" products take hi hi + hi lo + lo hi, and a X from both parts: 1.9e-6
//     off (four 1000 x 2047), binary32 throughout 3.2e-6.
// A gradient far below eps keeps its digits: X is multiplied by a further 2^k0,
// k0 = floor(-log2 |X0|), which shrinks by the iteration's growth every step.
//
// One GEMM kernel computes all three products; a symmetric result is computed
// in its upper tiles and mirrored.  Operands lie K-contiguous (X of the wide
// Gram product, A, P, X of the tall update) or K-major (X of the tall Gram
// product and of the wide update) and go from memory straight into an LDS
// ring of two to four slots; K-major tiles are read with the transposing LDS loads.
//
// Bound, for many matrices: 128 of 2048 x 768 (1.6 TFLOP) take 4.5 ms.  A and P run
// at 0.8 and 0.5 PFLOP/s counted without the mirrored half (matrix cores 51 % busy
// at the 1.9 GHz that the clock falls to), the update of X is memory bound (2.3 GB a
// step past the second-level cache, 4.4 TB/s).  Overlapping LDS reads with products
// by half stages changed them by 1 to 4 %.  One matrix leaves CUs idle: 5120 x 2048
// has 136 tiles of A for 256 CUs.
#include <type_traits>

#include "elem.h"
#include "gemm_common.h"
#include "launch.h"

namespace nvfp4 {

namespace {

typedef short short4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) short4_t lds_short4_t;

enum { kGram = 0, kPoly = 1, kApply = 2, kLast = 3 };

// ---- the norm and the first X ------------------------------------------------

// Partial sums of squares in binary64, grid: (parts, matrices).
template <int DT>
__global__ __launch_bounds__(256) void ns_norm_kernel(NsSource g, double* part) {
  typedef typename Elem<DT>::type T;
  __shared__ double red[4];
  const T* p = static_cast<const T*>(g.g) + (int64_t)blockIdx.y * g.ld_batch;
  double sum = 0.0;
  for (int64_t r = blockIdx.x; r < g.rows; r += gridDim.x) {
    const T* row = p + r * g.ld_row;
    for (int64_t c = (int64_t)threadIdx.x * Piece<DT>::kN; c < g.cols; c += 256 * Piece<DT>::kN) {
      Piece<DT> v;
      if (c + Piece<DT>::kN <= g.cols) v.load(row + c);
      else v.load_part(row + c, (int)(g.cols - c));
#pragma unroll
      for (int i = 0; i < Piece<DT>::kN; ++i) {
        const double d = v.get(i);
        sum += d * d;
      }
    }
  }
  for (int d = 32; d > 0; d /= 2) sum += __shfl_xor(sum, d);
  if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = sum;
  __syncthreads();
  if (threadIdx.x == 0) part[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = red[0] + red[1] + red[2] + red[3];
}

// hi and lo of X0 2^k0 scale, zeros in the columns up to ld.  Grid: (rows of
// four, matrices).
template <int DT>
__global__ __launch_bounds__(256) void ns_start_kernel(NsSource g, const double* part, int parts,
                                                       double eps, double scale, int64_t ld,
                                                       _Float16* hi, _Float16* lo, int32_t* k0_out) {
  typedef typename Elem<DT>::type T;
  const int64_t e = blockIdx.y;
  const int lane = threadIdx.x % kWave;
  double sum = 0.0;
  for (int i = lane; i < parts; i += kWave) sum += part[e * parts + i];
  for (int d = 32; d > 0; d /= 2) sum += __shfl_xor(sum, d);
  const double norm = sqrt(sum), below = norm + eps;
  // (a zero matrix stays zero whatever eps is; a norm that is no number gives NaN)
  int k0 = 0;
  if (norm > 0.0 && norm < below) k0 = -ilogb(norm / below) - 1;
  k0 = k0 < 0 ? 0 : k0;
  const double f = norm == 0.0 ? 0.0 : ldexp(scale, k0) / below;
  if (blockIdx.x == 0 && threadIdx.x == 0) k0_out[e] = k0;
  const int64_t r = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave;
  if (r >= g.rows) return;
  const T* row = static_cast<const T*>(g.g) + e * g.ld_batch + r * g.ld_row;
  const int64_t at = (e * g.rows + r) * ld;
  auto put = [&](int64_t c, const float (&x)[8]) {
    half8_t h, l;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double v = f * (double)x[i];
      h[i] = (_Float16)(float)v;
      l[i] = (_Float16)(float)(v - (double)h[i]);
    }
    *reinterpret_cast<half8_t*>(hi + at + c) = h;
    *reinterpret_cast<half8_t*>(lo + at + c) = l;
  };
  int64_t c = (int64_t)lane * 8;
  for (; c + 8 <= g.cols; c += kWave * 8) {
    T v[8];
    __builtin_memcpy(v, row + c, sizeof(v));
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = Elem<DT>::to_float(v[i]);
    put(c, x);
  }
  for (; c < ld; c += kWave * 8) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = c + i < g.cols ? Elem<DT>::to_float(row[c + i]) : 0.0f;
    put(c, x);
  }
}

// ---- the products --------------------------------------------------------------

// LDS tiles are unpadded and XOR-swizzled in 16-byte chunks (a direct-to-LDS
// load writes one contiguous KiB per wave instruction):
//   K-contiguous [T rows][BK k]: chunk c of row r at c ^ r % 8 (BK = 64), or
//     c ^ (r / 4) % 4 (BK = 32)
//   K-major [BK k][T columns]: chunk c of row r at c ^ 4 (r % 4)
__device__ __forceinline__ int swz_major(int r, int c) { return c ^ (4 * (r & 3)); }
template <int BK>
__device__ __forceinline__ int swz_row(int r, int c) {
  return BK == 64 ? c ^ (r & 7) : c ^ ((r >> 2) & 3);
}

// The matrix-core operand: lane l has row (column) r0 + l % 32 of the tile and
// k = k0 + 8 (l / 32) + 0..7.
template <int T, int BK, bool MAJOR>
__device__ __forceinline__ half8_t fragment(const _Float16* s, int r0, int k0, int lane) {
  if constexpr (MAJOR) {
    const int r = k0 + (lane >> 5) * 8 + ((lane & 15) >> 2);
    const int col = r0 + ((lane >> 4) & 1) * 16 + 4 * (lane & 3);
    const int off = 8 * swz_major(r, col >> 3) + (col & 7);      // rows r and r + 4 share it
    const short4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4_t*)(s + r * T + off));
    const short4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4_t*)(s + (r + 4) * T + off));
    const auto both = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    half8_t v;
    __builtin_memcpy(&v, &both, 16);
    return v;
  } else {
    const int r = r0 + (lane & 31), c = (k0 >> 3) + (lane >> 5);
    return *reinterpret_cast<const half8_t*>(s + r * BK + 8 * swz_row<BK>(r, c));
  }
}

__device__ __forceinline__ void split(const float (&v)[8], half8_t* hi, half8_t* lo) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const _Float16 h = (_Float16)v[i];
    (*hi)[i] = h;
    (*lo)[i] = (_Float16)(v[i] - (float)h);
  }
}

// Eight consecutive results of the last step, `count` of them inside.
template <int OT>
__device__ __forceinline__ void put8(void* out, int64_t at, int64_t count, const float (&v)[8]) {
  typename Elem<OT>::type o[8], *p = static_cast<typename Elem<OT>::type*>(out) + at;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = Elem<OT>::from_float(v[i]);
  if (count >= 8) {
    __builtin_memcpy(p, o, sizeof(o));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < count) p[i] = o[i];
  }
}

// A workgroup's TM x TN tile: 2 x TN / 64 waves that take every stage of 32 k (KG =
// 1), or two such groups that take half of each stage of 64 and add their sums in LDS.
template <int TM_, int TN_, int KG_, int RING_>
struct Tile {
  static constexpr int TM = TM_, TN = TN_, KG = KG_, RING = RING_, BK = 32 * KG_, NW = TN_ / 32 * KG_;
};
using Huge = Tile<256, 256, 1, 4>;     // 128 KiB of LDS, eight waves
using Wide = Tile<256, 128, 1, 3>;     // 72 KiB: two workgroups of four waves a CU
using Deep = Tile<128, 128, 2, 4>;     // 128 KiB, eight waves

// C = A B over k with the epilogue EPI; AM, BMAJ: the operand is K-major;
// EXACT: products of both parts, and A and P have two.
template <typename S, bool AM, bool BMAJ, int EPI, bool EXACT>
__global__ __launch_bounds__(64 * S::NW, 2) void ns_gemm_kernel(NsGemmArgs p) {
  constexpr int TM = S::TM, TN = S::TN, KG = S::KG, NW = S::NW;
  // exact stages hold both parts of 32 k
  constexpr int PARTS = EXACT ? 2 : 1, BK = EXACT ? 32 : S::BK, RING = EXACT && TM == 256 ? 2 : S::RING;
  constexpr int IB = TM / 64, JB = 2, WN = TN / 64;       // a wave's blocks of 32 x 32; waves along N
  constexpr int A_BYTES = TM * BK * 2, B_BYTES = TN * BK * 2;
  constexpr int QA = A_BYTES / 1024 / NW, QB = B_BYTES / 1024 / NW;   // load instructions per wave
  // one array per slot, so that the compiler sees that a load into one slot
  // does not write the slot being read
  constexpr int SLOT = PARTS * (A_BYTES + B_BYTES);
  __shared__ __align__(16) uint8_t S0[SLOT];
  __shared__ __align__(16) uint8_t S1[SLOT];
  __shared__ __align__(16) uint8_t S2[RING >= 3 ? SLOT : 16];
  __shared__ __align__(16) uint8_t S3[RING == 4 ? SLOT : 16];
  constexpr bool SYM = EPI == kGram || EPI == kPoly;
  const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);

  // consecutive tiles of a matrix on one XCD (workgroups go round the eight)
  const int nb = gridDim.x, xcd = blockIdx.x % 8, in = blockIdx.x / 8;
  const int t = xcd * (nb / 8) + (xcd < nb % 8 ? xcd : nb % 8) + in;
  const int tiles_n = (int)((p.n + TN - 1) / TN);
  const int e32 = t / p.tiles;
  const int64_t e = e32;
  int ti = 0, tj = t - e32 * p.tiles;
  if (SYM) {
    // row ti has the column tiles from the one that holds its first diagonal
    // element on
    for (; tj >= tiles_n - ti * (TM / TN); ++ti) tj -= tiles_n - ti * (TM / TN);
    tj += ti * (TM / TN);
  } else {
    ti = tj / tiles_n;
    tj %= tiles_n;
  }
  const bool mirror = SYM && tj >= (ti + 1) * (TM / TN);      // wholly above the diagonal
  const int64_t m0 = (int64_t)ti * TM, n0 = (int64_t)tj * TN;

  const __amdgpu_buffer_rsrc_t ahi = buffer_rsrc(p.a.hi + e * p.a.stride, p.a.bytes);
  const __amdgpu_buffer_rsrc_t bhi = buffer_rsrc(p.b.hi + e * p.b.stride, p.b.bytes);
  const __amdgpu_buffer_rsrc_t alo = buffer_rsrc(p.a.lo + e * p.a.stride, p.a.bytes);
  const __amdgpu_buffer_rsrc_t blo = buffer_rsrc(p.b.lo + e * p.b.stride, p.b.bytes);
  const int nst = (int)((p.k + BK - 1) / BK);

  // A lane's offsets of stage 0.  Rows past the matrix lie past its resource
  // and read zeros; columns past ld are masked.
  auto place = [&](auto major, auto tile, int64_t first, int64_t ld, int q) -> uint32_t {
    const int i = wave + NW * q;
    if constexpr (decltype(major)::value) {
      constexpr int kLanes = decltype(tile)::value / 8, kRows = kWave / kLanes;   // lanes of a row, rows of an instruction
      const int r = i * kRows + lane / kLanes, c = swz_major(r, lane % kLanes);
      const int64_t col = first + 8 * c;
      return col < ld ? (uint32_t)((r * ld + col) * 2) : kNone;
    } else {
      constexpr int kLanes = BK / 8, kRows = kWave / kLanes;
      const int r = kRows * i + lane / kLanes, c = swz_row<BK>(r, lane % kLanes);
      return (uint32_t)(((first + r) * ld + 8 * c) * 2);
    }
  };
  using TMc = std::integral_constant<int, TM>;
  using TNc = std::integral_constant<int, TN>;
  uint32_t ao[QA], bo[QB];
#pragma unroll
  for (int q = 0; q < QA; ++q) ao[q] = place(std::bool_constant<AM>{}, TMc{}, m0, p.a.ld, q);
#pragma unroll
  for (int q = 0; q < QB; ++q) bo[q] = place(std::bool_constant<BMAJ>{}, TNc{}, n0, p.b.ld, q);
  const uint32_t astep = AM ? (uint32_t)(p.a.ld * BK * 2) : BK * 2;
  const uint32_t bstep = BMAJ ? (uint32_t)(p.b.ld * BK * 2) : BK * 2;

  auto slot = [&](auto u) -> uint8_t* {
    constexpr int U = decltype(u)::value;
    if constexpr (U == 0) return S0;
    else if constexpr (U == 1) return S1;
    else if constexpr (U == 2) return S2;
    else return S3;
  };
  // stage st of both operands (and both parts); stages past the last read zeros
  uint32_t sa = 0, sb = 0;
  auto load = [&](auto u, int st) {
    const bool live = st < nst;
#pragma unroll
    for (int part = 0; part < PARTS; ++part) {
      uint8_t* s = slot(u) + part * (A_BYTES + B_BYTES);
#pragma unroll
      for (int q = 0; q < QA; ++q)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(part == 0 ? ahi : alo, (lds_void_t*)(s + (wave + NW * q) * 1024),
                                                 16, (int)(live ? ao[q] + sa : kNone), 0, 0, 0);
#pragma unroll
      for (int q = 0; q < QB; ++q)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(part == 0 ? bhi : blo,
                                                 (lds_void_t*)(s + A_BYTES + (wave + NW * q) * 1024), 16,
                                                 (int)(live ? bo[q] + sb : kNone), 0, 0, 0);
    }
    sa += astep;
    sb += bstep;
  };

  float16_t acc[IB][JB];
#pragma unroll
  for (int i = 0; i < IB; ++i)
#pragma unroll
    for (int j = 0; j < JB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  const int group = KG == 2 ? wave / 4 : 0;
  const int rm = (wave % 2) * (TM / 2), rn = (wave / 2 % WN) * 64;   // the wave's first row and column
  // The fragments of 16 k of a part.
  struct Half {
    half8_t a[IB], b[JB];
  };
  auto read = [&](auto u, int part, int k, Half& f) {
    const uint8_t* from = slot(u) + part * (A_BYTES + B_BYTES);
    const _Float16* la = reinterpret_cast<const _Float16*>(from);
    const _Float16* lb = reinterpret_cast<const _Float16*>(from + A_BYTES);
#pragma unroll
    for (int j = 0; j < JB; ++j) f.b[j] = fragment<TN, BK, BMAJ>(lb, rn + j * 32, k, lane);
#pragma unroll
    for (int i = 0; i < IB; ++i) f.a[i] = fragment<TM, BK, AM>(la, rm + i * 32, k, lane);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto multiply = [&](const half8_t (&a)[IB], const half8_t (&b)[JB]) {
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int i = 0; i < IB; ++i)
#pragma unroll
      for (int j = 0; j < JB; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(b[j], a[i], acc[i][j], 0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
  };

  // 16 k are multiplied while the next ones are read from LDS, and RING stages are
  // in LDS or on their way.  Before a stage's last products a wave waits for its own
  // loads of the next stage (leaving those of the later ones outstanding) and for its
  // LDS reads of this one, which the products may still be waiting for: behind the
  // barrier every wave's part of the next stage has landed, and this stage's slot is
  // free for the one RING further on.  Stages past the last are zeros.
  constexpr int LOADS = PARTS * (QA + QB), WAIT = (RING - 2) * LOADS, WAIT0 = (RING - 1) * LOADS;
  constexpr int WAIT_IMM = (WAIT & 15) | ((WAIT >> 4) << 14) | (7 << 4);       // vmcnt(WAIT) lgkmcnt(0)
  constexpr int WAIT0_IMM = (WAIT0 & 15) | ((WAIT0 >> 4) << 14) | (7 << 4);
  static_assert(WAIT0 < 64, "vmcnt range");
  using C0 = std::integral_constant<int, 0>;
  using C1 = std::integral_constant<int, 1>;
  using C2 = std::integral_constant<int, 2>;
  using C3 = std::integral_constant<int, 3>;
  constexpr int HALVES = BK / 16 / KG;            // a group's, of a stage
  const int kg = 16 * HALVES * group;             // its first k
  Half f0, f1, low;
  // the next stage's first fragments, behind the barrier
  auto change = [&](auto u, int st, Half& f) {
    using Next = std::integral_constant<int, (decltype(u)::value + 1) % RING>;
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_waitcnt(WAIT_IMM);
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    load(u, st + RING);
    read(Next{}, 0, kg, f);
  };
  auto turn = [&](auto u, int st) {
    if constexpr (!EXACT) {
      read(u, 0, kg + 16, f1);
      multiply(f0.a, f0.b);
      change(u, st, f0);
      multiply(f1.a, f1.b);
    } else if constexpr (HALVES == 2) {
      read(u, 1, kg, low);
      multiply(f0.a, f0.b);
      read(u, 0, kg + 16, f1);
      multiply(f0.a, low.b);
      multiply(low.a, f0.b);
      read(u, 1, kg + 16, low);
      multiply(f1.a, f1.b);
      change(u, st, f0);
      multiply(f1.a, low.b);
      multiply(low.a, f1.b);
    } else {                                      // (the ring is even: f0 and f1 in turn)
      Half& now = decltype(u)::value % 2 == 0 ? f0 : f1;
      read(u, 1, kg, low);
      multiply(now.a, now.b);
      change(u, st, decltype(u)::value % 2 == 0 ? f1 : f0);
      multiply(now.a, low.b);
      multiply(low.a, now.b);
    }
  };
  load(C0{}, 0);
  load(C1{}, 1);
  if constexpr (RING >= 3) load(C2{}, 2);
  if constexpr (RING == 4) load(C3{}, 3);
  __builtin_amdgcn_s_waitcnt(WAIT0_IMM);
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  read(C0{}, 0, kg, f0);
  int st = 0;
  for (; st + RING <= nst; st += RING) {
    turn(C0{}, st);
    turn(C1{}, st + 1);
    if constexpr (RING >= 3) turn(C2{}, st + 2);
    if constexpr (RING == 4) turn(C3{}, st + 3);
  }
  if (st < nst) turn(C0{}, st);
  if (RING >= 3 && st + 1 < nst) turn(C1{}, st + 1);
  if constexpr (RING == 4)
    if (st + 2 < nst) turn(C2{}, st + 2);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(7 << 4);      // no load into LDS outlives the loop, no read is left
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);

  // Two groups: each takes one of the wave's row blocks and the other's sums of it.
  if constexpr (KG == 2) {
    float* give = reinterpret_cast<float*>((wave / 4 == 0 ? S0 : S1) + (wave % 4) * 8192) + lane * 4;
    const float* take = reinterpret_cast<const float*>((wave / 4 == 0 ? S1 : S0) + (wave % 4) * 8192) + lane * 4;
#pragma unroll
    for (int j = 0; j < JB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float four[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) four[c] = group == 0 ? acc[1][j][4 * q + c] : acc[0][j][4 * q + c];
        __builtin_memcpy(give + (j * 4 + q) * 256, four, 16);
      }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < JB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float four[4];
        __builtin_memcpy(four, take + (j * 4 + q) * 256, 16);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          acc[0][j][4 * q + c] = (group == 0 ? acc[0][j][4 * q + c] : acc[1][j][4 * q + c]) + four[c];
      }
  }

  // ---- epilogue.  The operands are swapped in the products, so acc[i][j][4 q +
  // c] is row l % 32 and column 8 q + 4 (l / 32) + c of block (i, j).  32 rows x
  // 64 columns at a time go through the wave's own 8 KiB of the ring (16-byte
  // chunk c of row r at c ^ r % 16), so that memory is read and written in
  // 128-byte rows, and in 64-byte ones of the mirrored tile.
  float* const tile = reinterpret_cast<float*>(
      KG == 2 ? (wave / 4 == 0 ? S2 : S3) + (wave % 4) * 8192
              : WN == 4 ? (wave < 4 ? S0 : S1) + (wave % 4) * 8192 : (wave < 2 ? S0 : S1) + (wave % 2) * 8192);
  const int h = lane >> 5, l32 = lane & 31, lr = lane / 8, lc = lane % 8;
  const int k0 = p.k0[e], kj = k0 - p.drop > 0 ? k0 - p.drop : 0;
  const int kn = kj - p.growth > 0 ? kj - p.growth : 0;
  const float f = EPI == kGram ? ldexpf(p.f, -2 * kj) : p.f;
  const float up = EPI == kApply ? ldexpf(1.0f, kn - kj) : (EPI == kLast ? ldexpf(p.up, -kj) : 1.0f);
  // Eight values of Y from (row, col) on, and the eight results f acc + g Y there.
  constexpr bool kLow = EXACT || EPI == kApply || EPI == kLast;    // Y's lower part is taken,
  constexpr bool kHigh = EXACT || EPI == kPoly;                    // and its upper one
  struct Given {
    half8_t hi, lo;
  };
  auto given = [&](int64_t row, int64_t col) -> Given {
    Given y;
    const int64_t at = e * p.y.stride + row * p.y.ld + col;
    if constexpr (kHigh) y.hi = *reinterpret_cast<const half8_t*>(p.y.hi + at);
    if constexpr (kLow) y.lo = *reinterpret_cast<const half8_t*>(p.y.lo + at);
    return y;
  };
  auto finish = [&](int64_t row, int64_t col, const Given& y, float (&v)[8]) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      v[c] *= f;
      if constexpr (EPI != kGram) {
        if constexpr (kLow) v[c] = fmaf(p.g, (float)y.lo[c], v[c]);
        if constexpr (kHigh) v[c] += p.g * (float)y.hi[c];
        if constexpr (EPI == kPoly && !EXACT) v[c] += row == col + c ? p.up : 0.0f;
        v[c] *= up;
      }
    }
    if constexpr (EPI == kLast) {
      const int64_t at = (e * p.m + row) * p.n + col, count = p.n - col;
      if (p.out_dtype == 0) put8<0>(p.out, at, count, v);
      else if (p.out_dtype == 1) put8<1>(p.out, at, count, v);
      else put8<2>(p.out, at, count, v);
    } else {
      half8_t hi, lo;
      split(v, &hi, &lo);
      const int64_t at = e * p.c_stride + row * p.ldc + col;
      *reinterpret_cast<half8_t*>(p.c_hi + at) = hi;
      if constexpr (EXACT || EPI == kApply) *reinterpret_cast<half8_t*>(p.c_lo + at) = lo;
    }
  };
  constexpr int kBlocks = KG == 2 ? 1 : IB;
  const int64_t col0 = n0 + rn, col = col0 + 8 * lc;
  const bool col_in = col < (EPI == kLast ? p.n : p.ldc);
  auto block_row = [&](int i) { return m0 + rm + 32 * (KG == 2 ? group : i); };
  // Y of a block's rows; rows and columns outside take the last ones' (unused)
  auto fetch = [&](int i, Given (&y)[4]) {
    if constexpr (EPI != kGram) {
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int64_t row = block_row(i) + 8 * it + lr;
        y[it] = given(row < p.m ? row : p.m - 1, col_in ? col : 0);
      }
    }
  };
  Given y[2][4];
  fetch(0, y[0]);
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    if (i + 1 < kBlocks) fetch(i + 1, y[(i + 1) % 2]);
    const int64_t row0 = block_row(i);
#pragma unroll
    for (int j = 0; j < JB; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int c = 8 * j + 2 * q + h;
        const float16_t& a = acc[i][j];
        const float four[4] = {a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]};
        __builtin_memcpy(tile + l32 * 64 + 4 * (c ^ (l32 & 15)), four, 16);
      }
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int r = 8 * it + lr;
      float v[8];
      __builtin_memcpy(v, tile + r * 64 + 4 * ((2 * lc) ^ (r & 15)), 16);
      __builtin_memcpy(v + 4, tile + r * 64 + 4 * ((2 * lc + 1) ^ (r & 15)), 16);
      if (row0 + r < p.m && col_in) finish(row0 + r, col, y[i % 2][it], v);
    }
    if (mirror) {
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int c = 16 * it + lane / 4;
        const int64_t row = col0 + c, to = row0 + 8 * (lane % 4);
        if (row >= p.n || to >= p.ldc) continue;
        float v[8];
#pragma unroll
        for (int b = 0; b < 8; ++b) {
          const int r = 8 * (lane % 4) + b;
          v[b] = tile[r * 64 + 4 * ((c / 4) ^ (r & 15)) + c % 4];
        }
        Given m = {};
        if constexpr (EPI == kPoly) m = given(row, to);
        finish(row, to, m, v);
      }
    }
  }
}

template <typename S>
int64_t tiles_of(bool sym, int64_t m, int64_t n) {
  const int64_t tm = (m + S::TM - 1) / S::TM, tn = (n + S::TN - 1) / S::TN;
  if (!sym) return tm * tn;
  int64_t t = 0;
  for (int64_t i = 0; i * (S::TM / S::TN) < tn; ++i) t += tn - i * (S::TM / S::TN);
  return t;
}

template <typename S, bool AM, bool BM, int EPI, bool EXACT>
hipError_t gemm(NsGemmArgs a, hipStream_t s) {
  a.tiles = (int32_t)tiles_of<S>(EPI == kGram || EPI == kPoly, a.m, a.n);
  ns_gemm_kernel<S, AM, BM, EPI, EXACT><<<(unsigned)(a.tiles * a.batch), 64 * S::NW, 0, s>>>(a);
  return hipGetLastError();
}

template <typename S, bool EXACT>
hipError_t one_product(int epi, bool tall, const NsGemmArgs& a, hipStream_t s) {
  if (epi == kGram)
    return tall ? gemm<S, true, true, kGram, EXACT>(a, s) : gemm<S, false, false, kGram, EXACT>(a, s);
  if (epi == kPoly) return gemm<S, false, false, kPoly, EXACT>(a, s);
  if (epi == kApply) return gemm<S, false, true, kApply, EXACT>(a, s);
  return gemm<S, false, true, kLast, EXACT>(a, s);
}

hipError_t product(int epi, bool tall, const NsGemmArgs& a, hipStream_t s) {
  // Huge where it has two tiles for every CU, else Wide where it has one: larger
  // tiles read each operand less often, smaller ones leave fewer CUs idle.
  // Microseconds a launch, Deep / Wide / Huge: A of 5120 x 2048 46 / 76 / 113; 128 of
  // 2048 x 768: A 242 / 211 / 207, P 139 / 139 / 125, X 682 / 558 / 524.  (X of 5120 x
  // 2048, 160 tiles of Huge and 320 of Wide: the call takes 575 with Huge and 632 with
  // Wide, which the rule gives it.)  Exact stages hold twice as much, so that Wide would
  // run alone on a CU: Huge where it has a tile for every CU.  A call of four 1000 x 2047
  // 735 (Deep) / 1339 us, of sixteen 1536 x 2048 5391 / 4925, of 128 2048 x 768 10617 /
  // 9480 (in turn over three stages of one part each: 775, 5165, 9980).
  const bool sym = epi == kGram || epi == kPoly;
  if (a.exact)
    return a.batch * tiles_of<Huge>(sym, a.m, a.n) >= 256 ? one_product<Huge, true>(epi, tall, a, s)
                                                          : one_product<Deep, true>(epi, tall, a, s);
  if (a.batch * tiles_of<Huge>(sym, a.m, a.n) >= 512) return one_product<Huge, false>(epi, tall, a, s);
  if (a.batch * tiles_of<Wide>(sym, a.m, a.n) >= 256) return one_product<Wide, false>(epi, tall, a, s);
  return one_product<Deep, false>(epi, tall, a, s);
}

int64_t pad64(int64_t v) { return (v + 63) / 64 * 64; }

}  // namespace

// ---- host ------------------------------------------------------------------------

// The iteration's bounds from |X0| <= 1: the largest singular value of an X that
// is kept, of |b A + c A A|, and the bits that a small one grows by per step.
// false: the coefficients let X leave the range that binary16 holds.
//
// fast: how many steps, the last ones, products of 11 bits may take so that the result
// stays near bf16's own rounding, 1.7e-3 in the mean.  Such a rounding is 2e-4 off in the
// mean; a step makes it of P and of X in P X, and of A in P, 2e-4 sqrt(2 |P|^2 + (1.7 |b A +
// 2 c A A|)^2) with both at their largest, and the steps' errors, which turn the singular
// vectors, add up as their squares.  The usual coefficients: 2.3e-3 for five steps (measured
// 1.2e-3 to 1.6e-3 for five in all, up to 2.3e-3 for the last of more), 8.4e-3 for 64 (7e-3
// to 3.5e-2).  A step that takes a singular value below half of itself would raise what was
// made before: none then.  5120 x 2048: five steps 0.63 ms, six 0.87, ten 1.89 (all exact
// from six on: 1.70 and 2.80).
bool ns_bounds(int steps, float a, float b, float c, NsScales* out) {
  double u = 1.0, top = 1.0, least = 1e30, off[kMaxNsSteps];
  auto f = [&](double x) { return fabs(x * (a + x * x * ((double)b + (double)c * x * x))); };
  for (int i = 0; i < steps; ++i) {
    // the largest |b y + c y y| and |b y + 2 c y y| on [0, u^2], and the least factor of a
    // singular value there: at its ends and the parabolas' vertices
    double most_p = 0.0, most_a = 0.0;
    for (const double y : {0.0, u * u, c != 0.0f ? -0.5 * b / c : 0.0, c != 0.0f ? -0.25 * b / c : 0.0}) {
      if (!(y >= 0.0 && y <= u * u)) continue;
      most_p = fmax(most_p, fabs(b * y + c * y * y));
      most_a = fmax(most_a, fabs(b * y + 2.0 * c * y * y));
      least = fmin(least, (a > 0.0f ? 1.0 : -1.0) * (a + b * y + c * y * y));
    }
    off[i] = 2.0 * most_p * most_p + 2.89 * most_a * most_a;
    // the extrema of a x + b x^3 + c x^5 on [0, u]: its end and the roots of
    // a + 3 b y + 5 c y^2, y = x^2
    double best = f(u);
    const double qa = 5.0 * c, qb = 3.0 * b, d = qb * qb - 4.0 * qa * a;
    if (qa != 0.0 && d >= 0.0) {
      for (double sg : {-1.0, 1.0}) {
        const double y = (-qb + sg * sqrt(d)) / (2.0 * qa);
        if (y > 0.0 && y < u * u) best = fmax(best, f(sqrt(y)));
      }
    } else if (qa == 0.0 && qb != 0.0) {
      const double y = -(double)a / qb;
      if (y > 0.0 && y < u * u) best = fmax(best, f(sqrt(y)));
    }
    // (a little more for the roundings)
    u = best * 1.02;
    if (!(u <= 8.0)) return false;
    if (u < 1e-3) u = 1e-3;
    if (i + 1 < steps) top = fmax(top, u);
  }
  const double l = top * top;
  const double v = fmax(fabs(a) + fabs(b) * l + fabs(c) * l * l, 1e-3);    // of P + a I
  if (!(v <= 8192.0)) return false;
  auto scale = [](double most) { return exp2(floor(log2(32768.0 / most))); };
  out->x = (float)scale(top);
  out->a = (float)scale(l);
  out->p = (float)scale(v);
  out->fast = 0;
  double sum = 0.0;
  while (least >= 0.5 && out->fast < steps && 2e-4 * sqrt(sum += off[steps - 1 - out->fast]) <= 2.4e-3)
    ++out->fast;
  const double grow = fabs(a) + fabs(b) + fabs(c);
  out->growth = grow <= 1.0 ? 0 : (int)ceil(log2(grow));
  return true;
}

// Whether X's two parts hold the digits of what a multiplies: an X of 16384 x 16384 starts
// with elements of 2^-14, 2^1 as they are kept, and the lower part is rounded to 2^-24.
// 2^-8 of them, where that is 2e-6 in the mean, is as far as a may take them (0.5 in 20
// steps: 256 x 384 1e-4 off, in 8 steps 4e-8).
bool ns_keeps_small(int steps, float a) { return steps * log2(fmin(fabs((double)a), 1.0)) >= -8.0; }

// Matrices that are taken together: as many as fit 4 GiB of workspace (128 of
// 2048 x 768 together take 4.5 ms; 62 at a time 4.9, 16, whose X would stay in
// the last-level cache, 5.3: their launches do not fill the last round of CUs).
int64_t ns_batch(int64_t batch, int64_t rows, int64_t cols) {
  const int64_t n = rows < cols ? rows : cols;
  const int64_t one = 8 * rows * pad64(cols) + 8 * n * pad64(n);
  int64_t c = (4LL << 30) / one;
  c = c < 1 ? 1 : (c > 32768 ? 32768 : c);
  return c < batch ? c : batch;
}

int ns_norm_parts(int64_t batch, int64_t rows) {
  int64_t p = 2048 / batch;
  p = p < 1 ? 1 : (p > 1024 ? 1024 : p);
  return (int)(p < rows ? p : rows);
}

hipError_t launch_newton_schulz(const NsArgs& a, hipStream_t s) {
  const bool tall = a.src.rows > a.src.cols;
  const int64_t n = tall ? a.src.cols : a.src.rows;
  const int64_t ld = pad64(a.src.cols), ldn = pad64(n);
  const int64_t xs = a.src.rows * ld, ns = n * ldn;         // elements of one X, one A
  const int64_t most = ns_batch(a.batch, a.src.rows, a.src.cols);
  const int parts = ns_norm_parts(most, a.src.rows);
  const size_t e0 = a.src.dtype == 0 ? 4 : 2, e1 = a.out_dtype == 0 ? 4 : 2;
  for (int64_t first = 0; first < a.batch; first += most) {
    const int64_t m = a.batch - first < most ? a.batch - first : most;
    NsSource src = a.src;
    src.g = static_cast<const char*>(a.src.g) + (size_t)first * a.src.ld_batch * e0;
    const dim3 gn(parts, (unsigned)m), gs((unsigned)((src.rows + 3) / 4), (unsigned)m);
    _Float16 *x = a.x[0], *xl = a.x[1], *y = a.x[2], *yl = a.x[3];
    if (src.dtype == 0) {
      ns_norm_kernel<0><<<gn, 256, 0, s>>>(src, a.norms);
      ns_start_kernel<0><<<gs, 256, 0, s>>>(src, a.norms, parts, a.eps, a.scales.x, ld, x, xl, a.k0);
    } else if (src.dtype == 1) {
      ns_norm_kernel<1><<<gn, 256, 0, s>>>(src, a.norms);
      ns_start_kernel<1><<<gs, 256, 0, s>>>(src, a.norms, parts, a.eps, a.scales.x, ld, x, xl, a.k0);
    } else {
      ns_norm_kernel<2><<<gn, 256, 0, s>>>(src, a.norms);
      ns_start_kernel<2><<<gs, 256, 0, s>>>(src, a.norms, parts, a.eps, a.scales.x, ld, x, xl, a.k0);
    }
    hipError_t st = hipGetLastError();
    for (int i = 0; i < a.steps && st == hipSuccess; ++i) {
      const NsMatrix X = {x, xl, xs, ld, (uint32_t)(xs * 2)};
      const NsMatrix A = {a.sq[0], a.sq[1], ns, ldn, (uint32_t)(ns * 2)};
      const NsMatrix P = {a.sq[2], a.sq[3], ns, ldn, (uint32_t)(ns * 2)};
      NsGemmArgs g{};
      g.batch = m; g.exact = i < a.exact; g.k0 = a.k0; g.growth = a.scales.growth;
      g.drop = i * a.scales.growth;
      // A
      g.a = g.b = X; g.m = g.n = n; g.k = tall ? src.rows : src.cols;
      g.c_hi = a.sq[0]; g.c_lo = a.sq[1]; g.c_stride = ns; g.ldc = ldn;
      g.f = a.scales.a / (a.scales.x * a.scales.x);
      st = product(kGram, tall, g, s);
      if (st != hipSuccess) break;
      // P
      g.a = g.b = g.y = A; g.k = n;
      g.c_hi = a.sq[2]; g.c_lo = a.sq[3];
      g.f = a.c * a.scales.p / (a.scales.a * a.scales.a);
      g.g = a.b * a.scales.p / a.scales.a;
      g.up = a.a * a.scales.p;
      st = product(kPoly, tall, g, s);
      if (st != hipSuccess) break;
      // X
      const bool last = i + 1 == a.steps;
      g.a = tall ? X : P; g.b = tall ? P : X; g.y = X;
      g.m = src.rows; g.n = src.cols; g.k = n;
      g.c_hi = y; g.c_lo = yl; g.c_stride = xs; g.ldc = ld;
      g.f = 1.0f / a.scales.p; g.g = a.a; g.up = a.out_scale / a.scales.x;
      g.out = static_cast<char*>(a.out) + (size_t)(first * src.rows * src.cols) * e1;
      g.out_dtype = a.out_dtype;
      st = product(last ? kLast : kApply, tall, g, s);
      _Float16* sw = x; x = y; y = sw;
      sw = xl; xl = yl; yl = sw;
    }
    if (st != hipSuccess) return st;
  }
  return hipSuccess;
}

}  // namespace nvfp4
