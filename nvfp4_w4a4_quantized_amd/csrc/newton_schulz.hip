// newton_schulz.hip -- the orthogonalised update of a weight's gradient:
//   X0 = G / (|G|_F + eps),   X <- a X + P X,   P = b A + c A A,   A = X X^T
// for wide G (rows <= cols), and from the other side, A = X^T X, X <- a X + X P,
// for tall G, so that nothing is transposed and A is as small as it can be.
//
// Arithmetic.  X is kept as two binary16 parts (hi, and lo the rest: 22 bits)
// times a power of two that brings its largest possible element near the top of
// the range, and a X is taken from both.  The products run on the matrix cores
// in binary16 with binary32 sums:
//   - 16-bit "fast" products take hi alone.  What they lose, 2^-12 relative to P
//     X, is lost where P X is as large as the result; the small singular values,
//     which the iteration multiplies by a per step, keep the 22 bits of a X.
//     Against binary64 the result of 768 x 2048 gradients is 1e-3 off (bf16's own
//     rounding: 1.7e-3; bf16 products: 2e-2).
//   - "exact" products take hi hi + hi lo + lo hi: 1.8e-6 off, as binary32.
// A gradient far below eps keeps its digits: X is multiplied by a further 2^k0,
// k0 = floor(-log2 |X0|), which shrinks by the iteration's growth every step.
//
// One GEMM kernel computes all three products; a symmetric result is computed
// in its upper tiles and mirrored.  Operands lie K-contiguous (X of the wide
// Gram product, A, P, X of the tall update) or K-major (X of the tall Gram
// product and of the wide update) and go from memory straight into a four-slot
// LDS ring; K-major tiles are read with the transposing LDS loads.
#include <type_traits>

#include "elem.h"
#include "gemm_common.h"
#include "launch.h"

namespace nvfp4 {

namespace {

typedef _Float16 half4_t __attribute__((ext_vector_type(4)));
typedef short short4_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) short4_t lds_short4_t;

constexpr int kBK = 32;       // k of a stage

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
  double sum = 0.0;
  for (int i = 0; i < parts; ++i) sum += part[e * parts + i];
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
  for (int64_t c = (int64_t)(threadIdx.x % kWave) * 8; c < ld; c += kWave * 8) {
    half8_t h, l;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double v = c + i < g.cols ? f * (double)Elem<DT>::to_float(row[c + i]) : 0.0;
      h[i] = (_Float16)(float)v;
      l[i] = (_Float16)(float)(v - (double)h[i]);
    }
    *reinterpret_cast<half8_t*>(hi + at + c) = h;
    *reinterpret_cast<half8_t*>(lo + at + c) = l;
  }
}

// ---- the products --------------------------------------------------------------

// LDS tiles are unpadded and XOR-swizzled in 16-byte chunks (a direct-to-LDS
// load writes one contiguous KiB per wave instruction):
//   K-contiguous [T rows][32 k]: chunk c of row r at c ^ (r / 4) % 4
//   K-major [32 k][T columns]: chunk c of row r at c ^ 4 (r % 4)  (T = 64: 2 (r % 4))
template <int T>
__device__ __forceinline__ int swz_major(int r, int c) {
  return c ^ ((T >= 128 ? 4 : 2) * (r & 3));
}
__device__ __forceinline__ int swz_row(int r, int c) { return c ^ ((r >> 2) & 3); }

// The matrix-core operand: lane l has row (column) r0 + l % 32 of the tile and
// k = k0 + 8 (l / 32) + 0..7.
template <int T, bool MAJOR>
__device__ __forceinline__ half8_t fragment(const _Float16* s, int r0, int k0, int lane) {
  if constexpr (MAJOR) {
    const int r = k0 + (lane >> 5) * 8 + ((lane & 15) >> 2);
    const int col = r0 + ((lane >> 4) & 1) * 16 + 4 * (lane & 3);
    const int off = 8 * swz_major<T>(r, col >> 3) + (col & 7);   // rows r and r + 4 share it
    const short4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4_t*)(s + r * T + off));
    const short4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4_t*)(s + (r + 4) * T + off));
    const auto both = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    half8_t v;
    __builtin_memcpy(&v, &both, 16);
    return v;
  } else {
    const int r = r0 + (lane & 31), c = (k0 >> 3) + (lane >> 5);
    return *reinterpret_cast<const half8_t*>(s + r * 32 + 8 * swz_row(r, c));
  }
}

__device__ __forceinline__ void split(const float (&v)[4], half4_t* hi, half4_t* lo) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const _Float16 h = (_Float16)v[i];
    (*hi)[i] = h;
    (*lo)[i] = (_Float16)(v[i] - (float)h);
  }
}

// Four consecutive results of the last step.
template <int OT>
__device__ __forceinline__ void put4(void* out, int64_t at, int count, bool wide, const float (&v)[4]) {
  typename Elem<OT>::type o[4], *p = static_cast<typename Elem<OT>::type*>(out) + at;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = Elem<OT>::from_float(v[i]);
  if (wide) {
    __builtin_memcpy(p, o, sizeof(o));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < count) p[i] = o[i];
  }
}

// T x T tiles, NW waves in two rows, each IB x JB blocks of 32 x 32.
template <int T>
struct TileShape;
template <>
struct TileShape<256> {
  static constexpr int kNW = 8, kIB = 4, kJB = 2;
};
template <>
struct TileShape<128> {
  static constexpr int kNW = 4, kIB = 2, kJB = 2;
};

// C = A B over k with the epilogue EPI; AM, BM: the operand is K-major.
template <int T, bool AM, bool BMAJ, int EPI>
__global__ __launch_bounds__(64 * TileShape<T>::kNW, T == 256 ? 1 : 2) void ns_gemm_kernel(NsGemmArgs p) {
  constexpr int NW = TileShape<T>::kNW, IB = TileShape<T>::kIB, JB = TileShape<T>::kJB;
  constexpr int REGION = T * kBK * 2;           // bytes of one operand's stage
  constexpr int QN = REGION / 1024 / NW;        // its load instructions per wave
  __shared__ __align__(16) uint8_t S0[2 * REGION];
  __shared__ __align__(16) uint8_t S1[2 * REGION];
  __shared__ __align__(16) uint8_t S2[2 * REGION];
  __shared__ __align__(16) uint8_t S3[2 * REGION];
  constexpr bool SYM = EPI == kGram || EPI == kPoly;
  const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);

  // consecutive tiles of a matrix on one XCD (workgroups go round the eight)
  const int nb = gridDim.x, xcd = blockIdx.x % 8, in = blockIdx.x / 8;
  const int t = xcd * (nb / 8) + (xcd < nb % 8 ? xcd : nb % 8) + in;
  const int tiles_n = (int)((p.n + T - 1) / T);
  const int tiles_m = (int)((p.m + T - 1) / T);
  const int per = SYM ? tiles_n * (tiles_n + 1) / 2 : tiles_m * tiles_n;
  const int e = t / per;
  int ti = 0, tj = t % per;
  if (SYM) {
    while (tj >= tiles_n - ti) {                // row ti has tiles_n - ti tiles
      tj -= tiles_n - ti;
      ++ti;
    }
    tj += ti;
  } else {
    ti = tj / tiles_n;
    tj %= tiles_n;
  }
  const int64_t m0 = (int64_t)ti * T, n0 = (int64_t)tj * T;

  const __amdgpu_buffer_rsrc_t ahi = buffer_rsrc(p.a.hi + e * p.a.stride, p.a.bytes);
  const __amdgpu_buffer_rsrc_t bhi = buffer_rsrc(p.b.hi + e * p.b.stride, p.b.bytes);
  const __amdgpu_buffer_rsrc_t alo = buffer_rsrc(p.a.lo + e * p.a.stride, p.a.bytes);
  const __amdgpu_buffer_rsrc_t blo = buffer_rsrc(p.b.lo + e * p.b.stride, p.b.bytes);
  const int steps = (int)((p.k + kBK - 1) / kBK), nst = steps * p.parts;

  // A lane's offsets of stage 0.  Rows past the matrix lie past its resource
  // and read zeros; columns past ld are masked.
  uint32_t ao[QN], bo[QN];
  auto place = [&](bool major, int64_t first, int64_t ld, int q) -> uint32_t {
    const int i = wave + NW * q;
    if (major) {
      constexpr int kLanes = T / 8, kRows = kWave / kLanes;   // lanes of a row; rows of an instruction
      const int r = i * kRows + lane / kLanes, c = swz_major<T>(r, lane % kLanes);
      const int64_t col = first + 8 * c;
      return col < ld ? (uint32_t)((r * ld + col) * 2) : kNone;
    }
    const int r = 16 * i + lane / 4, c = swz_row(r, lane % 4);
    return (uint32_t)(((first + r) * ld + 8 * c) * 2);
  };
#pragma unroll
  for (int q = 0; q < QN; ++q) {
    ao[q] = place(AM, m0, p.a.ld, q);
    bo[q] = place(BMAJ, n0, p.b.ld, q);
  }
  const uint32_t astep = AM ? (uint32_t)(p.a.ld * kBK * 2) : kBK * 2;
  const uint32_t bstep = BMAJ ? (uint32_t)(p.b.ld * kBK * 2) : kBK * 2;

  auto slot = [&](auto u) -> uint8_t* {
    constexpr int U = decltype(u)::value;
    if constexpr (U == 0) return S0;
    else if constexpr (U == 1) return S1;
    else if constexpr (U == 2) return S2;
    else return S3;
  };
  // stage st: step st / parts of k, and of the parts hi hi, hi lo, lo hi the
  // (st % parts)-th; stages past the last read zeros
  int step = 0, part = 0;
  auto load = [&](auto u, int st) {
    uint8_t* s = slot(u);
    const bool live = st < nst;
    const uint32_t sa = (uint32_t)step * astep, sb = (uint32_t)step * bstep;
    const __amdgpu_buffer_rsrc_t ra = part == 2 ? alo : ahi, rb = part == 1 ? blo : bhi;
#pragma unroll
    for (int q = 0; q < QN; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_void_t*)(s + (wave + NW * q) * 1024), 16,
                                               (int)(live ? ao[q] + sa : kNone), 0, 0, 0);
#pragma unroll
    for (int q = 0; q < QN; ++q)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_void_t*)(s + REGION + (wave + NW * q) * 1024), 16,
                                               (int)(live ? bo[q] + sb : kNone), 0, 0, 0);
    if (++part == p.parts) {
      part = 0;
      ++step;
    }
  };

  float16_t acc[IB][JB];
#pragma unroll
  for (int i = 0; i < IB; ++i)
#pragma unroll
    for (int j = 0; j < JB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  const int wm = wave % 2, wn = wave / 2;
  const int rm = wm * IB * 32, rn = wn * JB * 32;        // the wave's first row and column
  auto multiply = [&](auto u) {
    const _Float16* la = reinterpret_cast<const _Float16*>(slot(u));
    const _Float16* lb = reinterpret_cast<const _Float16*>(slot(u) + REGION);
    half8_t fa[kBK / 16][IB], fb[kBK / 16][JB];
#pragma unroll
    for (int kk = 0; kk < kBK / 16; ++kk) {
#pragma unroll
      for (int j = 0; j < JB; ++j) fb[kk][j] = fragment<T, BMAJ>(lb, rn + j * 32, kk * 16, lane);
#pragma unroll
      for (int i = 0; i < IB; ++i) fa[kk][i] = fragment<T, AM>(la, rm + i * 32, kk * 16, lane);
    }
#pragma unroll
    for (int kk = 0; kk < kBK / 16; ++kk)
#pragma unroll
      for (int i = 0; i < IB; ++i)
#pragma unroll
        for (int j = 0; j < JB; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fb[kk][j], fa[kk][i], acc[i][j], 0, 0, 0);
  };

  // Stages st + 1 .. st + 3 are in flight while stage st is multiplied: the
  // wait leaves the two newest stages' loads outstanding, the barrier (without
  // a fence, which would wait for all) says that every wave's loads of st have
  // landed and that slot st + 3 is no longer read.
  constexpr int WAIT = 2 * 2 * QN;
  constexpr int WAIT_IMM = (WAIT & 15) | ((WAIT >> 4) << 14) | (7 << 4) | (15 << 8);
  using C0 = std::integral_constant<int, 0>;
  using C1 = std::integral_constant<int, 1>;
  using C2 = std::integral_constant<int, 2>;
  using C3 = std::integral_constant<int, 3>;
  auto turn = [&](auto u, int st) {
    using Next = std::integral_constant<int, (decltype(u)::value + 3) % 4>;
    __builtin_amdgcn_s_waitcnt(WAIT_IMM);
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    load(Next{}, st + 3);
    if (st < nst) multiply(u);
  };
  load(C0{}, 0);
  load(C1{}, 1);
  load(C2{}, 2);
  for (int st = 0; st < nst; st += 4) {
    turn(C0{}, st);
    turn(C1{}, st + 1);
    turn(C2{}, st + 2);
    turn(C3{}, st + 3);
  }
  __builtin_amdgcn_s_waitcnt((7 << 4) | (15 << 8));      // no load into LDS outlives the loop
  __atomic_signal_fence(__ATOMIC_SEQ_CST);

  // ---- epilogue: the operands are swapped in the products, so acc[i][j][4 q + c]
  // is row l % 32 and column 8 q + 4 (l / 32) + c of block (i, j).
  const int h = lane >> 5, l32 = lane & 31;
  const int k0 = p.k0[e], kj = k0 - p.drop > 0 ? k0 - p.drop : 0;
  const int kn = kj - p.growth > 0 ? kj - p.growth : 0;
  const float f = EPI == kGram ? ldexpf(p.f, -2 * kj) : p.f;
  const float up = EPI == kApply ? ldexpf(1.0f, kn - kj) : (EPI == kLast ? ldexpf(p.up, -kj) : 1.0f);
#pragma unroll
  for (int i = 0; i < IB; ++i) {
    const int64_t row = m0 + rm + i * 32 + l32;
    if (row >= p.m) continue;
#pragma unroll
    for (int j = 0; j < JB; ++j) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t col = n0 + rn + j * 32 + 8 * q + 4 * h;
        if (col >= p.ldc) continue;
        float v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) v[c] = f * acc[i][j][4 * q + c];
        const int64_t at = (int64_t)e * p.c_stride + row * p.ldc + col;
        if constexpr (EPI == kPoly || EPI == kApply || EPI == kLast) {
          // b A + c A A, or a X + P X, from both parts
          const half4_t yh = *reinterpret_cast<const half4_t*>(p.y.hi + e * p.y.stride + row * p.y.ld + col);
          const half4_t yl = p.y.lo ? *reinterpret_cast<const half4_t*>(p.y.lo + e * p.y.stride + row * p.y.ld + col)
                                    : (half4_t){0, 0, 0, 0};
#pragma unroll
          for (int c = 0; c < 4; ++c) v[c] = up * (fmaf(p.g, (float)yl[c], v[c]) + p.g * (float)yh[c]);
        }
        if constexpr (EPI == kLast) {
          const int count = p.n - col < 4 ? (int)(p.n - col) : 4;
          if (count <= 0) continue;
          const int64_t o = ((int64_t)e * p.m + row) * p.n + col;
          if (p.out_dtype == 0) put4<0>(p.out, o, count, p.wide, v);
          else if (p.out_dtype == 1) put4<1>(p.out, o, count, p.wide, v);
          else put4<2>(p.out, o, count, p.wide, v);
        } else {
          half4_t hi, lo;
          split(v, &hi, &lo);
          *reinterpret_cast<half4_t*>(p.c_hi + at) = hi;
          if (p.c_lo) *reinterpret_cast<half4_t*>(p.c_lo + at) = lo;
          if (SYM && ti < tj) {                  // the mirrored tile
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              if (col + c >= p.n) continue;
              const int64_t to = (int64_t)e * p.c_stride + (col + c) * p.ldc + row;
              p.c_hi[to] = hi[c];
              if (p.c_lo) p.c_lo[to] = lo[c];
            }
          }
        }
      }
    }
  }
}

template <int T, bool AM, bool BM, int EPI>
hipError_t gemm(const NsGemmArgs& a, hipStream_t s) {
  const int64_t tm = (a.m + T - 1) / T, tn = (a.n + T - 1) / T;
  const int64_t per = EPI == kGram || EPI == kPoly ? tn * (tn + 1) / 2 : tm * tn;
  ns_gemm_kernel<T, AM, BM, EPI><<<(unsigned)(per * a.batch), 64 * TileShape<T>::kNW, 0, s>>>(a);
  return hipGetLastError();
}

template <int T>
hipError_t one_product(int epi, bool tall, const NsGemmArgs& a, hipStream_t s) {
  if (epi == kGram) return tall ? gemm<T, true, true, kGram>(a, s) : gemm<T, false, false, kGram>(a, s);
  if (epi == kPoly) return gemm<T, false, false, kPoly>(a, s);
  if (epi == kApply) return tall ? gemm<T, false, true, kApply>(a, s) : gemm<T, false, true, kApply>(a, s);
  return gemm<T, false, true, kLast>(a, s);
}

hipError_t product(int epi, bool tall, const NsGemmArgs& a, hipStream_t s) {
  return one_product<128>(epi, tall, a, s);
}

int64_t pad64(int64_t v) { return (v + 63) / 64 * 64; }

}  // namespace

// ---- host ------------------------------------------------------------------------

// The iteration's bounds from |X0| <= 1: the largest singular value of an X that
// is kept, of |b A + c A A|, and the bits that a small one grows by per step.
// false: the coefficients let X leave the range that binary16 holds.
bool ns_bounds(int steps, float a, float b, float c, NsScales* out) {
  double u = 1.0, top = 1.0;
  auto f = [&](double x) { return fabs(x * (a + x * x * ((double)b + (double)c * x * x))); };
  for (int i = 0; i < steps; ++i) {
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
  const double v = fmax(fabs(b) * l + fabs(c) * l * l, 1e-3);
  if (!(v <= 8192.0)) return false;
  auto scale = [](double most) { return exp2(floor(log2(32768.0 / most))); };
  out->x = (float)scale(top);
  out->a = (float)scale(l);
  out->p = (float)scale(v);
  const double grow = fabs(a) + fabs(b) + fabs(c);
  out->growth = grow <= 1.0 ? 0 : (int)ceil(log2(grow));
  return true;
}

// Matrices that are taken together: as many as fit 1 GiB of workspace.
int64_t ns_batch(int64_t batch, int64_t rows, int64_t cols) {
  const int64_t n = rows < cols ? rows : cols;
  const int64_t one = 8 * rows * pad64(cols) + 8 * n * pad64(n);
  int64_t c = (1LL << 30) / one;
  c = c < 1 ? 1 : (c > 32768 ? 32768 : c);
  return c < batch ? c : batch;
}

int ns_norm_parts(int64_t batch, int64_t rows) {
  int64_t p = 1024 / batch;
  p = p < 1 ? 1 : (p > 64 ? 64 : p);
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
      g.batch = m; g.parts = a.exact ? 3 : 1; g.k0 = a.k0; g.growth = a.scales.growth;
      g.drop = i * a.scales.growth;
      // A
      g.a = g.b = X; g.m = g.n = n; g.k = tall ? src.rows : src.cols;
      g.c_hi = a.sq[0]; g.c_lo = a.exact ? a.sq[1] : nullptr; g.c_stride = ns; g.ldc = ldn;
      g.f = a.scales.a / (a.scales.x * a.scales.x);
      st = product(kGram, tall, g, s);
      if (st != hipSuccess) break;
      // P
      g.a = g.b = g.y = A; g.k = n;
      if (!a.exact) g.y.lo = nullptr;
      g.c_hi = a.sq[2]; g.c_lo = a.exact ? a.sq[3] : nullptr;
      g.f = a.c * a.scales.p / (a.scales.a * a.scales.a);
      g.g = a.b * a.scales.p / a.scales.a;
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
      g.wide = src.cols % 4 == 0;
      st = product(last ? kLast : kApply, tall, g, s);
      _Float16* sw = x; x = y; y = sw;
      sw = xl; xl = yl; yl = sw;
    }
    if (st != hipSuccess) return st;
  }
  return hipSuccess;
}

}  // namespace nvfp4
