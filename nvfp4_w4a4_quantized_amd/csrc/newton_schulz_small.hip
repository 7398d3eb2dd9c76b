// newton_schulz_small.hip -- the orthogonalised update of matrices with a short
// side n of at most 64 (a low-rank adapter's, say).  The iteration acts on the
// short side alone: with A0 = X0 X0^T, every X is Q X0 for a polynomial Q of A0,
//   B = a I + b A + c A A,   Q <- Q B,   A <- B A B
// so the long side m is touched twice, for A0 and for Q X0, whatever the number
// of steps: 3 n^2 m + 4 steps n^3 operations instead of steps (3 n^2 m + n^3).
// |G|_F^2 is the trace of G G^T, so no pass is spent on the norm either.
//
// A's small eigenvalues grow by a^2 per step, and so would its roundings: all of
// it is binary64 (MFMA 16x16x4, products of binary32 values are exact), which is
// off by no more than a^(2 steps) 2^-53 n (ns_is_small keeps that below 2^-21 of
// the result; the usual five steps: 2^-32).
//
// Bound: the latency of three dependent launches, of the iteration's chain of
// products above all.  Measured: 64 matrices of 16 x 2048 (float32, 16.8 MB with
// the result) 17 us a call, 4.8 + 8.0 + 6.0 us of kernels; the GEMM form took
// 351.  The iteration alone takes 8, 14, 22 and 44 us for n up to 16, 32, 48, 64
// (there two tiles' products a wave; with four waves instead of sixteen 62).
#include "elem.h"
#include "launch.h"

namespace nvfp4 {

namespace {

typedef double f64x4_t __attribute__((ext_vector_type(4)));

// Lane l of MFMA 16x16x4 (binary64) gives row l % 16 of A and column l % 16 of B
// at k = l / 16, and holds rows l / 16 + 4 r of column l % 16 of the result.
__device__ __forceinline__ f64x4_t product(double a, double b, f64x4_t acc) {
  return __builtin_amdgcn_mfma_f64_16x16x4f64(a, b, acc, 0, 0, 0);
}

// Elements at, at + 1, at + 2, at + 3 of a row of `end`, zeros outside.
template <int DT>
__device__ __forceinline__ void four(const typename Elem<DT>::type* row, int64_t at, int64_t end,
                                     bool in, double (&v)[4]) {
  typename Elem<DT>::type x[4] = {};
  if (in && at + 4 <= end) {
    __builtin_memcpy(x, row + at, sizeof(x));
  } else if (in) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at + i < end) x[i] = row[at + i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (double)Elem<DT>::to_float(x[i]);
}

// Partial G G^T (G^T G of a tall G) over a share of the long side.  Grid:
// (matrices, shares); the four waves take 16 of the long side in turn.
template <int DT, int NB, bool TALL>
__global__ __launch_bounds__(256) void ns_gram_kernel(NsSource g, int64_t share, double* part) {
  typedef typename Elem<DT>::type T;
  constexpr int kTiles = NB * (NB + 1) / 2;
  __shared__ double red[4][kTiles][256];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, i = lane % 16, q = lane / 16;
  const int n = (int)(TALL ? g.cols : g.rows);
  const int64_t m = TALL ? g.rows : g.cols;
  const T* p = static_cast<const T*>(g.g) + (int64_t)blockIdx.x * g.ld_batch;
  const int64_t k0 = blockIdx.y * share, k1 = k0 + share < m ? k0 + share : m;
  f64x4_t acc[kTiles];
#pragma unroll
  for (int t = 0; t < kTiles; ++t) acc[t] = (f64x4_t){0.0, 0.0, 0.0, 0.0};
  for (int64_t k = k0 + 16 * wave; k < k1; k += 64) {
    double v[NB][4];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int r = 16 * b + i;
      if constexpr (TALL) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t row = k + 4 * q + e;
          v[b][e] = r < n && row < k1 ? (double)Elem<DT>::to_float(p[row * g.ld_row + r]) : 0.0;
        }
      } else {
        four<DT>(p + (r < n ? r : 0) * g.ld_row, k + 4 * q, k1, r < n, v[b]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      int t = 0;
#pragma unroll
      for (int a = 0; a < NB; ++a)
#pragma unroll
        for (int b = a; b < NB; ++b, ++t) acc[t] = product(v[a][e], v[b][e], acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < kTiles; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][t][r * 64 + lane] = acc[t][r];
  __syncthreads();
  double* out = part + ((int64_t)blockIdx.x * gridDim.y + blockIdx.y) * (kTiles * 256);
  for (int v = threadIdx.x; v < kTiles * 256; v += 256)
    out[v] = ((red[0][v / 256][v % 256] + red[1][v / 256][v % 256]) + red[2][v / 256][v % 256]) +
             red[3][v / 256][v % 256];
}

// Tile (ti, tj) of a product of two symmetric matrices that commute, read along
// their rows.
template <int N>
__device__ __forceinline__ f64x4_t tile_product(const double* x, const double* y, int ti, int tj, int lane) {
  const int i = lane % 16, q = lane / 16;
  f64x4_t acc = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 4
  for (int k = 0; k < N; k += 4) acc = product(x[(k + q) * N + 16 * ti + i], y[(k + q) * N + 16 * tj + i], acc);
  return acc;
}

template <int N>
__device__ __forceinline__ void put_tile(double* x, int ti, int tj, int lane, f64x4_t v) {
  const int i = lane % 16, q = lane / 16;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = 16 * ti + 4 * r + q, col = 16 * tj + i;
    x[row * N + col] = v[r];
    if (ti != tj) x[col * N + row] = v[r];
  }
}

// A tile of a product to every wave where there are as many waves as tiles.
template <int NB>
constexpr int kIterateWaves = NB == 1 ? 4 : (NB == 2 ? 8 : 16);

// The iteration on the n x n matrices, a workgroup a matrix: Q f scale to `qs`,
// f = 1 / (|G|_F + eps).
template <int NB>
__global__ __launch_bounds__(64 * kIterateWaves<NB>) void ns_iterate_kernel(const double* part, int shares, int steps,
                                                         double a, double b, double c, double eps,
                                                         double scale, double* qs) {
  constexpr int N = 16 * NB, kTiles = NB * (NB + 1) / 2;
  constexpr int W = kIterateWaves<NB>, kMine = (kTiles + W - 1) / W;   // a wave's tiles of a product
  __shared__ double A[N * N], B[N * N], Q[N * N], T[N * N];
  __shared__ double diag[N];
  const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int i = lane % 16, q = lane / 16;
  const double* p = part + (int64_t)blockIdx.x * shares * (kTiles * 256);
  auto tile_at = [](int t, int* ti, int* tj) {      // the t-th upper tile
    int r = 0;
    while (t >= NB - r) {
      t -= NB - r;
      ++r;
    }
    *ti = r;
    *tj = r + t;
  };
  f64x4_t mine[kMine];
#pragma unroll
  for (int s = 0; s < kMine; ++s) {
    const int t = wave + W * s;
    if (t >= kTiles) continue;
    int ti, tj;
    tile_at(t, &ti, &tj);
    f64x4_t v = {0.0, 0.0, 0.0, 0.0};
    for (int w = 0; w < shares; ++w)
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] += p[(int64_t)w * (kTiles * 256) + t * 256 + r * 64 + lane];
    mine[s] = v;
    if (ti == tj) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (4 * r + q == i) diag[16 * ti + i] = v[r];
    }
  }
  __syncthreads();
  double square = 0.0;
  for (int r = 0; r < N; ++r) square += diag[r];
  const double norm = sqrt(square), f = norm == 0.0 ? 0.0 : 1.0 / (norm + eps);
#pragma unroll
  for (int s = 0; s < kMine; ++s) {
    const int t = wave + W * s;
    if (t >= kTiles) continue;
    int ti, tj;
    tile_at(t, &ti, &tj);
    // (f f alone may leave the range where G's values are tiny)
    put_tile<N>(A, ti, tj, lane, (mine[s] * f) * f);
  }
  __syncthreads();
  for (int step = 0; step < steps; ++step) {
    const bool last = step + 1 == steps;
    double* into = step == 0 ? Q : B;               // Q = B in the first step
#pragma unroll
    for (int s = 0; s < kMine; ++s) {
      const int t = wave + W * s;
      if (t >= kTiles) continue;
      int ti, tj;
      tile_at(t, &ti, &tj);
      f64x4_t v = tile_product<N>(A, A, ti, tj, lane);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * ti + 4 * r + q, col = 16 * tj + i;
        v[r] = c * v[r] + b * A[row * N + col] + (row == col ? a : 0.0);
      }
      put_tile<N>(into, ti, tj, lane, v);
    }
    __syncthreads();
    // Q B and A B beside each other
    f64x4_t qb[kMine];
#pragma unroll
    for (int s = 0; s < kMine; ++s) {
      const int t = (wave + W / 2) % W + W * s;         // (the waves without a tile of A B first)
      if (t >= kTiles || step == 0) continue;
      int ti, tj;
      tile_at(t, &ti, &tj);
      qb[s] = tile_product<N>(Q, B, ti, tj, lane);
    }
    if (!last) {
#pragma unroll
      for (int s = 0; s < kMine; ++s) {
        const int t = wave + W * s;
        if (t >= kTiles) continue;
        int ti, tj;
        tile_at(t, &ti, &tj);
        put_tile<N>(T, ti, tj, lane, tile_product<N>(A, into, ti, tj, lane));
      }
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < kMine; ++s) {
      const int t = (wave + W / 2) % W + W * s;
      if (t >= kTiles || step == 0) continue;
      int ti, tj;
      tile_at(t, &ti, &tj);
      put_tile<N>(Q, ti, tj, lane, qb[s]);
    }
    if (!last) {
#pragma unroll
      for (int s = 0; s < kMine; ++s) {
        const int t = wave + W * s;
        if (t >= kTiles) continue;
        int ti, tj;
        tile_at(t, &ti, &tj);
        put_tile<N>(A, ti, tj, lane, tile_product<N>(T, step == 0 ? into : B, ti, tj, lane));
      }
    }
    __syncthreads();
  }
  double* out = qs + (int64_t)blockIdx.x * (N * N);
  for (int v = threadIdx.x; v < N * N; v += 64 * W) out[v] = Q[v] * (f * scale);
}

template <int OT>
__device__ __forceinline__ void put4(void* out, int64_t at, int64_t count, const double (&v)[4]) {
  typename Elem<OT>::type o[4], *p = static_cast<typename Elem<OT>::type*>(out) + at;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = Elem<OT>::from_float((float)v[i]);
  if (count >= 4) {
    __builtin_memcpy(p, o, sizeof(o));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < count) p[i] = o[i];
  }
}

// Q G (G Q of a tall G).  Grid: (matrices, shares of the long side); a wave
// takes 64 columns (16 rows) at a time.
template <int DT, int NB, bool TALL>
__global__ __launch_bounds__(256) void ns_apply_kernel(NsSource g, int64_t share, const double* qs,
                                                       void* out, int out_dtype) {
  typedef typename Elem<DT>::type T;
  constexpr int N = 16 * NB, kStep = TALL ? 16 : 64;
  __shared__ double Q[N * N];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, i = lane % 16, q = lane / 16;
  const int n = (int)(TALL ? g.cols : g.rows);
  const int64_t m = TALL ? g.rows : g.cols;
  const T* p = static_cast<const T*>(g.g) + (int64_t)blockIdx.x * g.ld_batch;
  const int64_t o = (int64_t)blockIdx.x * g.rows * g.cols;
  for (int v = threadIdx.x; v < N * N; v += 256) Q[v] = qs[(int64_t)blockIdx.x * (N * N) + v];
  __syncthreads();
  auto put = [&](int64_t at, int64_t count, const double (&v)[4]) {
    if (out_dtype == 0) put4<0>(out, at, count, v);
    else if (out_dtype == 1) put4<1>(out, at, count, v);
    else put4<2>(out, at, count, v);
  };
  const int64_t k0 = blockIdx.y * share, k1 = k0 + share < m ? k0 + share : m;
  for (int64_t k = k0 + kStep * wave; k < k1; k += 4 * kStep) {
    if constexpr (TALL) {
      // result rows: columns j of G Q, in the order j = 4 (row % 4) + row / 4 of
      // the tile, so that a lane ends with four consecutive ones
      const int64_t row = k + i;
      f64x4_t acc[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[b] = (f64x4_t){0.0, 0.0, 0.0, 0.0};
#pragma unroll
      for (int s = 0; s < NB; ++s) {
        double v[4];
        four<DT>(p + (row < k1 ? row : k1 - 1) * g.ld_row, 16 * s + 4 * q, n, row < k1, v);
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int b = 0; b < NB; ++b)
            acc[b] = product(Q[(16 * s + 4 * q + e) * N + 16 * b + 4 * (i % 4) + i / 4], v[e], acc[b]);
      }
      if (row >= k1) continue;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const double v[4] = {acc[b][0], acc[b][1], acc[b][2], acc[b][3]};
        const int col = 16 * b + 4 * q;
        if (col < n) put(o + row * g.cols + col, n - col, v);
      }
    } else {
      const int64_t col = k + 4 * i;
      f64x4_t acc[NB][4];
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[b][e] = (f64x4_t){0.0, 0.0, 0.0, 0.0};
#pragma unroll
      for (int s = 0; s < N / 4; ++s) {
        const int r = 4 * s + q;
        double v[4];
        four<DT>(p + (r < n ? r : 0) * g.ld_row, col, k1, r < n, v);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const double w = Q[r * N + 16 * b + i];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[b][e] = product(w, v[e], acc[b][e]);
        }
      }
      if (col >= k1) continue;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * b + 4 * r + q;
          const double v[4] = {acc[b][0][r], acc[b][1][r], acc[b][2][r], acc[b][3][r]};
          if (row < n) put(o + row * g.cols + col, k1 - col, v);
        }
    }
  }
}

constexpr int64_t kMostMatrices = 32768;

template <int DT, int NB>
hipError_t run(const NsArgs& a, const NsSource& src, int64_t batch, void* out, hipStream_t s) {
  const bool tall = src.rows > src.cols;
  const int64_t m = tall ? src.rows : src.cols;
  const int shares = ns_small_shares(batch, m);
  const int64_t share = ((m + shares - 1) / shares + 63) / 64 * 64;
  const dim3 g1((unsigned)batch, shares);
  if (tall) ns_gram_kernel<DT, NB, true><<<g1, 256, 0, s>>>(src, share, a.small_parts);
  else ns_gram_kernel<DT, NB, false><<<g1, 256, 0, s>>>(src, share, a.small_parts);
  ns_iterate_kernel<NB><<<(unsigned)batch, 64 * kIterateWaves<NB>, 0, s>>>(a.small_parts, shares, a.steps, a.a, a.b, a.c,
                                                        a.eps, a.out_scale, a.small_q);
  // one round of a workgroup's waves while there are fewer than four a CU
  int64_t each = 256;
  while (each < 4096 && batch * ((m + each - 1) / each) > 2048) each *= 2;
  const dim3 g3((unsigned)batch, (unsigned)((m + each - 1) / each));
  if (tall) ns_apply_kernel<DT, NB, true><<<g3, 256, 0, s>>>(src, each, a.small_q, out, a.out_dtype);
  else ns_apply_kernel<DT, NB, false><<<g3, 256, 0, s>>>(src, each, a.small_q, out, a.out_dtype);
  return hipGetLastError();
}

template <int DT>
hipError_t run_dt(const NsArgs& a, const NsSource& src, int64_t batch, void* out, hipStream_t s) {
  const int64_t n = src.rows < src.cols ? src.rows : src.cols;
  if (n <= 16) return run<DT, 1>(a, src, batch, out, s);
  if (n <= 32) return run<DT, 2>(a, src, batch, out, s);
  if (n <= 48) return run<DT, 3>(a, src, batch, out, s);
  return run<DT, 4>(a, src, batch, out, s);
}

}  // namespace

// Whether the iteration runs on the short side alone: n <= 64, and binary64's
// roundings of A stay below 2^-21 of the result.
bool ns_is_small(int64_t rows, int64_t cols, int steps, float a, float b, float c) {
  const int64_t n = rows < cols ? rows : cols;
  const double grow = fmax(fabs((double)a), 1.0);
  return n <= 64 && 2.0 * steps * log2(grow) <= 26.0;
}

// Side of the tiles' matrix, and workgroups that share a matrix's long side: two
// a CU, of no less than 64 of it.
int64_t ns_small_side(int64_t n) { return (n + 15) / 16 * 16; }
int ns_small_shares(int64_t batch, int64_t m) {
  const int64_t want = 512 / batch, most = (m + 255) / 256;
  const int64_t w = want < most ? want : most;
  return (int)(w < 1 ? 1 : (w > 16 ? 16 : w));
}
int64_t ns_small_batch(int64_t batch) { return batch < kMostMatrices ? batch : kMostMatrices; }

hipError_t launch_newton_schulz_small(const NsArgs& a, hipStream_t s) {
  const size_t e0 = a.src.dtype == 0 ? 4 : 2, e1 = a.out_dtype == 0 ? 4 : 2;
  const int64_t most = ns_small_batch(a.batch);
  for (int64_t first = 0; first < a.batch; first += most) {
    const int64_t m = a.batch - first < most ? a.batch - first : most;
    NsSource src = a.src;
    src.g = static_cast<const char*>(a.src.g) + (size_t)first * a.src.ld_batch * e0;
    void* out = static_cast<char*>(a.out) + (size_t)(first * src.rows * src.cols) * e1;
    const hipError_t st = src.dtype == 0   ? run_dt<0>(a, src, m, out, s)
                          : src.dtype == 1 ? run_dt<1>(a, src, m, out, s)
                                           : run_dt<2>(a, src, m, out, s);
    if (st != hipSuccess) return st;
  }
  return hipSuccess;
}

}  // namespace nvfp4
