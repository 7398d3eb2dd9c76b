// tokens.hip -- tokens sorted by expert and back, in the tensors' own type
// (binary32, bf16 or fp16), with the router weights applied and the gradients
// of both.  With r = dst_row[t, j] the row of entry (t, j):
//   spread   rows[r] = w[t, j] tok[t]                (sort; unsort's gradient)
//            dw[t, j] = sum_h tok[t, h] given[r, h]  (unsort's weight gradient)
//   collect  tok[t] = sum_j w[t, j] rows[r]          (unsort; sort's gradient)
//            dw[t, j] = sum_h rows[r, h] given[t, h] (sort's weight gradient)
// Products and sums are binary32 (j ascending; a dot product's order is fixed
// by the launch), rounded once to the tensors' type.  Entries with dst_row
// outside [0, rows) move nothing and have a zero weight gradient.
//
// Bound: HBM.  A token's row is read once and its k rows written (or read)
// once, so a workgroup takes a whole token: its threads hold 16-byte pieces
// of the row and loop over the entries, eight of whose loads are issued before
// the first is used.  The weight gradient is taken on the way from the same
// registers, up to eight entries a token; sort's gradient with more reads the
// rows of entries 8, 9, ... and the token's own row once more for it (bf16, 8192
// tokens of 512, top-12: 34.5 us).  Rows move by non-temporal loads and stores: each is touched once
// per launch, and ordinary stores of 4 KiB rows scattered over the experts
// ran at 2.9 TB/s.  Measured (bf16, hidden 2048, top-8, interleaved): sorting
// 8192 tokens 104.3 -> 53.9 us (5.6 TB/s), unsorting them 89.4 -> 59.9 us,
// sort then unsort at 64 ... 16384 tokens 10.7 -> 8.1 ... 382 -> 220 us,
// unsort's gradient of 32768 tokens 712 -> 430 us (5.3 TB/s).
#include "elem.h"
#include "launch.h"

namespace nvfp4 {

namespace {

constexpr int kBatch = 8;   // entries whose rows are in flight together

// Sums of n <= kBatch values over the workgroup: thread j < n gets the j-th.
// (Every thread adding up every sum took 14.4 us instead of 10.9 for the gradient
// of a sort of 64 tokens of 7168, top-8, whose workgroups have 14 waves.)
// The thread's number is made opaque, so that its lane, addresses and comparisons
// are not kept in registers through the columns' loop: the collect then runs five
// waves a SIMD instead of four (32768 tokens of 512, top-8: 62.6 against 68.5 us;
// of 500, top-4: 46.2 against 50.6).
__device__ __forceinline__ float block_sums(const float (&v)[kBatch], int n, float* lds) {
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid % kWave, wave = tid / kWave;
  const int waves = blockDim.x / kWave;
  int own = 0;
#pragma unroll
  for (int j = 0; j < kBatch; ++j) {
    if (j < n) {
      const uint32_t s = wave_incl_scan_dpp(
          __float_as_uint(v[j]), [](uint32_t a, uint32_t b) {
            return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
          });
      const int total = __builtin_amdgcn_readlane((int)s, kWave - 1);
      own = lane == j ? total : own;
    }
  }
  float sum = __int_as_float(own);
  if (waves == 1) return sum;
  __syncthreads();   // the previous batch's sums have been read
  if (lane < kBatch) lds[wave * kBatch + lane] = sum;
  __syncthreads();
  if (tid < n) {
    sum = lds[tid];
    for (int w = 1; w < waves; ++w) sum += lds[w * kBatch + tid];
  }
  return sum;
}

// A thread's piece [c, c + kN) of a row, brought back inside the row: a last,
// partial piece becomes the row's last kN elements, its first `skip` of which
// another thread holds too (both write the same values; dot products leave
// them out).  Rows shorter than a piece are taken element by element.
template <int N>
struct Span {
  int64_t at;
  int skip, part;   // part: 0, or the elements of a row shorter than a piece
  __device__ __forceinline__ Span(int64_t c, int64_t hidden)
      : at(c + N <= hidden || hidden < N ? c : hidden - N), skip((int)(c - at)),
        part(hidden < N ? (int)hidden : 0) {}
};
template <int DT>
__device__ __forceinline__ void load_span(Piece<DT>& p, const typename Piece<DT>::T* row,
                                          const Span<Piece<DT>::kN>& s, bool once) {
  if (s.part) p.load_part(row, s.part);
  else if (once) p.load_once(row + s.at);
  else p.load(row + s.at);
}
template <int DT>
__device__ __forceinline__ void store_span(const Piece<DT>& p, typename Piece<DT>::T* row,
                                           const Span<Piece<DT>::kN>& s) {
  if (s.part) p.store_part(row, s.part);
  else p.store(row + s.at);
}
// dot += x . y over the piece's own elements
template <int DT>
__device__ __forceinline__ void dot_span(float& dot, const Piece<DT>& x, const Piece<DT>& y,
                                         const Span<Piece<DT>::kN>& s) {
#pragma unroll
  for (int i = 0; i < Piece<DT>::kN; ++i) {
    const float v = x.get(i) * y.get(i);
    dot += i >= s.skip ? v : 0.0f;
  }
}

// Row of entry (t, j), -1 if it has none.
__device__ __forceinline__ int64_t entry_row(const TokenRowsArgs& a, int64_t t, int j) {
  const int32_t r = a.dst_row[t * a.topk + j];
  return r >= 0 && r < a.rows_cap ? r : -1;
}

// Rows (-1 for none) and weights of entries [j0, j0 + kBatch) of token t, those
// past the last included: all loads are issued before the first is looked at.
// The collect takes its entries so, once per token instead of once per column
// step: 9.8 against 11.1 us at 1003 tokens of 1111, 8.05 against 8.55 at 256 of
// 2048. The spread does not (444 against 436 us at 32768 tokens of 2048): its
// time is traffic, and it looks at a token's entries only once anyway.
template <bool WEIGHTED>
__device__ __forceinline__ void load_entries(const TokenRowsArgs& a, int64_t t, int j0,
                                             int64_t (&row)[kBatch], float (&w)[kBatch]) {
  int32_t r[kBatch];
#pragma unroll
  for (int j = 0; j < kBatch; ++j) {
    const int64_t i = t * a.topk + (j0 + j < a.topk ? j0 + j : a.topk - 1);
    r[j] = a.dst_row[i];
    w[j] = WEIGHTED ? a.prob[i] : 1.0f;
  }
#pragma unroll
  for (int j = 0; j < kBatch; ++j)
    row[j] = j0 + j < a.topk && r[j] >= 0 && r[j] < a.rows_cap ? r[j] : -1;
}

}  // namespace

// Spread: blocks [0, token_blocks) take tokens, the rest zero the padding
// rows (row_src < 0) inside the experts' segments, `pad_rows` rows each.
template <int DT, bool WEIGHTED, bool DOT>
__global__ __launch_bounds__(256) void spread_kernel(TokenRowsArgs a, int64_t token_blocks,
                                                     int pad_rows) {
  typedef typename Elem<DT>::type T;
  typedef Piece<DT> P;
  __shared__ float sums[4 * kBatch];
  T* rows = static_cast<T*>(a.rows_out);
  if ((int64_t)blockIdx.x >= token_blocks) {
    const int64_t end = *a.rows_end < a.rows_cap ? *a.rows_end : a.rows_cap;
    const int64_t r0 = (int64_t)(blockIdx.x - token_blocks) * pad_rows;
    const int64_t r1 = r0 + pad_rows < end ? r0 + pad_rows : end;
    P zero;
    zero.load_part(rows, 0);
    for (int64_t b = r0; b < r1; b += kWave) {
      // every wave takes the same ballot, so the workgroup clears each row together
      const int64_t r = b + threadIdx.x % kWave;
      const bool pad = r < r1 && a.row_src[r] < 0;
      for (uint64_t m = __ballot(pad); m != 0; m &= m - 1) {
        T* row = rows + (b + __builtin_ctzll(m)) * a.hidden;
        for (int64_t c = (int64_t)threadIdx.x * P::kN; c < a.hidden; c += (int64_t)blockDim.x * P::kN)
          store_span<DT>(zero, row, Span<P::kN>(c, a.hidden));
      }
    }
    return;
  }
  for (int64_t t = blockIdx.x; t < a.tokens; t += token_blocks) {
    const T* tok = static_cast<const T*>(a.tok) + t * a.ld_tok;
    for (int j0 = 0; j0 < a.topk; j0 += kBatch) {
      const int n = a.topk - j0 < kBatch ? a.topk - j0 : kBatch;
      int64_t row[kBatch];
      float w[kBatch], dot[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        row[j] = j < n ? entry_row(a, t, j0 + j) : -1;
        w[j] = WEIGHTED && row[j] >= 0 ? a.prob[t * a.topk + j0 + j] : 1.0f;
        dot[j] = 0.0f;
      }
      for (int64_t c = (int64_t)threadIdx.x * P::kN; c < a.hidden; c += (int64_t)blockDim.x * P::kN) {
        const Span<P::kN> span(c, a.hidden);
        P x;
        load_span<DT>(x, tok, span, false);
        P g[DOT ? kBatch : 1];
        if (DOT) {
#pragma unroll
          for (int j = 0; j < kBatch; ++j)
            if (row[j] >= 0)
              load_span<DT>(g[DOT ? j : 0], static_cast<const T*>(a.given) + row[j] * a.ld_given, span,
                            true);
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          if (row[j] < 0) continue;
          P o = x;
          if (WEIGHTED) {
#pragma unroll
            for (int i = 0; i < P::kN; ++i) o.set(i, x.get(i) * w[j]);
          }
          store_span<DT>(o, rows + row[j] * a.hidden, span);
          if (DOT) dot_span<DT>(dot[j], x, g[DOT ? j : 0], span);
        }
      }
      if (DOT) {
        // (an entry without a row has added nothing: 0)
        const float dw = block_sums(dot, n, sums);
        if ((int)threadIdx.x < n) a.dprob[t * a.topk + j0 + threadIdx.x] = dw;
      }
    }
  }
}

template <int DT, bool WEIGHTED, bool DOT>
__global__ __launch_bounds__(1024) void collect_kernel(TokenRowsArgs a) {
  typedef typename Elem<DT>::type T;
  typedef Piece<DT> P;
  __shared__ float sums[16 * kBatch];
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    T* out = static_cast<T*>(a.tok_out) + t * a.hidden;
    const T* given = DOT ? static_cast<const T*>(a.given) + t * a.ld_given : nullptr;
    // Columns outermost while one batch holds every entry; with more entries
    // the dot products need the entries outermost, so the column's sum is
    // then taken over the batches in an inner loop of its own.
    for (int j0 = 0; j0 < (DOT ? a.topk : 1); j0 += kBatch) {
      int64_t row0[kBatch];
      float w0[kBatch], dot[kBatch];
      load_entries<WEIGHTED>(a, t, j0, row0, w0);
#pragma unroll
      for (int j = 0; j < kBatch; ++j) dot[j] = 0.0f;
      for (int64_t c = (int64_t)threadIdx.x * P::kN; c < a.hidden; c += (int64_t)blockDim.x * P::kN) {
        const Span<P::kN> span(c, a.hidden);
        float sum[P::kN];
#pragma unroll
        for (int i = 0; i < P::kN; ++i) sum[i] = 0.0f;
        P x;
        if (DOT) load_span<DT>(x, given, span, false);
        // the first pass over the columns takes every entry into the sum,
        // a later one (topk > kBatch) only its own entries' dot products
        const int last = j0 == 0 ? a.topk : (j0 + kBatch < a.topk ? j0 + kBatch : a.topk);
        for (int b = j0; b < last; b += kBatch) {
          P p[kBatch];
          int64_t row[kBatch];
          float w[kBatch];
          if (b == j0) {
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
              row[j] = row0[j];
              w[j] = w0[j];
            }
          } else {
            load_entries<WEIGHTED>(a, t, b, row, w);
          }
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            if (row[j] < 0) continue;
            load_span<DT>(p[j], static_cast<const T*>(a.rows) + row[j] * a.ld_rows, span, true);
          }
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            if (row[j] < 0) continue;
            if (j0 == 0) {
#pragma unroll
              for (int i = 0; i < P::kN; ++i)
                sum[i] += WEIGHTED ? w[j] * p[j].get(i) : p[j].get(i);
            }
            if (DOT && b == j0) dot_span<DT>(dot[j], x, p[j], span);
          }
        }
        if (j0 == 0) {
          P o;
#pragma unroll
          for (int i = 0; i < P::kN; ++i) o.set(i, sum[i]);
          store_span<DT>(o, out, span);
        }
      }
      if (DOT) {
        const int n = a.topk - j0 < kBatch ? a.topk - j0 : kBatch;
        // (an entry without a row has added nothing: 0)
        const float dw = block_sums(dot, n, sums);
        if ((int)threadIdx.x < n) a.dprob[t * a.topk + j0 + threadIdx.x] = dw;
      }
    }
  }
}

namespace {

// Threads of a token's workgroup: one 16-byte piece each while `most` reach,
// then an even share.
int token_threads(int64_t hidden, int dtype, int64_t most) {
  const int64_t pieces = (hidden * (dtype == 0 ? 4 : 2) + 15) / 16;
  const int64_t steps = (pieces + most - 1) / most;
  return (int)(((pieces + steps - 1) / steps + 63) / 64 * 64);
}
// (blocks x threads stays far below 2^32; larger batches loop)
int64_t token_grid(int64_t tokens) { return tokens < (1 << 22) ? tokens : (1 << 22); }

}  // namespace

#define NVFP4_TOKENS_CASE(D, LAUNCH)             \
  case 4 * D: LAUNCH(D, false, false); break;    \
  case 4 * D + 1: LAUNCH(D, false, true); break; \
  case 4 * D + 2: LAUNCH(D, true, false); break; \
  case 4 * D + 3: LAUNCH(D, true, true); break;

hipError_t launch_spread(const TokenRowsArgs& a, hipStream_t s) {
  const int threads = token_threads(a.hidden, a.dtype, 256);
  const int64_t tb = token_grid(a.tokens);
  // Padding is looked for in every row: arrays with more rows than entries
  // (align > 1) hold it throughout, 8 rows a block; others may hold some only
  // where entries were dropped and the arrays cut to fit.  More than 2^21
  // blocks take more rows each.
  int64_t pad_rows = a.rows_cap > a.tokens * a.topk ? 8 : 512;
  while (a.rows_cap / pad_rows >= 1 << 21) pad_rows *= 2;
  const int64_t pad = (a.rows_cap + pad_rows - 1) / pad_rows;
  if (tb + pad == 0) return hipSuccess;
#define NVFP4_SPREAD(D, W, G) \
  spread_kernel<D, W, G><<<(unsigned)(tb + pad), threads, 0, s>>>(a, tb, (int)pad_rows)
  switch (a.dtype * 4 + (a.prob ? 2 : 0) + (a.dprob ? 1 : 0)) {
    NVFP4_TOKENS_CASE(0, NVFP4_SPREAD)
    NVFP4_TOKENS_CASE(1, NVFP4_SPREAD)
    NVFP4_TOKENS_CASE(2, NVFP4_SPREAD)
  }
#undef NVFP4_SPREAD
  return hipGetLastError();
}

hipError_t launch_collect(const TokenRowsArgs& a, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
  // Where every token can have a CU, its whole row is taken at once: bf16, 7168
  // columns, top-8: 64 tokens 9.5 us, 18.9 with 256 threads; 256 tokens 11.3 /
  // 20.4; 1024 tokens 35.0 / 31.3 (the spread gains nothing: 8.9 / 8.2 at 256).
  const int threads = token_threads(a.hidden, a.dtype, a.tokens <= 256 ? 1024 : 256);
  const unsigned blocks = (unsigned)token_grid(a.tokens);
#define NVFP4_COLLECT(D, W, G) collect_kernel<D, W, G><<<blocks, threads, 0, s>>>(a)
  switch (a.dtype * 4 + (a.prob ? 2 : 0) + (a.dprob ? 1 : 0)) {
    NVFP4_TOKENS_CASE(0, NVFP4_COLLECT)
    NVFP4_TOKENS_CASE(1, NVFP4_COLLECT)
    NVFP4_TOKENS_CASE(2, NVFP4_COLLECT)
  }
#undef NVFP4_COLLECT
  return hipGetLastError();
}

#undef NVFP4_TOKENS_CASE

}  // namespace nvfp4
