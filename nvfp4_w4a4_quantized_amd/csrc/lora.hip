// lora.hip -- low-rank adapters of many requests beside a shared projection:
//   h[t] = A[s] x[t]          y[t] = base[t] + c_s B[s] h[t]        s = ids[t]
// and their gradients, with g[t] = c_s B[s]^T dy[t]:
//   dx[t] = base[t] + A[s]^T g[t]
//   dA[s] = sum over s's tokens of g[t] x[t]^T,  dB[s] = of c_s dy[t] h[t]^T
// A token whose id is no adapter has h = 0 and y = base.
//
// Both directions are the same two products: "down" contracts a long row with
// the rank's rows ([S, R, K], K contiguous), "up" multiplies R values into a
// long row ([S, N, R], R contiguous).  The way back takes B and A transposed,
// by a copy of them (the adapters are small beside the tokens).
//
// Tokens of one adapter are multiplied together.  Few tokens (up to kWindow):
// a workgroup per token looks its adapter's tokens up and the first of them
// does the work of all, 16 at a time (which costs many tokens of few adapters
// dear: 2048 -> 5120 of rank 16, one adapter, 64 tokens 23 us, 256 tokens 156, 257
// tokens 14).  Many: a workgroup takes consecutive tokens (16 to 64 down,
// 32 up) and does one adapter after the other, each keeping the results of its own
// tokens, so a batch whose requests lie together reads each token's row once and
// an adapter once per workgroup.
//
// Arithmetic: down multiplies in the type of x by MFMA 16x16x32 (binary32:
// 16x16x4) into binary32; h and g stay binary32.  What they enter are binary32
// products: of bf16 B, A, x and dy with the three bf16 parts of the binary32
// value (MFMA 16x16x32), else MFMA 16x16x4 of the exactly widened values.  Sums over K that several workgroups share are joined in workgroup
// order, sums over tokens in token order per chunk: results do not depend on
// timing.
//
// Bound: the long rows' bytes.  Measured (bf16): down 8192 x 5120 of rank 16 21 us
// (3.9 TB/s), 32768 x 5120 of rank 64 95 us (3.5 TB/s); up 4096 x 5120 with a base 27
// us (3.1 TB/s), 8192 x 2048 22 us (3.0), 32768 x 2048 of rank 64 83 us (3.4);
// gradients of 8192 tokens of rank 16 37 us (3.2 TB/s), of 32768 of rank 64 216 us
// (2.2 TB/s: vector instructions issue 26 % of the time, matrix cores 17 %, LDS bank
// conflicts 9 %; none is at its limit).  One token's 64 KB of A and 160 KB of B take
// 7 us, most of it latency.
#include <type_traits>

#include "elem.h"
#include "launch.h"

namespace nvfp4 {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kWindow = 256;    // most tokens that workgroups per token look through
constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;
constexpr int kRanks = 64;      // ranks of one pass
constexpr int kMostShares = 8;  // of K

// ---- the tokens of one adapter ------------------------------------------

__device__ __forceinline__ int key_of(int id, int adapters) {
  return id >= 0 && id < adapters ? id : -1;
}

__device__ __forceinline__ int bits_below(uint64_t mask) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                   __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
}

struct TokenList {
  uint16_t at[kWindow];
  uint64_t mask[kWaves];
};

// The tokens (up to kWindow in all) that share token `slot`'s adapter, into
// list.at in ascending order; returns their number, 0 if the slot is not the
// first of them.
__device__ __forceinline__ int tokens_like(const int32_t* ids, int tokens, int adapters, int slot,
                                           TokenList& list, int* adapter) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int key = key_of(ids[slot], adapters);
  const bool in = (int)threadIdx.x < tokens;
  const bool mine = in && key_of(ids[in ? threadIdx.x : 0], adapters) == key;
  const uint64_t mask = __ballot(mine);
  if (lane == 0) list.mask[wave] = mask;
  __syncthreads();
  int m = 0, before = 0;
  bool earlier = false;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const uint64_t b = list.mask[w];
    if (w < wave) before += __popcll(b);
    m += __popcll(b);
    const int to = slot - w * kWave;      // tokens of this wave before the slot
    if (to > 0) earlier |= (to >= kWave ? b : b & ((1ull << to) - 1)) != 0;
  }
  if (mine && !earlier) list.at[before + bits_below(mask)] = (uint16_t)threadIdx.x;
  __syncthreads();
  *adapter = key;
  return earlier ? 0 : m;
}

// Lane l's key among 64 consecutive tokens: the adapter, -1 without, -2 past the last.
__device__ __forceinline__ int key_at(const int32_t* ids, int64_t tokens, int adapters, int64_t t) {
  return t < tokens ? key_of(ids[t], adapters) : -2;
}

// ---- down: the long rows' products with the rank's rows --------------------

// 16 bytes of a row from element `at`, zeros from element `end` on.
template <int DT>
__device__ __forceinline__ Piece<DT> piece_until(const typename Elem<DT>::type* row, int64_t at,
                                                 int64_t end) {
  Piece<DT> p;
  if (at + Piece<DT>::kN <= end) p.load(row + at);
  else p.load_part(row + at, at < end ? (int)(end - at) : 0);
  return p;
}

template <int DT>
__device__ __forceinline__ f32x4_t product(const Piece<DT>& a, const Piece<DT>& b, f32x4_t acc) {
  if constexpr (DT == 0) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[e], b.v[e], acc, 0, 0, 0);
    return acc;
  } else if constexpr (DT == 1) {
    bf16x8_t u, v;
    __builtin_memcpy(&u, a.v, 16);
    __builtin_memcpy(&v, b.v, 16);
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(u, v, acc, 0, 0, 0);
  } else {
    half8_t u, v;
    __builtin_memcpy(&u, a.v, 16);
    __builtin_memcpy(&v, b.v, 16);
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(u, v, acc, 0, 0, 0);
  }
}

// acc[rt][j] += ranks' rows ar[rt] times tokens' rows xr[j] over [k0, k1), a
// wave's share of it: every fourth 128-byte piece.  Lane l has bytes 16 (l / 16)
// of each 64 of its rows.
template <int DT, int RT, int TT>
__device__ __forceinline__ void down_products(const typename Elem<DT>::type* const (&ar)[RT],
                                              const typename Elem<DT>::type* const (&xr)[TT],
                                              int64_t k0, int64_t k1, int wave, int q,
                                              f32x4_t (&acc)[RT][TT]) {
  constexpr int E = Piece<DT>::kN, kStep = 8 * E;   // elements of a piece; of 128 bytes
  int64_t c = k0 + wave * kStep;
  // whole pieces without a branch, so that their loads are in flight together
  for (; c + kStep <= k1; c += kWaves * kStep) {
    Piece<DT> a[2][RT], x[2][TT];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int j = 0; j < TT; ++j) x[u][j].load(xr[j] + c + (4 * u + q) * E);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) a[u][rt].load(ar[rt] + c + (4 * u + q) * E);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int j = 0; j < TT; ++j) acc[rt][j] = product<DT>(a[u][rt], x[u][j], acc[rt][j]);
  }
  if (c < k1) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t at = c + (4 * u + q) * E;
      Piece<DT> a[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) a[rt] = piece_until<DT>(ar[rt], at, k1);
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        const Piece<DT> x = piece_until<DT>(xr[j], at, k1);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) acc[rt][j] = product<DT>(a[rt], x, acc[rt][j]);
      }
    }
  }
}

// Grid: x = tokens (SLOT) or groups of 16 TT tokens, y = shares of K, z = 64
// ranks each.  Position p of a group is token list.at[g0 + p] (SLOT) or first + p.
template <int DT, int RT, int TT, bool SLOT>
__global__ __launch_bounds__(kThreads) void lora_down_kernel(LoraDownArgs p) {
  typedef typename Elem<DT>::type T;
  __shared__ TokenList list;
  __shared__ f32x4_t red[kWaves][TT][kWave];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int i = lane % 16, q = lane / 16;
  const int r0 = blockIdx.z * kRanks;
  const int64_t k0 = blockIdx.y * p.share, k1 = k0 + p.share < p.k ? k0 + p.share : p.k;
  float* const out = p.h + blockIdx.y * p.tokens * p.rank;
  const T* const x = static_cast<const T*>(p.x);
  auto one = [&](int s, const T* const (&xr)[TT], auto keep) {
    f32x4_t acc[RT][TT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int j = 0; j < TT; ++j) acc[rt][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
    if (s >= 0) {
      const T* ar[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int r = r0 + 16 * rt + i;
        ar[rt] = static_cast<const T*>(p.a) + ((int64_t)s * p.rank + (r < p.rank ? r : p.rank - 1)) * p.k;
      }
      down_products<DT, RT, TT>(ar, xr, k0, k1, wave, q, acc);
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < TT; ++j) red[wave][j][lane] = acc[rt][j];
      __syncthreads();
      if (wave >= TT) continue;
      f32x4_t v = red[0][wave % TT][lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += red[w][wave % TT][lane];
      const int r = r0 + 16 * rt + 4 * q;
      const int64_t tok = keep(16 * wave + i);
      if (tok < 0) continue;
      float* o = out + tok * p.rank + r;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (r + e < p.rank) o[e] = v[e];
    }
  };
  if constexpr (SLOT) {
    int s;
    const int m = tokens_like(p.ids, (int)p.tokens, p.adapters, blockIdx.x, list, &s);
    for (int g0 = 0; g0 < m; g0 += 16) {
      const T* xr[1] = {x + list.at[g0 + i < m ? g0 + i : g0] * p.ld_x};
      one(s, xr, [&](int at) -> int64_t { return g0 + at < m ? list.at[g0 + at] : -1; });
    }
  } else {
    const int64_t first = (int64_t)blockIdx.x * (16 * TT);
    const int key = lane < 16 * TT ? key_at(p.ids, p.tokens, p.adapters, first + lane) : -2;
    uint64_t todo = __ballot(key != -2);
    while (todo != 0) {
      const int lead = __builtin_ctzll(todo), s = __shfl(key, lead);
      const uint64_t mask = __ballot(key == s);
      // (other adapters' columns take the first token's row: no more is read)
      const T* xr[TT];
#pragma unroll
      for (int j = 0; j < TT; ++j)
        xr[j] = x + (first + ((mask >> (16 * j + i)) & 1 ? 16 * j + i : lead)) * p.ld_x;
      one(s, xr, [&](int at) -> int64_t { return (mask >> at) & 1 ? first + at : -1; });
      todo &= ~mask;
    }
  }
}

// ---- up: the rank's values into long rows ----------------------------------

// The three bf16 parts of a binary32 value: the upper half of its bits, of what
// is left of it, and the rest.  The lower parts of an infinity are the largest
// finite value's: they add to it with its sign.  A lower part that is zero holds
// 2^-32 of the value instead, and so does the returned fourth one, which stands
// where the operands repeat beside nothing: an infinity of the other operand times
// each part has the sign of its product with the value (NaN if that is zero).  The
// parts' sum is the value to 2^-30 of it, far below the binary32 sums that it enters.
__device__ __forceinline__ uint16_t bf16_parts(float v, uint16_t (&part)[3]) {
  part[0] = (uint16_t)(__float_as_uint(v) >> 16);
  v = __builtin_amdgcn_fmed3f(v, -__FLT_MAX__, __FLT_MAX__);
  const float least = v * 0x1p-32f;
#pragma unroll
  for (int i = 1; i < 3; ++i) {
    v -= __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
    part[i] = (uint16_t)(__float_as_uint(v == 0.0f ? least : v) >> 16);
  }
  return (uint16_t)(__float_as_uint(least) >> 16);
}

// c h of up to TOK tokens and PASS ranks, as the products' operand.  bf16: a step
// is 32 k of one MFMA, tokens' rows of 64 bytes (16-byte chunk k of row t at
// k ^ (t / 4) % 4).  Up to 16 ranks take two steps, the first two parts beside
// each other and the third beside the fourth; more take three, a part each, per 32
// ranks.  Else: rows of binary32.
template <int DT, int TOK, int PASS>
struct Ranked {
  static constexpr int kLd = PASS + 4;
  union {
    uint16_t part[DT == 1 ? 3 * TOK * PASS : 8];
    float row[DT == 1 ? 4 : TOK * kLd];
  };
  static __device__ __forceinline__ int at(int step, int t, int k) {
    return (step * TOK + t) * 32 + 8 * ((k / 8) ^ ((t >> 2) & 3)) + k % 8;
  }
  __device__ __forceinline__ void put(int t, int r, bool narrow, float v) {
    if constexpr (DT == 1) {
      uint16_t b[3];
      const uint16_t least = bf16_parts(v, b);
      if (narrow) {
        part[at(0, t, r)] = b[0];
        part[at(0, t, 16 + r)] = b[1];
        part[at(1, t, r)] = b[2];
        part[at(1, t, 16 + r)] = least;
      } else {
#pragma unroll
        for (int i = 0; i < 3; ++i) part[at(r / 32 * 3 + i, t, r % 32)] = b[i];
      }
    } else {
      row[t * kLd + r] = v;
    }
  }
};

// The rows' values of B from rank r on: 8 of bf16, 4 of the others.
template <int DT>
struct RankPiece {
  static constexpr int kN = DT == 1 ? 8 : 4;
  typename Elem<DT>::type v[kN];
  __device__ __forceinline__ void load(const typename Elem<DT>::type* row, int r, int end) {
    if (r + kN <= end) {
      __builtin_memcpy(v, row + r, sizeof(v));
    } else {
#pragma unroll
      for (int e = 0; e < kN; ++e) v[e] = r + e < end ? row[r + e] : (typename Elem<DT>::type)0;
    }
  }
  // end a multiple of kN: zeros from there on
  __device__ __forceinline__ void load_whole(const typename Elem<DT>::type* row, int r, int end) {
    const bool in = r < end;
    __builtin_memcpy(v, row + (in ? r : 0), sizeof(v));
    uint32_t w[sizeof(v) / 4];
    __builtin_memcpy(w, v, sizeof(v));
#pragma unroll
    for (uint32_t& x : w) x = in ? x : 0u;
    __builtin_memcpy(v, w, sizeof(v));
  }
};

// N values from `at` on, `left` of them inside (zeros behind).
template <int DT, int N>
__device__ __forceinline__ void get_some(const void* from, int64_t at, int64_t left, float (&v)[N]) {
  typedef typename Elem<DT>::type T;
  const T* b = static_cast<const T*>(from) + at;
  T x[N];
  if (left >= N) {
    __builtin_memcpy(x, b, sizeof(x));
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = e < left ? b[e] : (T)0;
  }
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = Elem<DT>::to_float(x[e]);
}

// Grid: x = tokens (SLOT) or groups of 16 TT tokens, y = p.wide columns each, 64
// a wave at a time.  Which of the wave's 64 columns is row i of product j is chosen
// so that a lane ends with 16-byte pieces of its token, and a load or store covers
// 64 consecutive bytes of every token (32 bytes a lane, in two halves of 16 each,
// cost 4096 x 5120 29.6 us instead of 27.4).  Beyond kWindow tokens the three waves a SIMD
// leave registers in scratch, 8 to 154 of them, in every form of fp16, of binary32 with a
// base or any width, and of bf16 into binary32 of any width.
// The sums start from the base's values, which are loaded a turn ahead.  BIG:
// more than 32 ranks, 64 at a time.  WHOLE: whole pieces everywhere and the kind of
// base known, so that no branch stands around a load (the compiler waits for every
// load in flight where its paths join).  DIRECT: each workgroup computes h itself, the
// whole of A[s] x, so that a few tokens take one launch.
enum { kAny = 0, kNoBase = 1, kSameBase = 2, kWideBase = 3 };    // kWideBase: binary32
template <int DT, int OT, int TT, bool SLOT, bool BIG, bool DIRECT, int WHOLE>
__global__ __launch_bounds__(kThreads, BIG ? 2 : 3) void lora_up_kernel(LoraUpArgs p) {
  typedef typename Elem<DT>::type T;
  typedef typename Elem<OT>::type O;
  constexpr int TOK = 16 * TT;
  constexpr int kPass = BIG ? kRanks : 32, kPieces = kPass / (DT == 1 ? 32 : 16);
  constexpr int kN = Piece<OT>::kN, kBase = 16 / kN;     // columns of a piece, pieces of a lane
  __shared__ TokenList list;
  __shared__ __align__(16) Ranked<DT, TOK, kPass> hs;
  __shared__ f32x4_t red[DIRECT ? kWaves : 1][2][kWave];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int i = lane % 16, q = lane / 16;
  const int64_t first = SLOT ? 0 : (int64_t)blockIdx.x * TOK;
  const int64_t w0 = (int64_t)blockIdx.y * p.wide, n_end = w0 + p.wide < p.n ? w0 + p.wide : p.n;
  int s = -1, m = TOK, key = -2;
  if constexpr (SLOT) {
    m = tokens_like(p.ids, (int)p.tokens, p.adapters, blockIdx.x, list, &s);
  } else {
    key = lane < TOK ? key_at(p.ids, p.tokens, p.adapters, first + lane) : -2;
  }
  const bool narrow = !BIG && p.rank <= 16;
  const uint64_t here = SLOT ? 0 : __ballot(key != -2);

  for (int g0 = 0; g0 < m; g0 += TOK) {
    const uint64_t in = SLOT ? (m - g0 >= TOK ? (1ull << (TOK % 64)) - 1 : (1ull << (m - g0)) - 1) : here;
    auto token = [&](int at) -> int64_t { return SLOT ? list.at[g0 + at] : first + at; };

    // c h of the group's tokens, ranks r0 and on: four of a token's ranks a
    // thread, its shares in flight together and added in order
    auto fetch_h = [&](int v, int r0, int padded, float (&h)[kMostShares][4]) {
      const int t = v / (padded / 4), r = 4 * (v % (padded / 4));
      const int ranks = p.rank - r0 < kPass ? p.rank - r0 : kPass;
      const bool live = t < TOK && r < ranks && (SLOT ? g0 + t < m : first + t < p.tokens);
      const float* from = p.h + (live ? token(t) * p.rank + r0 + r : 0);
      const int64_t step = p.tokens * p.rank;
      if (WHOLE != kAny || p.rank % 4 == 0) {
#pragma unroll
        for (int w = 0; w < kMostShares; ++w) __builtin_memcpy(h[w], from + (w < p.shares ? w * step : 0), 16);
      } else {
#pragma unroll
        for (int w = 0; w < kMostShares; ++w)
#pragma unroll
          for (int e = 0; e < 4; ++e) h[w][e] = w < p.shares && live && r + e < ranks ? from[w * step + e] : 0.0f;
      }
    };
    auto put_h = [&](int v, int r0, int padded, const float (&h)[kMostShares][4]) {
      const int t = v / (padded / 4), r = 4 * (v % (padded / 4));
      const int ranks = p.rank - r0 < kPass ? p.rank - r0 : kPass;
      const bool live = t < TOK && r < ranks && (in >> (t & 63)) & 1;
      const int a = SLOT ? s : __shfl(key, t & 63);
      const float c = a >= 0 && p.scale ? p.scale[a] : 1.0f;
      float f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[e] = h[0][e];
#pragma unroll
        for (int w = 1; w < kMostShares; ++w) f[e] = w < p.shares ? f[e] + h[w][e] : f[e];
        if (!live || a < 0) f[e] = 0.0f;
      }
      if (live && p.h_out && blockIdx.y == 0) {
        float* to = p.h_out + token(t) * p.rank + r0 + r;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (r + e < ranks) to[e] = p.h_scaled ? c * f[e] : f[e];
      }
      if (t < TOK) {
        // (ranks past the last stay zero whatever the scale is)
#pragma unroll
        for (int e = 0; e < 4; ++e) hs.put(t, r + e, narrow, live && a >= 0 && r + e < ranks ? c * f[e] : 0.0f);
      }
    };
    auto padded_ranks = [&](int r0) -> int {
      const int ranks = p.rank - r0 < kPass ? p.rank - r0 : kPass;
      return DT == 1 ? (narrow ? 16 : (ranks + 31) / 32 * 32) : (ranks + 15) / 16 * 16;
    };
    auto stage = [&](int r0) {
      const int padded = padded_ranks(r0);
      // (every thread takes every turn: put_h exchanges values in the wave)
      for (int v = threadIdx.x; v - (int)threadIdx.x < TOK * padded / 4; v += kThreads) {
        float h[kMostShares][4];
        fetch_h(v, r0, padded, h);
        put_h(v, r0, padded, h);
      }
    };
    // the same from x: every wave a share of K, added in wave order
    auto stage_x = [&](auto rt_c) {
      constexpr int RT = decltype(rt_c)::value;
      f32x4_t acc[RT][1];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) acc[rt][0] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
      if (s >= 0) {
        const T* xr[1] = {static_cast<const T*>(p.x) + token((in >> i) & 1 ? i : 0) * p.ld_x};
        const T* ar[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const int r = 16 * rt + i;
          ar[rt] = static_cast<const T*>(p.a) + ((int64_t)s * p.rank + (r < p.rank ? r : p.rank - 1)) * p.k;
        }
        down_products<DT, RT, 1>(ar, xr, 0, p.k, wave, q, acc);
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) red[wave][rt][lane] = acc[rt][0];
      __syncthreads();
      if (wave < RT) {
        f32x4_t v = red[0][wave % 2][lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += red[w][wave % 2][lane];
        const float c = s >= 0 && p.scale ? p.scale[s] : 1.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 16 * wave + 4 * q + e;
          const bool live = r < p.rank && (in >> i) & 1;
          if (live && p.h_out && blockIdx.y == 0) p.h_out[token(i) * p.rank + r] = v[e];
          hs.put(i, r, narrow, live ? c * v[e] : 0.0f);
        }
      }
    };
    auto load_b = [&](int adapter, int64_t n0, int j, int r0, RankPiece<DT> (&b)[kPieces]) {
      const int64_t n = n0 + (kN == 8 ? 32 * (j / 2) + 8 * (i / 4) + 4 * (j % 2) + i % 4 : 16 * j + i);
      const T* row = static_cast<const T*>(p.b) + ((int64_t)adapter * p.n + (n < p.n ? n : p.n - 1)) * p.rank;
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int r = r0 + (DT == 1 ? (narrow ? 8 * (q % 2) : 32 * k + 8 * q) : 16 * k + 4 * q);
        if constexpr (WHOLE != kAny) b[k].load_whole(row, r, p.rank);
        else if ((DT == 1 ? 32 : 16) * k < p.rank - r0) b[k].load(row, r, p.rank);
      }
    };
    // acc[j][t] += B h for the products [J, J + JN)
    auto products = [&](const RankPiece<DT>* b, int r0, auto jn_c, f32x4_t (*acc)[TT]) {
      constexpr int JN = decltype(jn_c)::value;
      const int ranks = p.rank - r0 < kPass ? p.rank - r0 : kPass;
      if constexpr (DT == 1) {
        const int steps = narrow ? 2 : (ranks + 31) / 32 * 3;
#pragma unroll
        for (int st = 0; st < 3 * kPieces; ++st) {
          if (st >= steps) continue;
#pragma unroll
          for (int t = 0; t < TT; ++t) {
            const bf16x8_t h = *reinterpret_cast<const bf16x8_t*>(hs.part + Ranked<DT, TOK, kPass>::at(st, 16 * t + i, 8 * q));
#pragma unroll
            for (int j = 0; j < JN; ++j) {
              bf16x8_t u;
              __builtin_memcpy(&u, b[j * kPieces + st / 3].v, 16);
              acc[j][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(u, h, acc[j][t], 0, 0, 0);
            }
          }
        }
      } else {
#pragma unroll
        for (int rb = 0; rb < kPieces; ++rb) {
          if (16 * rb >= ranks) continue;
#pragma unroll
          for (int t = 0; t < TT; ++t) {
            const f32x4_t h = *reinterpret_cast<const f32x4_t*>(hs.row + (16 * t + i) * Ranked<DT, TOK, kPass>::kLd + 16 * rb + 4 * q);
#pragma unroll
            for (int j = 0; j < JN; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                acc[j][t] = __builtin_amdgcn_mfma_f32_16x16x4f32(Elem<DT>::to_float(b[j * kPieces + rb].v[e]), h[e], acc[j][t], 0, 0, 0);
          }
        }
      }
    };
    // the lane's piece c, and the tokens' base there
    auto column = [&](int64_t n0, int c) -> int64_t { return n0 + 64 / kBase * c + kN * q; };
    const bool same = WHOLE != kAny ? WHOLE == kSameBase : p.base && p.base_dtype == OT;
    auto fetch = [&](int64_t n0, Piece<OT> (&raw)[TT][kBase]) {
      if (WHOLE != kAny && n0 >= n_end) n0 = w0;      // (a wave without columns: not used)
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const O* b = static_cast<const O*>(p.base) + token((in >> (16 * t + i)) & 1 ? 16 * t + i : 0) * p.ld_base;
#pragma unroll
        for (int c = 0; c < kBase; ++c)
          if (same && (WHOLE != kAny || column(n0, c) + kN <= n_end)) raw[t][c].load(b + column(n0, c));
      }
    };
    // what the first turn needs is in flight together: h (all of a thread's, where
    // the ranks fit one pass of up to 32), then the adapter's rows, then the base
    Piece<OT> raw[TT][kBase];
    RankPiece<DT> b[4][kPieces];
    const bool once = !BIG || p.rank <= kPass;
    float mine[kMostShares][4];
    const int padded = padded_ranks(0);
    if constexpr (!BIG && !DIRECT) fetch_h(threadIdx.x, 0, padded, mine);
    uint64_t todo = in;
    int a = SLOT ? s : __shfl(key, __builtin_ctzll(todo));
    auto load_all = [&](int64_t n0) {
      if (a >= 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) load_b(a, n0, j, 0, b[j]);
      }
    };
    load_all(w0 + wave * kWave);
    fetch(w0 + wave * kWave, raw);
    if (once) {
      __syncthreads();
      if constexpr (BIG) stage(0);
      else if constexpr (!DIRECT) put_h(threadIdx.x, 0, padded, mine);
      else if (narrow) stage_x(std::integral_constant<int, 1>{});
      else stage_x(std::integral_constant<int, 2>{});
      __syncthreads();
    }
    for (int64_t turn = w0; turn < n_end; turn += kThreads) {
      const int64_t n0 = turn + wave * kWave;
      f32x4_t acc[4][TT];
      if (WHOLE != kAny && !BIG && n0 >= n_end) break;      // (a turn of BIG has barriers)
      if (turn != w0) {
        todo = in;
        a = SLOT ? s : __shfl(key, __builtin_ctzll(todo));
        load_all(n0);
      }
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int c = 0; c < kBase; ++c) {
          const int64_t left = WHOLE != kAny ? kN : n_end - column(n0, c);
          float v[kN];
          if (same && left >= kN) {
#pragma unroll
            for (int e = 0; e < kN; ++e) v[e] = raw[t][c].get(e);
          } else {
#pragma unroll
            for (int e = 0; e < kN; ++e) v[e] = 0.0f;
            const int64_t at = token((in >> (16 * t + i)) & 1 ? 16 * t + i : 0) * p.ld_base + column(n0, c);
            if constexpr (WHOLE == kAny) {
              if (same && left > 0) get_some<OT, kN>(p.base, at, left, v);
              else if (p.base && left > 0) get_some<0, kN>(p.base, at, left, v);
            } else if constexpr (WHOLE == kWideBase) {
              get_some<0, kN>(p.base, at, kN, v);
            }
          }
#pragma unroll
          for (int e = 0; e < kN; ++e) acc[kN / 4 * c + e / 4][t][e % 4] = v[e];
        }
      if (turn + kThreads < n_end) fetch(n0 + kThreads, raw);
      for (;;) {
        const uint64_t mask = SLOT ? in : __ballot(key == a);
        todo &= ~mask;
        for (int r0 = 0; r0 < (BIG ? p.rank : 1); r0 += kPass) {
          if (!once) {
            __syncthreads();
            stage(r0);
            __syncthreads();
          }
          if (a < 0) continue;
          if (r0 > 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) load_b(a, n0, j, r0, b[j]);
          }
          if (mask == in) {
            products(&b[0][0], r0, std::integral_constant<int, 4>{}, acc);
            continue;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // only its own tokens take an adapter's results: another's infinity
            // or NaN times their zeros would not be zero
            f32x4_t now[1][TT];
#pragma unroll
            for (int t = 0; t < TT; ++t) now[0][t] = acc[j][t];
            products(b[j], r0, std::integral_constant<int, 1>{}, now);
#pragma unroll
            for (int t = 0; t < TT; ++t)
              if ((mask >> (16 * t + i)) & 1) acc[j][t] = now[0][t];
          }
        }
        if (todo == 0) break;
        a = __shfl(key, __builtin_ctzll(todo));
        load_all(n0);
      }
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        if (!((in >> (16 * t + i)) & 1)) continue;
        O* const o = static_cast<O*>(p.out) + token(16 * t + i) * p.n;
#pragma unroll
        for (int c = 0; c < kBase; ++c) {
          const int64_t n = column(n0, c), left = WHOLE != kAny ? kN : n_end - n;
          Piece<OT> w;
#pragma unroll
          for (int e = 0; e < kN; ++e) w.set(e, acc[kN / 4 * c + e / 4][t][e % 4]);
          if (left >= kN) __builtin_memcpy(o + n, w.v, 16);
          else if (left > 0) w.store_part(o + n, (int)left);
        }
      }
    }
  }
}

// ---- the way back -----------------------------------------------------------

// h[t, r] = the sum of its shares, in order.
__global__ __launch_bounds__(256) void lora_join_shares_kernel(const float* in, int shares,
                                                               int64_t elements, float* out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= elements) return;
  float v = in[i];
  for (int w = 1; w < shares; ++w) v += in[w * elements + i];
  out[i] = v;
}

// What the way back lays out first, in one launch: workgroup 0 sorts the tokens,
// the others transpose A and B, 64 x 64 elements each.
//
// The sort: tokens in adapter order (ascending inside an adapter) and the chunks
// that the gradients are summed in, by sixteen waves with a consecutive share of
// the tokens each.  entry = {adapter, first row, end row, 1 + the chunk's part, or 0
// where its adapter has no other chunk}; every adapter has one chunk at least, unused
// entries have adapter -1.  Adapter s's parts are part0[s] to part0[s + 1].
constexpr int kSortWaves = 16, kAhead = 16;

// Calls f(first token, key) for every 64 tokens of [t0, t1), kAhead loads in flight.
template <typename F>
__device__ __forceinline__ void walk_keys(const LoraSortArgs& p, int t0, int t1, F f) {
  const int lane = threadIdx.x % kWave;
  for (int base = t0; base < t1; base += kAhead * kWave) {
    int id[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int t = base + u * kWave + lane;
      id[u] = p.ids[t < t1 ? t : t1 - 1];
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int t = base + u * kWave + lane;
      if (base + u * kWave < t1) f(t, t < t1 ? key_of(id[u], p.adapters) : -1);
    }
  }
}

__device__ __forceinline__ void lora_sort(const LoraSortArgs& p, int32_t* place, int32_t (*sums)[kSortWaves]) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int S = p.adapters, tokens = (int)p.tokens;
  const int per = (tokens + kSortWaves * kWave - 1) / (kSortWaves * kWave) * kWave;
  const int t0 = wave * per < tokens ? wave * per : tokens, t1 = t0 + per < tokens ? t0 + per : tokens;
  // written by one lane, read by the others of its wave
  volatile int32_t* mine = place + wave * S;           // [wave][adapter]
  for (int i = threadIdx.x; i < kSortWaves * S; i += kSortWaves * kWave) place[i] = 0;
  __syncthreads();
  // The run's adapter and its count so far stay in registers: a request's tokens
  // lie together, and a turn through LDS for every 64 takes 27 us for 32768.
  int run = -1, at = 0;
  auto open = [&](int key) {
    if (key == run) return;
    if (run >= 0 && lane == 0) mine[run] = at;
    __builtin_amdgcn_wave_barrier();
    if (key >= 0) at = mine[key];
    __builtin_amdgcn_wave_barrier();
    run = key;
  };
  auto each = [&](int k, auto f) {
    uint64_t todo = __ballot(k >= 0);
    while (todo != 0) {
      const int key = __builtin_amdgcn_readfirstlane(__shfl(k, __builtin_ctzll(todo)));
      const uint64_t mask = __ballot(k == key);
      open(key);
      f(key, mask);
      at += __popcll(mask);
      todo &= ~mask;
    }
  };
  walk_keys(p, t0, t1, [&](int, int k) { each(k, [](int, uint64_t) {}); });
  open(-1);
  __syncthreads();
  // thread s: adapter s's tokens and chunks, then sums over the adapters before
  const int s = threadIdx.x;
  int count = 0;
  if (s < S)
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = place[w * S + s];
      place[w * S + s] = count;
      count += c;
    }
  const int chunks = s < S ? (count > p.chunk ? (count + p.chunk - 1) / p.chunk : 1) : 0;
  const int parts = chunks > 1 ? chunks : 0;
  int v[3] = {count, chunks, parts}, before[3];
#pragma unroll
  for (int a = 0; a < 3; ++a) {
    int x = v[a];
    for (int d = 1; d < kWave; d *= 2) {
      const int y = __shfl_up(x, d);
      if (lane >= d) x += y;
    }
    if (lane == kWave - 1) sums[a][wave] = x;
    before[a] = x - v[a];
  }
  __syncthreads();
  for (int w = 0; w < wave; ++w)
#pragma unroll
    for (int a = 0; a < 3; ++a) before[a] += sums[a][w];
  if (s < S) {
    for (int w = 0; w < kSortWaves; ++w) place[w * S + s] += before[0];
    p.part0[s] = before[2];
    for (int c = 0; c < chunks; ++c) {
      const int r0 = before[0] + c * p.chunk;
      const int r1 = r0 + p.chunk < before[0] + count ? r0 + p.chunk : before[0] + count;
      p.entries[before[1] + c] = make_int4(s, r0, r1, parts > 0 ? 1 + before[2] + c : 0);
    }
    if (s == S - 1) {
      sums[3][0] = before[0] + count;       // all routed tokens
      p.part0[S] = before[2] + parts;
      for (int c = before[1] + chunks; c < p.max_entries; ++c) p.entries[c] = make_int4(-1, 0, 0, 0);
    }
  }
  __syncthreads();
  for (int r = sums[3][0] + threadIdx.x; r < tokens + kRowsBehind; r += kSortWaves * kWave) p.rows[r] = 0;
  walk_keys(p, t0, t1, [&](int t, int k) {
    each(k, [&](int key, uint64_t mask) {
      if (k == key) p.rows[at + bits_below(mask)] = t;
    });
  });
}

// Tile t of [groups, rows, cols] to [groups, cols, rows].
template <typename T>
__device__ __forceinline__ void transpose_tile(const T* in, int64_t rows, int64_t cols, T* out, int64_t t,
                                               T (*tile)[65]) {
  const int64_t tc = (cols + 63) / 64, tr = (rows + 63) / 64;
  const int64_t r0 = t / tc % tr * 64, c0 = t % tc * 64, group = t / (tc * tr) * rows * cols;
  const int tx = threadIdx.x % 64, ty = threadIdx.x / 64;
#pragma unroll
  for (int r = ty; r < 64; r += kSortWaves)
    if (r0 + r < rows && c0 + tx < cols) tile[r][tx] = in[group + (r0 + r) * cols + c0 + tx];
  __syncthreads();
#pragma unroll
  for (int c = ty; c < 64; c += kSortWaves)
    if (c0 + c < cols && r0 + tx < rows) out[group + (c0 + c) * rows + r0 + tx] = tile[tx][c];
}

template <typename T>
__global__ __launch_bounds__(kSortWaves * kWave) void lora_prepare_kernel(LoraPrepareArgs p) {
  union Shared {
    struct {
      int32_t place[kSortWaves * kMaxAdapters];
      int32_t sums[4][kSortWaves];
    } sort;
    T tile[64][65];
  };
  __shared__ Shared sh;
  if (blockIdx.x == 0) {
    lora_sort(p.sort, sh.sort.place, sh.sort.sums);
    return;
  }
  const int64_t t = (int64_t)blockIdx.x - 1, na = (int64_t)p.sort.adapters * ((p.rank + 63) / 64) * ((p.k + 63) / 64);
  if (t < na) transpose_tile(static_cast<const T*>(p.a), p.rank, p.k, static_cast<T*>(p.at), t, sh.tile);
  else transpose_tile(static_cast<const T*>(p.b), p.n, p.rank, static_cast<T*>(p.bt), t - na, sh.tile);
}

// Grid: x = 128 columns of x, then of dy; y = chunks; z = 64 ranks each.  The
// waves take the chunk's tokens in turn, four at a time: lane l has rank
// l % 16 and columns 8 (l % 16) .. + 7 of token l / 16, so the rows are read
// 16 bytes a lane and nothing is transposed.  An adapter of one chunk writes
// its gradient, others a part each.
template <int DT, int RT>
__global__ __launch_bounds__(kThreads) void lora_grad_kernel(LoraGradArgs p) {
  typedef typename Elem<DT>::type T;
  __shared__ f32x4_t red[kWaves][8][kWave];
  const int4 e = p.entries[blockIdx.y];
  if (e.x < 0) return;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int i = lane % 16, q = lane / 16, z0 = blockIdx.z * kRanks;
  const int tiles_a = (int)((p.k + 127) / 128);
  const bool down = (int)blockIdx.x < tiles_a;       // dA (g, x), else dB (c h, dy)
  const int64_t width = down ? p.k : p.n, ld = down ? p.ld_x : p.ld_dy;
  const int64_t c0 = (int64_t)(down ? blockIdx.x : blockIdx.x - tiles_a) * 128 + 8 * i;
  const T* long_rows = static_cast<const T*>(down ? p.x : p.dy);
  const float* values = down ? p.g : p.h;
  const float c = down || !p.scale ? 1.0f : p.scale[e.x];
  f32x4_t acc[RT][8];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[rt][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};
  constexpr int U = 4;
  for (int t = e.y + 4 * wave; t < e.z; t += U * 4 * kWaves) {
    int64_t tok[U];
    bool in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = t + u * 4 * kWaves + q;
      in[u] = r < e.z;
      tok[u] = p.rows[in[u] ? r : e.z - 1];
    }
    float v[U][RT], x[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int r = z0 + 16 * rt + i;
        v[u][rt] = values[tok[u] * p.rank + (r < p.rank ? r : p.rank - 1)];
      }
      const T* row = long_rows + tok[u] * ld;
#pragma unroll
      for (int h = 0; h < 8; h += Piece<DT>::kN) {
        const Piece<DT> piece = piece_until<DT>(row, c0 + h, width);
#pragma unroll
        for (int b = 0; b < Piece<DT>::kN; ++b) x[u][h + b] = in[u] ? piece.get(b) : 0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const float a = in[u] ? c * v[u][rt] : 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          acc[rt][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(a, x[u][j], acc[rt][j], 0, 0, 0);
      }
  }
  const int64_t wide = (int64_t)p.rank * (p.k + p.n);
  float* out = e.w > 0 ? p.parts + (e.w - 1) * wide + (down ? 0 : p.rank * p.k)
                       : (down ? p.da + (int64_t)e.x * p.rank * p.k : p.db + (int64_t)e.x * p.rank * p.n);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) red[wave][j][lane] = acc[rt][j];
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = 2 * wave + h;
      f32x4_t v = red[0][j][lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += red[w][j][lane];
      const int64_t col = c0 + j;
      const int r = z0 + 16 * rt + 4 * q;
      if (col >= width) continue;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (r + b < p.rank) out[down ? (r + b) * p.k + col : col * p.rank + r + b] = v[b];
    }
  }
}

// The same for bf16 rows on MFMA 16x16x32: the g or c h of 32 tokens go through
// LDS as their three bf16 parts, token by token of a rank, and the rows' values
// are brought from eight tokens' registers into a column's by byte permutes.  A wave
// takes 64 columns, a workgroup eight waves (four waves of 128 columns: 74 us instead
// of 35 for 8192 tokens of rank 16), or with 64 ranks four waves (222 us for 32768
// tokens, eight 230 to 239, with longer chunks; columns read two turns ahead instead
// of one 213).  Grid: x = 512 (256) columns of x, then of dy.
// The binary32 form above is bound by its matrix instructions from rank 32 on
// (rank 64: 512 us for 470 MB).  Ranks 17 to 64 leave 5 and 10 registers in scratch.
template <int RT>
__global__ __launch_bounds__(RT == 4 ? 256 : 512, RT == 4 ? 3 : 4) void lora_grad16_kernel(LoraGradArgs p) {
  constexpr int R = 16 * RT, W = RT == 4 ? 4 : 8, C = 4;    // waves, columns of a lane
  // [part][rank][32 tokens], 16-byte chunk c of row r at c ^ (r / 4) % 4
  __shared__ __align__(16) uint16_t parts[2][3 * R * 32];
  const int4 e = p.entries[blockIdx.y];
  if (e.x < 0) return;
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int i = lane % 16, q = lane / 16, z0 = blockIdx.z * kRanks;
  constexpr int kCols = 16 * C * W;
  const int tiles_a = (int)((p.k + kCols - 1) / kCols);
  const bool down = (int)blockIdx.x < tiles_a;       // dA (g, x), else dB (c h, dy)
  const int64_t width = down ? p.k : p.n, ld = down ? p.ld_x : p.ld_dy;
  const int64_t c0 = (int64_t)(down ? blockIdx.x : blockIdx.x - tiles_a) * kCols + 16 * C * wave + C * i;
  const uint16_t* const rows = static_cast<const uint16_t*>(down ? p.x : p.dy);
  const float* const values = down ? p.g : p.h;
  const float c = down || !p.scale ? 1.0f : p.scale[e.x];
  const bool whole = c0 + C <= width;
  f32x4_t acc[RT][C];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int j = 0; j < C; ++j) acc[rt][j] = (f32x4_t){0.f, 0.f, 0.f, 0.f};

  // Tokens of the 32 from the chunk's row t on: the lane's eight, whose columns it
  // reads, and the one whose values the thread spreads.  (Rows past the chunk's are
  // another adapter's or the zeros behind the last: valid tokens, not used.)
  struct Tokens {
    int x[8], v;
  };
  auto tokens = [&](int t, Tokens& k) {
    __builtin_memcpy(k.x, p.rows + t + 8 * q, 32);
    k.v = p.rows[t + (int)threadIdx.x / (2 * W)];
  };
  struct Columns {
    uint16_t v[C];
  };
  auto fetch = [&](const Tokens& k, Columns (&x)[8]) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint16_t* row = rows + k.x[u] * ld + c0;
      if (whole) {
        __builtin_memcpy(x[u].v, row, sizeof(x[u].v));
      } else {
#pragma unroll
        for (int j = 0; j < C; ++j) x[u].v[j] = c0 + j < width ? row[j] : (uint16_t)0;
      }
    }
  };
  constexpr int kMine = R / (2 * W);      // ranks of a thread
  auto gather = [&](int t, int token, float (&v)[kMine]) {
    const bool in = t + (int)threadIdx.x / (2 * W) < e.z;
    const float* from = values + (int64_t)token * p.rank + z0;
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      const int rank = threadIdx.x % (2 * W) + 2 * W * m;
      const float f = from[z0 + rank < p.rank ? rank : 0];
      v[m] = in && z0 + rank < p.rank ? c * f : 0.0f;
    }
  };
  auto spread = [&](uint16_t* to, const float (&v)[kMine]) {
    const int t = threadIdx.x / (2 * W);
#pragma unroll
    for (int m = 0; m < kMine; ++m) {
      const int r = threadIdx.x % (2 * W) + 2 * W * m;
      uint16_t b[3];
      bf16_parts(v[m], b);
#pragma unroll
      for (int k = 0; k < 3; ++k) to[(k * R + r) * 32 + 8 * ((t / 8) ^ ((r >> 2) & 3)) + t % 8] = b[k];
    }
  };
  // The columns are read two turns ahead, the tokens three, the values one.
  Columns x0[8], x1[8];
  Tokens now, next;
  float v[kMine];
  int v1 = 0, at = 0;
  auto turn = [&](int t, Columns (&x)[8]) {
    __syncthreads();
    gather(t + 32, v1, v);
    // column b of the lane's: a dword of two tokens from words b / 2 of both
    bf16x8_t col[C];
#pragma unroll
    for (int b = 0; b < C; ++b) {
      uint32_t w[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint32_t lo, hi;
        __builtin_memcpy(&lo, x[2 * u].v + b / 2 * 2, 4);
        __builtin_memcpy(&hi, x[2 * u + 1].v + b / 2 * 2, 4);
        w[u] = __builtin_amdgcn_perm(hi, lo, b % 2 ? 0x07060302u : 0x05040100u);
        // (rows past the chunk's are zeros: no infinity times zero)
        const int r = t + 8 * q + 2 * u;
        w[u] = r + 1 < e.z ? w[u] : (r < e.z ? w[u] & 0xFFFFu : 0u);
      }
      __builtin_memcpy(&col[b], w, 16);
    }
    fetch(next, x);
    v1 = next.v;
    tokens(t + 96, next);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const int r = 16 * rt + i;
        const bf16x8_t a = *reinterpret_cast<const bf16x8_t*>(parts[at] + (k * R + r) * 32 + 8 * (q ^ ((r >> 2) & 3)));
#pragma unroll
        for (int b = 0; b < C; ++b) acc[rt][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, col[b], acc[rt][b], 0, 0, 0);
      }
    at ^= 1;
    spread(parts[at], v);
  };
  if (e.y < e.z) {
    tokens(e.y, now);
    tokens(e.y + 32, next);
    fetch(now, x0);
    gather(e.y, now.v, v);
    v1 = next.v;
    fetch(next, x1);
    tokens(e.y + 64, next);
    spread(parts[0], v);
    for (int t = e.y; t < e.z; t += 64) {
      turn(t, x0);
      if (t + 32 < e.z) turn(t + 32, x1);
    }
  }
  const int64_t wide = (int64_t)p.rank * (p.k + p.n);
  float* out = e.w > 0 ? p.parts + (e.w - 1) * wide + (down ? 0 : p.rank * p.k)
                       : (down ? p.da + (int64_t)e.x * p.rank * p.k : p.db + (int64_t)e.x * p.rank * p.n);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int r = z0 + 16 * rt + 4 * q;
    if (down) {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        if (r + b >= p.rank) continue;
        float* o = out + (r + b) * p.k + c0;
        float f[C];
#pragma unroll
        for (int j = 0; j < C; ++j) f[j] = acc[rt][j][b];
        if (whole) {
          __builtin_memcpy(o, f, sizeof(f));
        } else {
#pragma unroll
          for (int j = 0; j < C; ++j)
            if (c0 + j < width) o[j] = f[j];
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < C; ++j) {
        if (c0 + j >= width) continue;
        float* o = out + (c0 + j) * p.rank + r;
        if (r + 4 <= p.rank) {
          __builtin_memcpy(o, &acc[rt][j], 16);
        } else {
#pragma unroll
          for (int b = 0; b < 4; ++b)
            if (r + b < p.rank) o[b] = acc[rt][j][b];
        }
      }
    }
  }
}

// The gradients of adapters of several chunks: the parts added in chunk order.
__global__ __launch_bounds__(256) void lora_join_parts_kernel(LoraGradArgs p, const int32_t* part0) {
  const int s = blockIdx.y, c0 = part0[s], c1 = part0[s + 1];
  if (c1 == c0) return;
  const int64_t na = p.rank * p.k, wide = na + p.rank * p.n;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= wide) return;
  float v = p.parts[c0 * wide + i];
  for (int c = c0 + 1; c < c1; ++c) v += p.parts[c * wide + i];
  if (i < na) p.da[s * na + i] = v;
  else p.db[s * (wide - na) + i - na] = v;
}

template <int DT, int RT>
void down_rt(const LoraDownArgs& a, int group, dim3 grid, hipStream_t s) {
  if (group == 1) lora_down_kernel<DT, RT, 1, true><<<grid, kThreads, 0, s>>>(a);
  else if (group == 16) lora_down_kernel<DT, RT, 1, false><<<grid, kThreads, 0, s>>>(a);
  else if (group == 32) lora_down_kernel<DT, RT, 2, false><<<grid, kThreads, 0, s>>>(a);
  else lora_down_kernel<DT, RT, 4, false><<<grid, kThreads, 0, s>>>(a);
}

template <int DT>
void down_dt(const LoraDownArgs& a, int group, dim3 grid, hipStream_t s) {
  if (a.rank <= 16) down_rt<DT, 1>(a, group, grid, s);
  else if (a.rank <= 32) down_rt<DT, 2>(a, group, grid, s);
  else down_rt<DT, 4>(a, group, grid, s);
}

template <int DT, int OT, int WHOLE>
void up_kind(const LoraUpArgs& a, int group, dim3 grid, hipStream_t s) {
  const bool big = a.rank > 32;
  if (a.x)
    lora_up_kernel<DT, OT, 1, true, false, true, WHOLE><<<grid, kThreads, 0, s>>>(a);
  else if (group == 1)
    big ? lora_up_kernel<DT, OT, 1, true, true, false, WHOLE><<<grid, kThreads, 0, s>>>(a)
        : lora_up_kernel<DT, OT, 1, true, false, false, WHOLE><<<grid, kThreads, 0, s>>>(a);
  else
    big ? lora_up_kernel<DT, OT, 2, false, true, false, WHOLE><<<grid, kThreads, 0, s>>>(a)
        : lora_up_kernel<DT, OT, 2, false, false, false, WHOLE><<<grid, kThreads, 0, s>>>(a);
}

template <int DT, int OT>
void up_out(const LoraUpArgs& a, int group, dim3 grid, hipStream_t s) {
  if constexpr (DT == OT) {
    if (a.n % (a.rank > 32 ? kThreads : kWave) == 0 && a.rank % (DT == 1 ? 8 : 4) == 0) {
      if (!a.base) return up_kind<DT, OT, kNoBase>(a, group, grid, s);
      if (a.base_dtype == OT) return up_kind<DT, OT, kSameBase>(a, group, grid, s);
      return up_kind<DT, OT, kWideBase>(a, group, grid, s);
    }
  }
  up_kind<DT, OT, kAny>(a, group, grid, s);
}

template <int DT>
void up_dt(const LoraUpArgs& a, int group, dim3 grid, hipStream_t s) {
  if (a.out_dtype == 0) up_out<DT, 0>(a, group, grid, s);
  else if (a.out_dtype == 1) up_out<DT, 1>(a, group, grid, s);
  else up_out<DT, 2>(a, group, grid, s);
}

template <int DT>
void grad_dt(const LoraGradArgs& a, dim3 grid, hipStream_t s) {
  if (a.rank <= 16) lora_grad_kernel<DT, 1><<<grid, kThreads, 0, s>>>(a);
  else if (a.rank <= 32) lora_grad_kernel<DT, 2><<<grid, kThreads, 0, s>>>(a);
  else lora_grad_kernel<DT, 4><<<grid, kThreads, 0, s>>>(a);
}

// Tokens of a workgroup of the down products (1: the slots of up to kWindow): as
// many as the batch can spare with up to kMostShares shares of K, so that the
// adapter is read least often (rank 16, 8192 x 5120: 64 tokens 21.4 us, 32 23.3, 16
// 28.0; rank 64, 32768 x 5120: 96, 159, 222; 1003 x 1999 15.0, 10.3, 10.1).
int down_group(int64_t tokens) {
  if (tokens <= kWindow) return 1;
  return tokens >= 2048 ? 64 : (tokens >= 1024 ? 32 : 16);
}
int up_group(int64_t tokens) { return tokens <= kWindow ? 1 : 32; }
int64_t groups(int64_t tokens, int group) { return (tokens + group - 1) / group; }

}  // namespace

// Shares of K: as many as bring the launch to two workgroups a CU, of no less
// than one 128-byte piece a wave.
int lora_shares(int64_t tokens, int64_t k) {
  const int64_t blocks = groups(tokens, down_group(tokens)), most = (k + 255) / 256;
  int64_t w = blocks > 0 ? (512 + blocks - 1) / blocks : 1;
  w = w < most ? w : most;
  return (int)(w < 1 ? 1 : (w > kMostShares ? kMostShares : w));
}

// Tokens of a chunk of the gradients: enough chunks for three workgroups a CU.
int32_t lora_chunk(int dtype, int64_t tokens, int64_t k, int64_t n, int32_t rank) {
  const int64_t each = dtype == 1 ? (rank > 32 ? 256 : 512) : 128, tiles = (k + each - 1) / each + (n + each - 1) / each;
  const int64_t want = (768 + tiles - 1) / tiles;
  const int64_t c = ((tokens + want - 1) / want + 63) / 64 * 64;
  return (int32_t)(c < 64 ? 64 : c);
}

// Whether the up products may compute h themselves: up to 32 ranks of 160 KB in
// all, and 16 MB read by the call's workgroups (with the projection, 1 x 5120 x 2048
// of rank 16: 18.3 us a call, in two launches 19.7; 7 x 1001 x 1040 binary32 18.4,
// 21.3).
bool lora_direct(int dtype, int64_t tokens, int64_t k, int64_t n, int32_t rank) {
  const int64_t bytes = (int64_t)rank * k * (dtype == 0 ? 4 : 2);
  return tokens <= kWindow && rank <= 32 && bytes <= (160 << 10) &&
         bytes * tokens * ((n + 255) / 256) <= (16 << 20);
}

hipError_t launch_lora_down(LoraDownArgs a, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
  const int shares = lora_shares(a.tokens, a.k), group = down_group(a.tokens);
  a.share = ((a.k + shares - 1) / shares + 255) / 256 * 256;
  const dim3 grid((unsigned)groups(a.tokens, group), shares, (a.rank + kRanks - 1) / kRanks);
  if (a.dtype == 0) down_dt<0>(a, group, grid, s);
  else if (a.dtype == 1) down_dt<1>(a, group, grid, s);
  else down_dt<2>(a, group, grid, s);
  return hipGetLastError();
}

hipError_t launch_lora_up(LoraUpArgs a, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
  const int group = up_group(a.tokens);
  // 256 columns a workgroup; more while there are enough for eight (four) a CU
  // (256, 512, 1024 and 2048 columns: 4096 x 5120 28.6, 26.6, 30.4, 42.7 us, 8192 x
  // 2048 24.0, 22.7, 22.4, 33.8).  Up to kWindow tokens the workgroups of an adapter's
  // other tokens are counted with it and have nothing to do.
  const int64_t many = group == 1 ? 2048 : 1024, blocks = groups(a.tokens, group);
  a.wide = kThreads;
  while (a.wide < 4096 && blocks * ((a.n + 2 * a.wide - 1) / (2 * a.wide)) >= many) a.wide *= 2;
  const dim3 grid((unsigned)blocks, (unsigned)((a.n + a.wide - 1) / a.wide));
  if (a.dtype == 0) up_dt<0>(a, group, grid, s);
  else if (a.dtype == 1) up_dt<1>(a, group, grid, s);
  else up_dt<2>(a, group, grid, s);
  return hipGetLastError();
}

hipError_t launch_lora_prepare(const LoraPrepareArgs& a, hipStream_t s) {
  const int64_t ranks = (a.rank + 63) / 64, S = a.sort.adapters;
  const int64_t tiles = S * ranks * ((a.k + 63) / 64 + (a.n + 63) / 64);
  if (a.dtype == 0) lora_prepare_kernel<uint32_t><<<(unsigned)(1 + tiles), kSortWaves * kWave, 0, s>>>(a);
  else lora_prepare_kernel<uint16_t><<<(unsigned)(1 + tiles), kSortWaves * kWave, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_lora_join_shares(const float* in, int shares, int64_t elements, float* out,
                                   hipStream_t s) {
  if (elements == 0) return hipSuccess;
  lora_join_shares_kernel<<<(unsigned)((elements + 255) / 256), 256, 0, s>>>(in, shares, elements, out);
  return hipGetLastError();
}

hipError_t launch_lora_grad(const LoraGradArgs& a, int32_t max_entries, const int32_t* part0,
                            hipStream_t s) {
  const int64_t each = a.dtype == 1 ? (a.rank > 32 ? 256 : 512) : 128;
  const unsigned tiles = (unsigned)((a.k + each - 1) / each + (a.n + each - 1) / each);
  const dim3 grid(tiles, (unsigned)max_entries, (a.rank + kRanks - 1) / kRanks);
  if (a.dtype == 0) grad_dt<0>(a, grid, s);
  else if (a.dtype == 2) grad_dt<2>(a, grid, s);
  else if (a.rank <= 16) lora_grad16_kernel<1><<<grid, 512, 0, s>>>(a);
  else if (a.rank <= 32) lora_grad16_kernel<2><<<grid, 512, 0, s>>>(a);
  else lora_grad16_kernel<4><<<grid, 256, 0, s>>>(a);
  if (hipGetLastError() != hipSuccess) return hipErrorLaunchFailure;
  if (max_entries > a.adapters) {      // some adapter may have several chunks
    const int64_t wide = a.rank * (a.k + a.n);
    lora_join_parts_kernel<<<dim3((unsigned)((wide + 255) / 256), (unsigned)a.adapters), 256, 0, s>>>(a, part0);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
