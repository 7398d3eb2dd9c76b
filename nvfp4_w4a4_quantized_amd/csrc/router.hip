// router.hip -- the MoE router's top-k choice and its gradient.
//
// For a token's logits l over E experts (and an optional bias b that counts
// for the choice alone):
//   key_e = fl32(l_e + b_e), or, with the bias on the score, fl32(s_e + b_e) where
//   s is the softmax over all experts or the sigmoid (the two rank differently:
//   the score saturates); the k largest keys are picked, ties to the lower
//   expert id; an expert whose key is -inf (masked) is never picked, so a
//   token may have fewer than k picks (expert id -1, weight 0);
//   softmax score: w_j = exp(l_j) / sum over all experts, or, renormalised,
//                  over the picks; sigmoid score: w_j = s(l_j), or that over
//                  the sum of the picks' s.
// Renormalised sums are taken as a softmax over the picks (of l, or of
// log s(l) = min(l, 0) - log1p(exp(-|l|))), so neither very large nor very
// negative logits overflow or leave 0 / 0.
// Gradient, with q the unscaled weights and S the picks:
//   softmax, renormalised: dl_j = q_j (dw_j - sum_S q dw), 0 outside S
//   softmax:               dl_e = [e in S] q_e dw_e - P_e sum_S q dw
//   sigmoid, renormalised: dl_j = q_j (dw_j - sum_S q dw)(1 - s_j)
//   sigmoid:               dl_j = dw_j s_j (1 - s_j)
// All statistics are binary32.
//
// Bound: the logits are read once (and the gradient written once), but at
// E = 128 the picking is the larger part: 636 vector instructions a wave of
// four tokens, of which the eight picks take 490 -- 8.5 of the 11.5 us of 32768
// tokens (fp32), whose 19 MB would pass in 4.  A token's row lies in the
// registers of L lanes, V consecutive experts each, so a pick is a local
// maximum of integer keys, four DPP rotations and the same for the lowest
// index among equals: no shared memory and no barrier (router_shape has L and V).
// The gradient of 8191 x 1000 bf16 logits takes 14 us (33 MB: 7 us).
#include "elem.h"
#include "launch.h"

#include <math.h>

namespace nvfp4 {

namespace {

constexpr int kRouterThreads = 256;
constexpr float kNegInf = -__builtin_huge_valf();

template <int N>
__device__ __forceinline__ int row_rotate(int v) {
  return __builtin_amdgcn_mov_dpp(v, 0x120 + N, 0xf, 0xf, true);   // row_ror:N
}

// Reduction over a token's L lanes (16: one DPP row; 64: the wave), the
// result in every lane.  All lanes of the wave are active.
template <int L, class Op>
__device__ __forceinline__ int group_reduce(int v, Op op) {
  v = op(v, row_rotate<8>(v));
  v = op(v, row_rotate<4>(v));
  v = op(v, row_rotate<2>(v));
  v = op(v, row_rotate<1>(v));
  if (L == 64) {
    const int a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
    const int c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    v = op(op(a, b), op(c, d));
  }
  return v;
}
template <int L>
__device__ __forceinline__ int group_max_int(int v) {
  return group_reduce<L>(v, [](int a, int b) { return a > b ? a : b; });
}
template <int L>
__device__ __forceinline__ int group_min_int(int v) {
  return group_reduce<L>(v, [](int a, int b) { return a < b ? a : b; });
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
  return __int_as_float(group_reduce<L>(__float_as_int(v), [](int a, int b) {
    return __float_as_int(__int_as_float(a) + __int_as_float(b));
  }));
}

// A binary32 value as an integer of the same order (both zeros alike, NaN
// below everything), and back: integer maxima need no canonicalisation.
constexpr int kKeyNan = (int)0x80000000;
constexpr int kKeyNegInf = (int)0x807FFFFF;
__device__ __forceinline__ int key_of(float f) {
  const int b = __float_as_int(f + 0.0f);
  const int k = b ^ ((b >> 31) & 0x7FFFFFFF);
  return f == f ? k : kKeyNan;
}
__device__ __forceinline__ float value_of(int k) {
  return __int_as_float(k ^ ((k >> 31) & 0x7FFFFFFF));
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
  return value_of(group_max_int<L>(key_of(v)));
}

// e^x for x <= 0, within (|x| + 2) 2^-24 relative (the argument's product is
// rounded once; results below 2^-126 flush to zero).
__device__ __forceinline__ float exp_neg(float x) {
  return __builtin_amdgcn_exp2f(x * 1.44269504088896340736f);
}
__device__ __forceinline__ float log_sigmoid(float z) {
  return fminf(z, 0.0f) - log1pf(expf(-fabsf(z)));
}
__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }

// V consecutive logits from element e0 of a row of `experts`, -inf past it,
// in 16-byte pieces: whole pieces are one load each, and the element loop is
// skipped where no lane holds a partial one (any width that is a multiple of
// a piece).
template <int DT, int V>
__device__ __forceinline__ void load_logits(float (&v)[V], const void* row, int e0, int experts) {
  typedef Piece<DT> P;
  constexpr int N = P::kN < V ? P::kN : V;
  const typename P::T* p = static_cast<const typename P::T*>(row);
#pragma unroll
  for (int c = 0; c < V; c += N) {
    const int left = experts - (e0 + c);
    typename P::T raw[N];
    if (left >= N) {
      __builtin_memcpy(raw, p + e0 + c, sizeof(raw));
    } else if (left > 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) raw[i] = i < left ? p[e0 + c + i] : (typename P::T)0;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[c + i] = i < left ? Elem<DT>::to_float(raw[i]) : kNegInf;
  }
}

template <int DT>
__device__ __forceinline__ const void* row_ptr(const void* base, int64_t t, int64_t ld) {
  return static_cast<const typename Elem<DT>::type*>(base) + t * ld;
}
template <int DT>
__device__ __forceinline__ float logit_at(const void* row, int e) {
  return Elem<DT>::to_float(static_cast<const typename Elem<DT>::type*>(row)[e]);
}

// The picks' statistics, lane j of the group holding picks j, j + L, ...:
// val (l or log s(l); -inf for none) in `vals`, and the softmax over them.
template <int L>
__device__ __forceinline__ void pick_softmax(const float* vals, int topk, int lane, float* mx,
                                             float* sum) {
  float m = kNegInf;
  for (int j = lane; j < topk; j += L) m = fmaxf(m, vals[j]);
  m = group_max<L>(m);
  float s = 0.0f;
  if (m > kNegInf)
    for (int j = lane; j < topk; j += L) s += exp_neg(vals[j] - m);
  *mx = m;
  *sum = group_sum<L>(s);
}

// exp(v - max) of a whole row, their sum; zeros for a row of -inf alone.
template <int L, int V>
__device__ __forceinline__ void row_softmax(const float (&v)[V], float (&p)[V], float* mx, float* sum) {
  float m = kNegInf;
#pragma unroll
  for (int i = 0; i < V; ++i) m = fmaxf(m, v[i]);
  m = group_max<L>(m);
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    p[i] = m > kNegInf ? exp_neg(v[i] - m) : 0.0f;
    s += p[i];
  }
  *mx = m;
  *sum = group_sum<L>(s);
}

// LDS lines of one token's lanes are written and read by the same wave only,
// in program order; the fence keeps the compiler to that order.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

}  // namespace

// SCORE_BIAS: a.bias is added to the scores (in a kernel of its own: the scores
// beside the logits take 12 to 28 registers, a wave per SIMD at 16 a lane).
template <int DT, int L, int V, bool SCORE_BIAS>
__global__ __launch_bounds__(kRouterThreads) void router_kernel(RouterArgs a) {
  extern __shared__ char lds[];
  constexpr int kGroups = kRouterThreads / L;
  const int group = threadIdx.x / L, lane = threadIdx.x % L;
  int32_t* pick = reinterpret_cast<int32_t*>(lds) + group * 2 * a.topk;
  float* vals = reinterpret_cast<float*>(pick + a.topk);
  const int64_t step = (int64_t)gridDim.x * kGroups;
  const int64_t rounds = (a.tokens + step - 1) / step;   // the same for every wave's lanes
  int64_t t = (int64_t)blockIdx.x * kGroups + group;
  for (int64_t it = 0; it < rounds; ++it, t += step) {
    const bool live = t < a.tokens;
    const void* row = row_ptr<DT>(a.logits, live ? t : 0, a.ld);
    const int e0 = lane * V;
    float v[V];
    load_logits<DT, V>(v, row, e0, a.num_experts);
    bool bad = false;   // NaN or +inf anywhere makes the row's weights NaN
#pragma unroll
    for (int i = 0; i < V; ++i) bad = bad || !(v[i] < __builtin_huge_valf());
    float mx = 0.0f, sum = 0.0f;
    if (a.score == 0 && (!a.renormalize || SCORE_BIAS)) {
      float p[V];
      row_softmax<L, V>(v, p, &mx, &sum);
      if (SCORE_BIAS) {
        const float inv = 1.0f / sum;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = v[i] > kNegInf ? p[i] * inv : kNegInf;
      }
    }
    if (a.score == 1 && SCORE_BIAS) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = v[i] > kNegInf ? sigmoid(v[i]) : kNegInf;
    }
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e0 + i < a.num_experts) v[i] += a.bias[e0 + i];
    }
    int key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) key[i] = key_of(v[i]);
    for (int j = 0, at = 0; j < a.topk; ++j, at = at + 1 == L ? 0 : at + 1) {
      int m = key[0];
#pragma unroll
      for (int i = 1; i < V; ++i) m = m > key[i] ? m : key[i];
      m = group_max_int<L>(m);
      int cand = 0x7FFFFFFF;
#pragma unroll
      for (int i = V - 1; i >= 0; --i) cand = key[i] == m ? e0 + i : cand;
      const int e = group_min_int<L>(cand);
      const int in = e - e0;
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = in == i ? kKeyNan : key[i];
      if (lane == at) {
        pick[j] = m > kKeyNegInf ? e : -1;
        vals[j] = value_of(m);
      }
    }
    wave_lds_fence();
    if (a.bias || (a.score == 1 && a.renormalize)) {
      for (int j = lane; j < a.topk; j += L) {
        const int e = pick[j];
        const float z = e < 0 ? kNegInf : (a.bias ? logit_at<DT>(row, e) : vals[j]);
        vals[j] = e >= 0 && a.score == 1 && a.renormalize ? log_sigmoid(z) : z;
      }
      wave_lds_fence();
    }
    if (a.renormalize) pick_softmax<L>(vals, a.topk, lane, &mx, &sum);
    const bool any_bad = group_max_int<L>(bad ? 1 : 0) != 0;
    for (int j = lane; j < a.topk; j += L) {
      const int e = pick[j];
      float w = 0.0f;
      if (e >= 0)
        w = a.score == 1 && !a.renormalize ? sigmoid(vals[j]) : exp_neg(vals[j] - mx) / sum;
      if (any_bad) w = __builtin_nanf("");
      if (live) {
        a.topk_idx[t * a.topk + j] = e;
        a.topk_prob[t * a.topk + j] = w * a.scale;
      }
    }
    wave_lds_fence();   // the next round writes the same lines
  }
}

template <int DT, int L, int V>
__global__ __launch_bounds__(kRouterThreads) void router_backward_kernel(RouterBackwardArgs a) {
  extern __shared__ char lds[];
  typedef typename Elem<DT>::type T;
  constexpr int kGroups = kRouterThreads / L;
  const int group = threadIdx.x / L, lane = threadIdx.x % L;
  int32_t* pick = reinterpret_cast<int32_t*>(lds) + group * 2 * a.topk;
  float* vals = reinterpret_cast<float*>(pick + a.topk);
  const bool full = a.score == 0 && !a.renormalize;   // every expert has a gradient
  const int64_t step = (int64_t)gridDim.x * kGroups;
  const int64_t rounds = (a.tokens + step - 1) / step;
  int64_t t = (int64_t)blockIdx.x * kGroups + group;
  for (int64_t it = 0; it < rounds; ++it, t += step) {
    const bool live = t < a.tokens;
    const int64_t tt = live ? t : 0;
    const void* row = row_ptr<DT>(a.logits, tt, a.ld);
    const int e0 = lane * V;
    float v[V];
    load_logits<DT, V>(v, row, e0, a.num_experts);
    bool bad = false;
#pragma unroll
    for (int i = 0; i < V; ++i) bad = bad || !(v[i] < __builtin_huge_valf());
    const bool any_bad = group_max_int<L>(bad ? 1 : 0) != 0;
    for (int j = lane; j < a.topk; j += L) {
      int e = a.topk_idx[tt * a.topk + j];
      if (e < 0 || e >= a.num_experts) e = -1;
      pick[j] = e;
      float z = e >= 0 ? logit_at<DT>(row, e) : kNegInf;
      vals[j] = e >= 0 && a.score == 1 && a.renormalize ? log_sigmoid(z) : z;
    }
    wave_lds_fence();
    float mx = 0.0f, sum = 1.0f;
    float p[V];
    if (full) {
      row_softmax<L, V>(v, p, &mx, &sum);
    } else if (a.renormalize) {
      pick_softmax<L>(vals, a.topk, lane, &mx, &sum);
    }
    const bool some = sum > 0.0f;   // a row with nothing to weigh has no gradient
    const float inv = some ? 1.0f / sum : 0.0f;
    // sum over the picks of q dw (not needed by the plain sigmoid)
    float mean = 0.0f;
    if (some && (full || a.renormalize)) {
      for (int j = lane; j < a.topk; j += L)
        if (pick[j] >= 0)
          mean += exp_neg(vals[j] - mx) * inv * (a.dprob[tt * a.topk + j] * a.scale);
    }
    mean = group_sum<L>(mean);
    for (int j = lane; j < a.topk; j += L) {
      const int e = pick[j];
      float d = 0.0f;
      if (e >= 0 && some) {
        const float dw = a.dprob[tt * a.topk + j] * a.scale;
        const float z = vals[j];
        if (full) {
          d = exp_neg(z - mx) * inv * dw;
        } else if (a.renormalize) {
          d = exp_neg(z - mx) * inv * (dw - mean);
          // vals holds log s(l) there; 1 - s(l) = s(-l)
          if (a.score == 1) d *= sigmoid(-logit_at<DT>(row, e));
        } else {
          d = dw * sigmoid(z) * sigmoid(-z);
        }
      }
      vals[j] = d;   // lane j reads and writes its own entries only
    }
    wave_lds_fence();
    float dz[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
      dz[i] = full ? -(p[i] * inv) * mean : 0.0f;
    for (int j = 0; j < a.topk; ++j) {
      const int at = pick[j] - e0;
      const float d = vals[j];
      if (pick[j] >= 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) dz[i] += at == i ? d : 0.0f;
      }
    }
    if (live) {
      T* out = static_cast<T*>(a.dlogits) + t * a.num_experts;
      constexpr int N = Piece<DT>::kN < V ? Piece<DT>::kN : V;
#pragma unroll
      for (int c = 0; c < V; c += N) {
        T raw[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
          raw[i] = Elem<DT>::from_float(any_bad ? __builtin_nanf("") : dz[c + i]);
        const int left = a.num_experts - (e0 + c);
        if (left >= N) {
          __builtin_memcpy(out + e0 + c, raw, sizeof(raw));
        } else if (left > 0) {
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (i < left) out[e0 + c + i] = raw[i];
        }
      }
    }
    wave_lds_fence();
  }
}

namespace {

// The shape for a call: lanes per token and consecutive experts per lane.  16
// lanes take four tokens a wave, so a pick costs a quarter of the reduction, with
// up to 128 experts always and up to 512 where 8192 tokens fill the chip; else
// the wave takes one.  A lane holds no more experts than needed.  Measured, bf16:
//   32768 tokens, top-2 of 8: 1 expert a lane 5.4 us, 8 experts 7.2; top-4 of 16
//   6.0 / 8.8; top-6 of 64: 4 experts 8.1, 8 experts 10.2; top-10 of 512, the
//   wave: 8 experts 46, 16 experts 70;
//   16 lanes / the wave: top-6 of 160: 2048 tokens 6.1 / 5.3, 4096 6.1 / 6.5, 8192
//   6.8 / 9.4, 32768 15.4 / 26.8; its gradient, 4096 tokens 6.3 / 6.0, 8192 6.4 /
//   8.5; top-10 of 512: 4096 tokens 10.8 / 9.8, 8192 12.7 / 14.9, 32768 37.5 / 46.3;
//   top-8 of 1000, 8192 tokens 22.3 / 19.3, 32768 72 / 61.
struct RouterShape { int lanes, per_lane; unsigned blocks; size_t lds; };
RouterShape router_shape(int64_t tokens, int32_t experts, int32_t topk) {
  RouterShape s;
  s.lanes = experts <= 128 || (experts <= 512 && tokens >= 8192) ? 16 : 64;
  const int least = (experts + s.lanes - 1) / s.lanes;
  s.per_lane = least == 1 ? 1 : (least <= 4 ? 4 : (least <= 8 ? 8 : (least <= 16 ? 16 : 32)));
  const int groups = kRouterThreads / s.lanes;
  const int64_t blocks = (tokens + groups - 1) / groups;
  s.blocks = (unsigned)(blocks < (1 << 20) ? blocks : 1 << 20);
  s.lds = (size_t)groups * 2 * topk * 4;
  return s;
}

}  // namespace

// LAUNCH(dtype, lanes, per lane) for the call's shape
#define NVFP4_ROUTER_CASE(LAUNCH, L, V)        \
  case L * 100 + V:                            \
    if (a.dtype == 0) LAUNCH(0, L, V);         \
    else if (a.dtype == 1) LAUNCH(1, L, V);    \
    else LAUNCH(2, L, V);                      \
    break;
#define NVFP4_ROUTER_CASES(LAUNCH)                                        \
  do {                                                                    \
    const RouterShape sh = router_shape(a.tokens, a.num_experts, a.topk); \
    switch (sh.lanes * 100 + sh.per_lane) {                               \
      NVFP4_ROUTER_CASE(LAUNCH, 16, 1)                                    \
      NVFP4_ROUTER_CASE(LAUNCH, 16, 4)                                    \
      NVFP4_ROUTER_CASE(LAUNCH, 16, 8)                                    \
      NVFP4_ROUTER_CASE(LAUNCH, 16, 16)                                   \
      NVFP4_ROUTER_CASE(LAUNCH, 16, 32)                                   \
      NVFP4_ROUTER_CASE(LAUNCH, 64, 4)                                    \
      NVFP4_ROUTER_CASE(LAUNCH, 64, 8)                                    \
      NVFP4_ROUTER_CASE(LAUNCH, 64, 16)                                   \
    }                                                                     \
  } while (0)

hipError_t launch_router(const RouterArgs& a, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
#define NVFP4_ROUTER(D, L, V) \
  router_kernel<D, L, V, false><<<sh.blocks, kRouterThreads, sh.lds, s>>>(a)
#define NVFP4_ROUTER_SCORE_BIAS(D, L, V) \
  router_kernel<D, L, V, true><<<sh.blocks, kRouterThreads, sh.lds, s>>>(a)
  if (a.bias_on_score) NVFP4_ROUTER_CASES(NVFP4_ROUTER_SCORE_BIAS);
  else NVFP4_ROUTER_CASES(NVFP4_ROUTER);
#undef NVFP4_ROUTER_SCORE_BIAS
#undef NVFP4_ROUTER
  return hipGetLastError();
}

hipError_t launch_router_backward(const RouterBackwardArgs& a, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
#define NVFP4_ROUTER_BACKWARD(D, L, V) \
  router_backward_kernel<D, L, V><<<sh.blocks, kRouterThreads, sh.lds, s>>>(a)
  NVFP4_ROUTER_CASES(NVFP4_ROUTER_BACKWARD);
#undef NVFP4_ROUTER_BACKWARD
  return hipGetLastError();
}

#undef NVFP4_ROUTER_CASES
#undef NVFP4_ROUTER_CASE

}  // namespace nvfp4
