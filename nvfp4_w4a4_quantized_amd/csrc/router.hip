// router.hip -- the MoE router's top-k choice and its gradient.
//
// For a token's logits l over E experts (and an optional bias b that counts
// for the choice alone):
//   key_e = fl32(l_e + b_e); the k largest keys are picked, ties to the lower
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
// Bound: the logits are read once (and the gradient written once); at E = 128
// the picking itself is the larger part.  A token's row lies in the registers
// of L lanes, V consecutive experts each, so a pick is a local maximum, a
// lane reduction by DPP rotations and the same for the lowest index among
// equals: no shared memory and no barrier.
#include "launch.h"
#include "elem.h"

#include <math.h>

namespace nvfp4 {

namespace {

constexpr int kRouterThreads = 256;
constexpr float kNegInf = -__builtin_huge_valf();

template <int N>
__device__ __forceinline__ uint32_t row_rotate(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x120 + N, 0xf, 0xf, false);   // row_ror:N
}

// Reduction over a token's L lanes (16: one DPP row; 64: the wave), the
// result in every lane.  All lanes of the wave are active.
template <int L, class Op>
__device__ __forceinline__ uint32_t group_reduce_bits(uint32_t v, Op op) {
  v = op(v, row_rotate<8>(v));
  v = op(v, row_rotate<4>(v));
  v = op(v, row_rotate<2>(v));
  v = op(v, row_rotate<1>(v));
  if (L == 64) {
    const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)v, 0);
    const uint32_t b = (uint32_t)__builtin_amdgcn_readlane((int)v, 16);
    const uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)v, 32);
    const uint32_t d = (uint32_t)__builtin_amdgcn_readlane((int)v, 48);
    v = op(op(a, b), op(c, d));
  }
  return v;
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
  return __uint_as_float(group_reduce_bits<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
  return __uint_as_float(group_reduce_bits<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int L>
__device__ __forceinline__ uint32_t group_min_u32(uint32_t v) {
  return group_reduce_bits<L>(v, [](uint32_t a, uint32_t b) { return a < b ? a : b; });
}

__device__ __forceinline__ float log_sigmoid(float z) {
  return fminf(z, 0.0f) - log1pf(expf(-fabsf(z)));
}
__device__ __forceinline__ float sigmoid(float z) { return 1.0f / (1.0f + expf(-z)); }

// V consecutive logits from element e0 of a row of `experts`; -inf past it.
template <int DT, int V>
__device__ __forceinline__ void load_logits(float (&v)[V], const void* row, int e0, int experts) {
  typedef typename Elem<DT>::type T;
  const T* p = static_cast<const T*>(row);
  if (e0 + V <= experts) {
    T raw[V];
    __builtin_memcpy(raw, p + e0, sizeof(raw));
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = Elem<DT>::to_float(raw[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = e0 + i < experts ? Elem<DT>::to_float(p[e0 + i]) : kNegInf;
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
    for (int j = lane; j < topk; j += L) s += expf(vals[j] - m);
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

template <int DT, int L, int V>
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
    if (a.score == 0 && !a.renormalize) {
      mx = kNegInf;
#pragma unroll
      for (int i = 0; i < V; ++i) mx = fmaxf(mx, v[i]);
      mx = group_max<L>(mx);
      if (mx > kNegInf) {
#pragma unroll
        for (int i = 0; i < V; ++i) sum += expf(v[i] - mx);
      }
      sum = group_sum<L>(sum);
    }
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e0 + i < a.num_experts) v[i] += a.bias[e0 + i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = v[i] == v[i] ? v[i] : kNegInf;
    for (int j = 0; j < a.topk; ++j) {
      float m = v[0];
#pragma unroll
      for (int i = 1; i < V; ++i) m = fmaxf(m, v[i]);
      m = group_max<L>(m);
      uint32_t cand = 0x7FFFFFFFu;
#pragma unroll
      for (int i = V - 1; i >= 0; --i) cand = v[i] == m ? (uint32_t)(e0 + i) : cand;
      const uint32_t e = group_min_u32<L>(cand);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = (uint32_t)(e0 + i) == e ? kNegInf : v[i];
      if (lane == j % L) pick[j] = m > kNegInf ? (int32_t)e : -1;
    }
    wave_lds_fence();
    for (int j = lane; j < a.topk; j += L) {
      const int e = pick[j];
      float z = e >= 0 ? logit_at<DT>(row, e) : kNegInf;
      vals[j] = e >= 0 && a.score == 1 && a.renormalize ? log_sigmoid(z) : z;
    }
    wave_lds_fence();
    if (a.renormalize) pick_softmax<L>(vals, a.topk, lane, &mx, &sum);
    const bool any_bad = group_max<L>(bad ? 1.0f : 0.0f) > 0.0f;
    for (int j = lane; j < a.topk; j += L) {
      const int e = pick[j];
      float w = 0.0f;
      if (e >= 0)
        w = a.score == 1 && !a.renormalize ? sigmoid(vals[j]) : expf(vals[j] - mx) / sum;
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
    const bool any_bad = group_max<L>(bad ? 1.0f : 0.0f) > 0.0f;
    for (int j = lane; j < a.topk; j += L) {
      int e = a.topk_idx[tt * a.topk + j];
      if (e < 0 || e >= a.num_experts) e = -1;
      pick[j] = e;
      float z = e >= 0 ? logit_at<DT>(row, e) : kNegInf;
      vals[j] = e >= 0 && a.score == 1 && a.renormalize ? log_sigmoid(z) : z;
    }
    wave_lds_fence();
    float mx = 0.0f, sum = 1.0f;
    if (full) {
      mx = kNegInf;
#pragma unroll
      for (int i = 0; i < V; ++i) mx = fmaxf(mx, v[i]);
      mx = group_max<L>(mx);
      sum = 0.0f;
      if (mx > kNegInf) {
#pragma unroll
        for (int i = 0; i < V; ++i) sum += expf(v[i] - mx);
      }
      sum = group_sum<L>(sum);
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
          mean += expf(vals[j] - mx) * inv * (a.dprob[tt * a.topk + j] * a.scale);
    }
    mean = group_sum<L>(mean);
    for (int j = lane; j < a.topk; j += L) {
      const int e = pick[j];
      float d = 0.0f;
      if (e >= 0 && some) {
        const float dw = a.dprob[tt * a.topk + j] * a.scale;
        const float z = vals[j];
        if (full) {
          d = expf(z - mx) * inv * dw;
        } else if (a.renormalize) {
          d = expf(z - mx) * inv * (dw - mean);
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
      dz[i] = full && some ? -(expf(v[i] - mx) * inv) * mean : 0.0f;
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
      T raw[V];
#pragma unroll
      for (int i = 0; i < V; ++i)
        raw[i] = Elem<DT>::from_float(any_bad ? __builtin_nanf("") : dz[i]);
      if (e0 + V <= a.num_experts) {
        __builtin_memcpy(out + e0, raw, sizeof(raw));
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (e0 + i < a.num_experts) out[e0 + i] = raw[i];
      }
    }
    wave_lds_fence();
  }
}

namespace {

// Lanes per token: 16 (four tokens a wave) up to 128 experts, the wave above.
struct RouterShape { int lanes; int64_t blocks; size_t lds; };
RouterShape router_shape(int64_t tokens, int32_t experts, int32_t topk) {
  RouterShape s;
  s.lanes = experts <= 128 ? 16 : 64;
  const int groups = kRouterThreads / s.lanes;
  s.blocks = (tokens + groups - 1) / groups;
  if (s.blocks > 1 << 20) s.blocks = 1 << 20;
  s.lds = (size_t)groups * 2 * topk * 4;
  return s;
}

}  // namespace

#define NVFP4_ROUTER_CASES(KERNEL)                                                     \
  do {                                                                                 \
    const RouterShape sh = router_shape(a.tokens, a.num_experts, a.topk);              \
    const unsigned blocks = (unsigned)sh.blocks;                                       \
    const int v = a.num_experts <= 128 ? 8 : (a.num_experts <= 256 ? 4 : 16);          \
    switch (a.dtype * 100 + v) {                                                       \
      case 8: KERNEL<0, 16, 8><<<blocks, kRouterThreads, sh.lds, s>>>(a); break;       \
      case 4: KERNEL<0, 64, 4><<<blocks, kRouterThreads, sh.lds, s>>>(a); break;       \
      case 16: KERNEL<0, 64, 16><<<blocks, kRouterThreads, sh.lds, s>>>(a); break;     \
      case 108: KERNEL<1, 16, 8><<<blocks, kRouterThreads, sh.lds, s>>>(a); break;     \
      case 104: KERNEL<1, 64, 4><<<blocks, kRouterThreads, sh.lds, s>>>(a); break;     \
      case 116: KERNEL<1, 64, 16><<<blocks, kRouterThreads, sh.lds, s>>>(a); break;    \
      case 208: KERNEL<2, 16, 8><<<blocks, kRouterThreads, sh.lds, s>>>(a); break;     \
      case 204: KERNEL<2, 64, 4><<<blocks, kRouterThreads, sh.lds, s>>>(a); break;     \
      default: KERNEL<2, 64, 16><<<blocks, kRouterThreads, sh.lds, s>>>(a); break;     \
    }                                                                                  \
  } while (0)

hipError_t launch_router(const RouterArgs& a, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
  NVFP4_ROUTER_CASES(router_kernel);
  return hipGetLastError();
}

hipError_t launch_router_backward(const RouterBackwardArgs& a, hipStream_t s) {
  if (a.tokens == 0) return hipSuccess;
  NVFP4_ROUTER_CASES(router_backward_kernel);
  return hipGetLastError();
}

#undef NVFP4_ROUTER_CASES

}  // namespace nvfp4
