// Expert selection from router logits, and its gradient.
//
// Forward, per token (a warp): scores s_e = softmax(l)_e or 1 / (1 + e^-l_e); the keys that decide are the
// logits when there is no balance bias (the scores' own order) and s_e + b_e otherwise; optional groups of
// experts scored by their largest key or by the sum of their two largest s_e + b_e, the best groups kept; the
// top_k largest keys in order, lower index on ties; weights scale * s_e (/ their sum).  The bias moves the
// choice and never the weights (the selection rule of auxiliary-loss-free balancing).
//
// Keys with a bias are compared in 64 bits: with thousands of tokens and hundreds of experts, scores that f32
// cannot tell apart do occur next to the border, and the choice must not depend on rounding.  The choice is first made
// in f32, and made again in 64 bits only where two keys it depends on are nearer to each other than f32 errors:
// 64-bit exponentials for every expert bound the kernel (73 us for 8192 tokens of 256 experts).
//
// Backward with the selection held constant: with n_k = s_k / S, S = sum_k s_k,
//   ds_k = scale / S (dw_k - sum_j dw_j n_j)  (renormalised)  or  scale dw_k,  plus d_scores;
//   softmax: dl_e = s_e (ds_e - sum_j ds_j s_j);  sigmoid: dl_e = ds_e s_e (1 - s_e).
#include "kernels.h"

namespace moe {

namespace {

constexpr int kSlots = 8;  // experts per lane: e = lane + 32 i
constexpr int kWarpsPerCta = 4;
constexpr unsigned kAll = 0xffffffffu;

// Order-preserving integer keys of f32 and f64 numbers (a > b iff key(a) > key(b), -0 as +0), their values, and the
// largest of a warp.  Zero is below every key.
template <typename F>
struct Keys;
template <>
struct Keys<float> {
  using type = uint32_t;
  static constexpr uint32_t kMinusInf = 0x007fffffu;
  static __device__ __forceinline__ uint32_t of(float v) {
    const uint32_t u = __float_as_uint(v == 0.f ? 0.f : v);
    return (u >> 31) ? ~u : (u | 0x80000000u);
  }
  static __device__ __forceinline__ float value(uint32_t k) {
    return __uint_as_float((k >> 31) ? (k & 0x7fffffffu) : ~k);
  }
  static __device__ __forceinline__ uint32_t largest(uint32_t k) { return __reduce_max_sync(kAll, k); }
};
template <>
struct Keys<double> {
  using type = unsigned long long;
  static constexpr unsigned long long kMinusInf = 0x000fffffffffffffull;
  static __device__ __forceinline__ unsigned long long of(double v) {
    const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(v == 0.0 ? 0.0 : v));
    return (u >> 63) ? ~u : (u | (1ull << 63));
  }
  static __device__ __forceinline__ double value(unsigned long long k) {
    return __longlong_as_double(static_cast<long long>((k >> 63) ? (k & ~(1ull << 63)) : ~k));
  }
  static __device__ __forceinline__ unsigned long long largest(unsigned long long k) {
    const uint32_t hi = __reduce_max_sync(kAll, static_cast<uint32_t>(k >> 32));
    const uint32_t lo = __reduce_max_sync(kAll, static_cast<uint32_t>(k >> 32) == hi ? static_cast<uint32_t>(k) : 0u);
    return (static_cast<unsigned long long>(hi) << 32) | lo;
  }
};

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_grad(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename F>
__device__ __forceinline__ F warp_add(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
// Largest of the lane's and the warp's logits (NaN left out).
__device__ __forceinline__ float row_max(const float (&l)[kSlots]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) m = max(m, l[i] == l[i] ? Keys<float>::of(l[i]) : 0u);
  m = __reduce_max_sync(kAll, m);
  return m ? Keys<float>::value(m) : -INFINITY;
}

// FAST: the quick exponential and quotient, for keys that are only compared with a margin.
template <bool FAST>
__device__ __forceinline__ float exp_of(float v) {
  return FAST ? __expf(v) : expf(v);
}
template <bool FAST>
__device__ __forceinline__ double exp_of(double v) {
  return exp(v);
}
template <bool FAST>
__device__ __forceinline__ float one_over(float v) {
  return FAST ? __fdividef(1.f, v) : 1.f / v;
}
template <bool FAST>
__device__ __forceinline__ double one_over(double v) {
  return 1.0 / v;
}

// Scores of the lane's experts from its logits (entries beyond E: -inf) and their maximum m.  A row of -inf alone
// scores 0.
template <typename F, bool FAST>
__device__ __forceinline__ void scores_of(const float (&l)[kSlots], float m, int E, int scoring, F (&s)[kSlots]) {
  const int lane = threadIdx.x & 31;
  if (scoring == MOE_GATING_SIGMOID) {
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
      s[i] = lane + 32 * i < E ? one_over<FAST>(F(1) + exp_of<FAST>(-static_cast<F>(l[i]))) : F(0);
    return;
  }
  F sum = 0;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    s[i] = lane + 32 * i < E && !(l[i] == -INFINITY) ? exp_of<FAST>(static_cast<F>(l[i]) - static_cast<F>(m)) : F(0);
    sum += s[i];
  }
  sum = warp_add(sum);
  const F inv = sum == F(0) ? F(0) : one_over<FAST>(sum);
#pragma unroll
  for (int i = 0; i < kSlots; ++i) s[i] *= inv;
}

// Value that lane `expert % 32` holds for `expert`, in every lane.
__device__ __forceinline__ float of_expert(const float (&v)[kSlots], int expert) {
  float mine = 0.f;
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if ((threadIdx.x & 31) + 32 * i == expert) mine = v[i];
  return __shfl_sync(kAll, mine, expert & 31);
}

// An f32 score is within kErr of the exact one (both are at most 1): with the quick forms, s (1 - s) times 2 + 1.2 |l|
// steps of 2^-23 from the exponential (below 1.3 2^-24 for every l), two steps from the quotient and one from the
// sum; for softmax e^-x times 2 + 1.7 x steps, and as much again for a sum of 256 terms in a tree.  A key s + b adds
// half a step of its size.
constexpr float kStep = 1.f / 16777216.f;
constexpr float kErr = 16.f * kStep;

// The token's choice: `chosen` of lane k < K becomes the k-th expert.  F = double decides every case.  F = float
// returns false where two keys, or two groups' scores, that the choice depends on are too near to each other for f32
// (about one token in a thousand).
template <typename F>
__device__ __forceinline__ bool choose(const float (&l)[kSlots], const F (&s)[kSlots], const float* bias,
                                       const SelectCfg& c, int& chosen) {
  using K_ = Keys<F>;
  using Key = typename K_::type;
  constexpr bool kExact = sizeof(F) == 8;
  const int lane = threadIdx.x & 31;
  const int E = c.E, K = c.K;
  const bool top2 = c.n_groups > 1 && c.group_score == MOE_GROUP_TOP2;
  Key key[kSlots];  // 0: not eligible
  Key by[kSlots];   // what groups are scored by
  uint32_t big = 0x3f800000u;  // largest |key|, as bits
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int e = lane + 32 * i;
    key[i] = by[i] = 0;
    if (e < E) {
      const F b = bias ? s[i] + static_cast<F>(bias[e]) : static_cast<F>(l[i]);
      const F v = l[i] == -INFINITY || b != b ? -INFINITY : b;
      key[i] = K_::of(v);
      by[i] = key[i];
      if (!bias && top2) by[i] = K_::of(l[i] == -INFINITY || s[i] != s[i] ? -INFINITY : s[i]);
      if (!kExact && bias && v != -INFINITY) big = max(big, __float_as_uint(static_cast<float>(v)) & 0x7fffffffu);
    }
  }
  // keys that are logits are compared exactly, without a margin
  float rounding = kStep, margin = 0.f;
  if (!kExact && bias) {
    rounding = __uint_as_float(__reduce_max_sync(kAll, big)) * kStep;
    margin = 2.f * (kErr + rounding);
    if (!(rounding < 1.f)) return false;  // infinite or enormous biases
  }
  if (c.n_groups > 1) {
    const int gs = E / c.n_groups;
    Key mine = 0;  // lane g: the key of group g's score
    auto score_of = [&](Key a, Key b) {  // from each lane's two largest of the group
      const Key m1 = K_::largest(a);
      if (!top2) return m1;
      const int who = __ffs(__ballot_sync(kAll, a == m1)) - 1;
      const Key m2 = K_::largest(lane == who ? b : a);
      return m2 > K_::kMinusInf ? K_::of(K_::value(m1) + K_::value(m2)) : m1;
    };
    if ((gs & 31) == 0) {  // whole slots: slot i belongs to group 32 i / gs in every lane
      Key a = 0, b = 0;
      int g = 0, left = gs;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        if (32 * i >= E) break;
        b = max(b, min(a, by[i]));
        a = max(a, by[i]);
        left -= 32;
        if (left == 0) {
          const Key v = score_of(a, b);
          if (lane == g) mine = v;
          a = b = 0;
          left = gs;
          ++g;
        }
      }
    } else {
      for (int g = 0; g < c.n_groups; ++g) {
        Key a = 0, b = 0;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
          const int e = lane + 32 * i;
          const Key v = e >= g * gs && e < (g + 1) * gs ? by[i] : Key(0);
          b = max(b, min(a, v));
          a = max(a, v);
        }
        const Key v = score_of(a, b);
        if (lane == g) mine = v;
      }
    }
    // rank of lane g's group: the groups that score more, and the equal ones before it
    int rank = 0;
    for (int g = 0; g < c.n_groups; ++g) {
      const Key o = __shfl_sync(kAll, mine, g);
      rank += o > mine || (o == mine && g < lane);
    }
    const bool in = lane < c.n_groups && rank < c.topk_groups;
    const unsigned kept = __ballot_sync(kAll, in);
    if (!kExact && c.topk_groups < c.n_groups && (bias || top2)) {
      // the last group kept against the first one dropped: twice a sum of two keys' errors, and its rounding
      const uint32_t lo = __reduce_min_sync(kAll, in ? static_cast<uint32_t>(mine) : 0xffffffffu);
      const uint32_t hi = __reduce_max_sync(kAll, lane < c.n_groups && !in ? static_cast<uint32_t>(mine) : 0u);
      const float gap = Keys<float>::value(lo) - Keys<float>::value(hi);
      if (hi > Keys<float>::kMinusInf && !(gap > 4.f * (kErr + 2.f * rounding))) return false;
    }
    if ((gs & 31) == 0) {
      int g = 0, left = gs;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        if (!((kept >> (g & 31)) & 1u)) key[i] = 0;
        left -= 32;
        if (left == 0) {
          left = gs;
          ++g;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        const int e = lane + 32 * i;
        if (e < E && !((kept >> (e / gs)) & 1u)) key[i] = 0;
      }
    }
  }
  // Each lane's keys in order (the lower slot first among equal ones), then a round is a maximum over the lanes' first
  // keys; the lane that held it (the lowest expert of several) moves its others up.
  int slot[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) slot[i] = i;
  auto order = [&](int a, int b) {
    const bool swap = key[b] > key[a] || (key[b] == key[a] && slot[b] < slot[a]);
    const Key ka = key[a];
    const int sa = slot[a];
    key[a] = swap ? key[b] : key[a];
    key[b] = swap ? ka : key[b];
    slot[a] = swap ? slot[b] : slot[a];
    slot[b] = swap ? sa : slot[b];
  };
  // odd-even merge sort of eight
  order(0, 1); order(2, 3); order(4, 5); order(6, 7);
  order(0, 2); order(1, 3); order(4, 6); order(5, 7);
  order(1, 2); order(5, 6);
  order(0, 4); order(1, 5); order(2, 6); order(3, 7);
  order(2, 4); order(3, 5);
  order(1, 2); order(3, 4); order(5, 6);
  Key last = 0;
  const int rounds = K + (margin > 0.f ? 1 : 0);  // one more to see how far the first one left behind is
  for (int k = 0; k < rounds; ++k) {
    const Key top = K_::largest(key[0]);
    if (!kExact && margin > 0.f && k > 0 && top > K_::kMinusInf &&
        !(static_cast<float>(K_::value(last) - K_::value(top)) > margin))
      return false;
    last = top;
    if (k == K) break;
    const unsigned e = __reduce_min_sync(kAll, key[0] == top ? static_cast<unsigned>(lane + 32 * slot[0]) : 0x7fffffffu);
    if (lane == k) chosen = static_cast<int>(e);
    if (lane + 32 * slot[0] == static_cast<int>(e)) {
#pragma unroll
      for (int i = 0; i + 1 < kSlots; ++i) {
        key[i] = key[i + 1];
        slot[i] = slot[i + 1];
      }
      key[kSlots - 1] = 0;
      slot[kSlots - 1] = 0x100000;  // no expert
    }
  }
  return true;
}

// Not inlined, so that what a token in a thousand needs does not take the others' registers.
__device__ __noinline__ int choose64(const float (&l_)[kSlots], float m, const float* bias, const SelectCfg& c) {
  float l[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) l[i] = l_[i];
  double s[kSlots];
  scores_of<double, false>(l, m, c.E, c.scoring, s);
  int chosen = 0;
  choose<double>(l, s, bias, c, chosen);
  return chosen;
}

template <typename LT>
__global__ void __launch_bounds__(32 * kWarpsPerCta)
    select_kernel(const LT* __restrict__ logits, long long stride, const float* __restrict__ bias, SelectCfg c,
                  int32_t* __restrict__ ids, float* __restrict__ w, float* __restrict__ scores) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  const long long t = static_cast<long long>(blockIdx.x) * kWarpsPerCta + warp;
  if (t >= c.T) return;
  const int E = c.E, K = c.K;
  float l[kSlots], s[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int e = lane + 32 * i;
    l[i] = e < E ? load_logit(logits + t * stride + e) : -INFINITY;
    s[i] = 0.f;
  }
  const bool softmax = c.scoring == MOE_GATING_SOFTMAX;
  const float m = softmax ? row_max(l) : 0.f;
  if (scores) {
    scores_of<float, false>(l, m, E, c.scoring, s);
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
      if (lane + 32 * i < E) scores[t * E + lane + 32 * i] = s[i];
  } else if (bias || (c.n_groups > 1 && c.group_score == MOE_GROUP_TOP2)) {
    scores_of<float, true>(l, m, E, c.scoring, s);
  }
  int e = 0;
  if (!choose<float>(l, s, bias, c, e)) e = choose64(l, m, bias, c);
  // the chosen scores again, from their logits; a softmax's own sum only where the weights are not renormalised
  float sum = 0.f;
  if (softmax && !c.renorm) {
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
      if (lane + 32 * i < E && !(l[i] == -INFINITY)) sum += expf(l[i] - m);
    sum = warp_add(sum);
  }
  float v = 0.f;
  if (lane < K) {
    const float x = load_logit(logits + t * stride + e);
    v = x == -INFINITY ? 0.f : softmax ? expf(x - m) : 1.f / (1.f + expf(-x));
  }
  if (c.renorm) sum = warp_add(v);
  if (lane < K) {
    ids[t * K + lane] = e;
    if (softmax || c.renorm) v = sum == 0.f ? 0.f : v / sum;
    w[t * K + lane] = c.scale * v;
  }
}

template <typename LT>
__global__ void __launch_bounds__(32 * kWarpsPerCta)
    select_backward_kernel(const LT* __restrict__ logits, long long stride, const int32_t* __restrict__ ids,
                           const float* __restrict__ d_w, const float* __restrict__ d_scores, SelectCfg c,
                           LT* __restrict__ d_logits, int* status) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  const long long t = static_cast<long long>(blockIdx.x) * kWarpsPerCta + warp;
  if (t >= c.T) return;
  const int E = c.E, K = c.K;
  float l[kSlots], ds[kSlots], s[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int e = lane + 32 * i;
    l[i] = e < E ? load_logit(logits + t * stride + e) : -INFINITY;
    ds[i] = e < E && d_scores ? d_scores[t * E + e] : 0.f;
  }
  int my_id = -1;
  float my_dw = 0.f;
  if (lane < K) {
    my_id = ids[t * K + lane];
    my_dw = c.scale * d_w[t * K + lane];
  }
  const bool bad = lane < K && (my_id < 0 || my_id >= E);
  if (bad) {
    record_status(status, MOE_ERR_DEVICE_INDEX);
    my_id = -1;
  }
  scores_of<float, false>(l, c.scoring == MOE_GATING_SOFTMAX ? row_max(l) : 0.f, E, c.scoring, s);
  if (c.renorm) {
    float my_s = 0.f;
    for (int k = 0; k < K; ++k) {
      const int id = __shfl_sync(kAll, my_id, k);
      const float v = of_expert(s, max(id, 0));
      if (lane == k && id >= 0) my_s = v;
    }
    const float sum = warp_add(my_s);
    const float mean = warp_add(my_id >= 0 ? my_dw * my_s : 0.f);
    my_dw = sum == 0.f ? 0.f : (my_dw - mean / sum) / sum;
  }
  for (int k = 0; k < K; ++k) {  // in slot order, so that an expert named twice sums the same way every time
    const int id = __shfl_sync(kAll, my_id, k);
    const float d = __shfl_sync(kAll, my_dw, k);
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
      if (lane + 32 * i == id) ds[i] += d;
  }
  float dot = 0.f;
  if (c.scoring == MOE_GATING_SOFTMAX) {
#pragma unroll
    for (int i = 0; i < kSlots; ++i) dot += ds[i] * s[i];
    dot = warp_add(dot);
  }
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int e = lane + 32 * i;
    if (e < E)
      store_grad(d_logits + t * E + e,
                 c.scoring == MOE_GATING_SOFTMAX ? s[i] * (ds[i] - dot) : ds[i] * s[i] * (1.f - s[i]));
  }
}

}  // namespace

cudaError_t launch_select(const Ctx& c, const void* logits, int logits_dtype, int64_t stride, const float* bias,
                          const SelectCfg& cfg, int32_t* ids, float* w, float* scores) {
  const dim3 grid((cfg.T + kWarpsPerCta - 1) / kWarpsPerCta), block(32 * kWarpsPerCta);
  KernelScope ks(c, "select");
  if (logits_dtype == MOE_F32)
    return launch_kernel(c, select_kernel<float>, grid, block, 0, static_cast<const float*>(logits),
                         static_cast<long long>(stride), bias, cfg, ids, w, scores);
  return launch_kernel(c, select_kernel<__nv_bfloat16>, grid, block, 0, static_cast<const __nv_bfloat16*>(logits),
                       static_cast<long long>(stride), bias, cfg, ids, w, scores);
}

cudaError_t launch_select_backward(const Ctx& c, const void* logits, int logits_dtype, int64_t stride,
                                   const SelectCfg& cfg, const int32_t* ids, const float* d_w, const float* d_scores,
                                   void* d_logits) {
  const dim3 grid((cfg.T + kWarpsPerCta - 1) / kWarpsPerCta), block(32 * kWarpsPerCta);
  KernelScope ks(c, "select_backward");
  if (logits_dtype == MOE_F32)
    return launch_kernel(c, select_backward_kernel<float>, grid, block, 0, static_cast<const float*>(logits),
                         static_cast<long long>(stride), ids, d_w, d_scores, cfg, static_cast<float*>(d_logits),
                         c.status);
  return launch_kernel(c, select_backward_kernel<__nv_bfloat16>, grid, block, 0,
                       static_cast<const __nv_bfloat16*>(logits), static_cast<long long>(stride), ids, d_w, d_scores,
                       cfg, static_cast<__nv_bfloat16*>(d_logits), c.status);
}

}  // namespace moe
