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
// in f32, and only what it depends on is compared again in 64 bits, where two keys are nearer to each other than f32
// errors: 64-bit exponentials for every expert bound the kernel (73 us for 8192 tokens of 256 experts).
//
// A lane holds a run of consecutive experts, so that a group is a few whole lanes and its two largest keys meet in as
// many steps.  The choice itself: the K-th largest of the 32 lanes' largest keys bounds the K-th largest of all from
// below; the few keys not under it (20 or so of 256) move to a lane each, which counts the keys before its own.  That
// is two thirds fewer instructions than a sort in every lane and K rounds of a maximum over the warp, which took 24 us
// for 8192 tokens of 256 experts in 8 groups; now 12 us, of 1030 instructions a token, for the 8.9 MB read and written:
// bound by dependent instructions at the five warps a scheduler that 80 registers allow (one issued every 8.4 cycles of
// a warp), no pipe being full.
//
// Backward with the selection held constant: with n_k = s_k / S, S = sum_k s_k,
//   ds_k = scale / S (dw_k - sum_j dw_j n_j)  (renormalised)  or  scale dw_k,  plus d_scores;
//   softmax: dl_e = s_e (ds_e - sum_j ds_j s_j);  sigmoid: dl_e = ds_e s_e (1 - s_e).
// Renormalised, with a chosen score below 2^-60, the products s_k ds_k = scale n_k (dw_k - sum_j dw_j n_j) are formed
// without s_k and S, which can be too small for f32 where n_k is not; their sum over k is 0.
#include "kernels.h"

namespace moe {

namespace {

constexpr int kSlots = 8;  // experts per lane, at most: forward [lane per, + per), backward lane + 32 i
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
    const uint32_t u = __float_as_uint(v + 0.f);  // -0 + 0 = +0
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
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

// Scores of the lane's experts from its logits (-inf where it has none) and their maximum m.  A row of -inf alone
// scores 0.
template <bool SIGMOID, bool FAST, typename F>
__device__ __forceinline__ F score_term(float l, float m) {
  if (SIGMOID) return one_over<FAST>(F(1) + exp_of<FAST>(-static_cast<F>(l)));
  return l == -INFINITY ? F(0) : exp_of<FAST>(static_cast<F>(l) - static_cast<F>(m));
}
template <typename F, bool FAST>
__device__ __forceinline__ void scores_of(const float (&l)[kSlots], float m, int scoring, F (&s)[kSlots]) {
  if (scoring == MOE_GATING_SIGMOID) {
#pragma unroll
    for (int i = 0; i < kSlots; ++i) s[i] = score_term<true, FAST, F>(l[i], m);
    return;
  }
  F sum = 0;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    s[i] = score_term<false, FAST, F>(l[i], m);
    sum += s[i];
  }
  sum = warp_add(sum);
  const F inv = sum == F(0) ? F(0) : one_over<FAST>(sum);
#pragma unroll
  for (int i = 0; i < kSlots; ++i) s[i] *= inv;
}

// A chosen expert's score times a factor common to the token's choices, from its logit x and the largest chosen logit,
// `top` (`mine`: x is one of them; NaN left out): e^(x - top), or with sigmoid, whose score is e^min(x, 0) / (1 + e^-|x|),
// the same with x - min(top, 0) in the exponent.  The ratios survive where the scores do not: with a bias or groups the
// chosen softmax scores can all lie below f32's range, 104 under the row's maximum, sigmoid's do for logits below -88.
__device__ __forceinline__ float shifted_score(float x, bool mine, bool softmax) {
  const uint32_t k = __reduce_max_sync(kAll, mine && x == x ? Keys<float>::of(x) : 0u);
  const float top = k ? Keys<float>::value(k) : -INFINITY;
  if (!mine || x == -INFINITY) return 0.f;
  return softmax ? expf(x - top) : expf(fminf(x, 0.f) - fminf(top, 0.f)) / (1.f + expf(-fabsf(x)));
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

// The lane's `per` logits from `first` on (-inf beyond E).  Rows of 256 are read 16 bytes at a time where they can be.
__device__ __forceinline__ void load_run(const float* row, int first, int per, int E, float (&l)[kSlots]) {
  if (per == kSlots && E == 32 * kSlots && (reinterpret_cast<uintptr_t>(row) & 15) == 0) {
    const float4 a = *reinterpret_cast<const float4*>(row + first), b = *reinterpret_cast<const float4*>(row + first + 4);
    l[0] = a.x; l[1] = a.y; l[2] = a.z; l[3] = a.w;
    l[4] = b.x; l[5] = b.y; l[6] = b.z; l[7] = b.w;
    return;
  }
#pragma unroll
  for (int i = 0; i < kSlots; ++i) l[i] = i < per && first + i < E ? row[first + i] : -INFINITY;
}
__device__ __forceinline__ void load_run(const __nv_bfloat16* row, int first, int per, int E, float (&l)[kSlots]) {
  if (per == kSlots && E == 32 * kSlots && (reinterpret_cast<uintptr_t>(row) & 15) == 0) {
    const uint4 a = *reinterpret_cast<const uint4*>(row + first);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      l[2 * i] = __uint_as_float(w[i] << 16);
      l[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kSlots; ++i) l[i] = i < per && first + i < E ? __bfloat162float(row[first + i]) : -INFINITY;
}

// The key that decides for an expert, and the one its group is scored by.
template <typename F>
__device__ __forceinline__ F deciding(float l, F s, bool biased, float bias) {
  const F b = biased ? s + static_cast<F>(bias) : static_cast<F>(l);
  return l == -INFINITY || b != b ? F(-INFINITY) : b;
}
template <typename F>
__device__ __forceinline__ typename Keys<F>::type grouping(float l, F s, F key, bool by_score) {
  return Keys<F>::of(!by_score ? key : l == -INFINITY || s != s ? F(-INFINITY) : s);
}

// The groups kept, as bits, from the lanes' runs of keys (0: no expert); lane g gets group g's score in `mine`.
template <typename F>
__device__ __forceinline__ unsigned kept_groups(const typename Keys<F>::type (&by)[kSlots], int first,
                                                const SelectCfg& c, typename Keys<F>::type& mine) {
  using K_ = Keys<F>;
  using Key = typename K_::type;
  const int lane = threadIdx.x & 31;
  const bool top2 = c.group_score == MOE_GROUP_TOP2;
  auto score = [&](Key a, Key b) { return top2 && b > K_::kMinusInf ? K_::of(K_::value(a) + K_::value(b)) : a; };
  mine = 0;
  if (c.E % 32 == 0 && 32 % c.n_groups == 0) {  // whole lanes
    const int lanes = 32 / c.n_groups;
    Key a = 0, b = 0;  // the two largest
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      b = max(b, min(a, by[i]));
      a = max(a, by[i]);
    }
    for (int o = 1; o < lanes; o <<= 1) {
      const Key oa = __shfl_xor_sync(kAll, a, o), ob = __shfl_xor_sync(kAll, b, o);
      b = max(min(a, oa), max(b, ob));
      a = max(a, oa);
    }
    mine = __shfl_sync(kAll, score(a, b), lane * lanes & 31);
  } else {
    const int gs = c.E / c.n_groups;
    for (int g = 0; g < c.n_groups; ++g) {
      Key a = 0, b = 0;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        const int e = first + i;
        const Key v = e >= g * gs && e < (g + 1) * gs ? by[i] : Key(0);
        b = max(b, min(a, v));
        a = max(a, v);
      }
      const Key m1 = K_::largest(a);
      const int who = __ffs(__ballot_sync(kAll, a == m1)) - 1;
      const Key m2 = K_::largest(lane == who ? b : a);
      if (lane == g) mine = score(m1, m2);
    }
  }
  // rank of lane g's group: the groups that score more, and the equal ones before it
  int rank = 0;
  for (int g = 0; g < c.n_groups; ++g) {
    const Key o = __shfl_sync(kAll, mine, g);
    rank += o > mine || (o == mine && g < lane);
  }
  return __ballot_sync(kAll, lane < c.n_groups && rank < c.topk_groups);
}

// The choice in 64 bits throughout, for any row: lane k < K returns the k-th expert.  Not inlined, so that what a token
// in thousands needs does not take the others' registers.
template <typename LT>
__device__ __noinline__ int choose64(const LT* row, const float* bias, const SelectCfg& c) {
  using K_ = Keys<double>;
  using Key = K_::type;
  const int lane = threadIdx.x & 31, per = (c.E + 31) / 32, first = lane * per;
  float l[kSlots];
  load_run(row, first, per, c.E, l);
  double s[kSlots];
  scores_of<double, false>(l, c.scoring == MOE_GATING_SOFTMAX ? row_max(l) : 0.f, c.scoring, s);
  Key key[kSlots], by[kSlots];  // 0: not eligible
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int e = first + i;
    key[i] = by[i] = 0;
    if (i >= per || e >= c.E) continue;
    const double v = deciding<double>(l[i], s[i], bias, bias ? bias[e] : 0.f);
    key[i] = K_::of(v);
    by[i] = grouping<double>(l[i], s[i], v, !bias && c.group_score == MOE_GROUP_TOP2);
  }
  if (c.n_groups > 1) {
    Key mine;
    const unsigned kept = kept_groups<double>(by, first, c, mine);
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
      if (key[i] && !((kept >> ((first + i) / (c.E / c.n_groups))) & 1u)) key[i] = 0;
  }
  int chosen = 0;
  for (int k = 0; k < c.K; ++k) {
    Key m = 0;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) m = max(m, key[i]);
    const Key top = K_::largest(m);
    unsigned e = 0x7fffffffu;
#pragma unroll
    for (int i = kSlots - 1; i >= 0; --i)
      if (key[i] == top) e = first + i;
    e = __reduce_min_sync(kAll, e);
    if (lane == k) chosen = static_cast<int>(e);
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
      if (first + i == static_cast<int>(e)) key[i] = 0;
  }
  return chosen;
}

// A warp's keys (lane's run: [8 lane, + 8)), and the candidates' places among them in the experts' order.
struct Candidates {
  alignas(16) float key[32 * kSlots];
  alignas(16) float cand[32];
  int at[32];
};

// The token's choice in f32, made again in 64 bits where that may differ: each lane's expert, its logit and its place
// (K or more: not chosen).  False: neither decides (two groups' scores too near, infinite biases, more than 32
// candidates that differ by nothing).
template <typename LT>
__device__ __forceinline__ bool choose32(const LT* row, const float (&l)[kSlots], const float (&s)[kSlots], float m,
                                         int first, int per, const float* bias, const SelectCfg& c, Candidates& cand,
                                         int& expert, float& logit, int& rank) {
  using K_ = Keys<float>;
  const int lane = threadIdx.x & 31;
  const bool by_score = !bias && c.group_score == MOE_GROUP_TOP2;
  const int have = min(max(c.E - first, 0), per);
  uint32_t key[kSlots], by[kSlots];  // 0: not eligible
  float v[kSlots], b[kSlots] = {};
  float big = 1.f;  // largest |key|
  if (bias) load_run(bias, first, per, c.E, b);
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    v[i] = deciding<float>(l[i], s[i], bias, b[i]);
    key[i] = i < have ? K_::of(v[i]) : 0u;
    by[i] = by_score ? (i < have ? grouping<float>(l[i], s[i], v[i], true) : 0u) : key[i];
    big = fmaxf(big, v[i] == -INFINITY ? 0.f : fabsf(v[i]));
  }
  // keys that are logits are compared exactly, without a margin
  float rounding = kStep, margin = 0.f;
  if (bias) {
    rounding = __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(big))) * kStep;
    margin = 2.f * (kErr + rounding);
    if (!(rounding < 1.f)) return false;  // infinite or enormous biases
  }
  if (c.n_groups > 1) {
    uint32_t mine;
    const unsigned kept = kept_groups<float>(by, first, c, mine);
    if (c.topk_groups < c.n_groups && (bias || by_score)) {
      // the last group kept against the first one dropped: twice a sum of two keys' errors, and its rounding
      const bool in = (kept >> lane) & 1u;
      const uint32_t lo = __reduce_min_sync(kAll, in ? mine : 0xffffffffu);
      const uint32_t hi = __reduce_max_sync(kAll, lane < c.n_groups && !in ? mine : 0u);
      const float gap = K_::value(lo) - K_::value(hi);
      if (hi > K_::kMinusInf && !(gap > 4.f * (kErr + 2.f * rounding))) return false;
    }
    if (c.E % 32 == 0 && 32 % c.n_groups == 0) {
      const bool in = (kept >> (lane * c.n_groups >> 5)) & 1u;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) key[i] = in ? key[i] : 0;
    } else {
      const int gs = c.E / c.n_groups;
#pragma unroll
      for (int i = 0; i < kSlots; ++i)
        if (key[i] && !((kept >> ((first + i) / gs)) & 1u)) key[i] = 0;
    }
  }
  // The K-th largest of the lanes' largest keys, equal ones counted once, is a bound: K keys at least are not under it
  // (1 where fewer lanes have a key).
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) top = max(top, key[i]);
  const uint32_t largest = K_::largest(top);
  uint32_t bound = largest;
  for (int k = 1; k < c.K && bound; ++k) {
    top = top == bound ? 0u : top;
    bound = K_::largest(top);
  }
  bound = max(bound, 1u);
  // Candidates: the keys not under the bound, and those within the margin (and the subtraction's rounding) of it
  unsigned mine;
  int before, n;
  uint32_t least;
  auto count = [&]() {
    least = bound;
    if (margin > 0.f && bound > K_::kMinusInf) least = K_::of(K_::value(bound) - 2.f * margin);
    mine = 0;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) mine |= (key[i] >= least ? 1u : 0u) << i;
    before = __popc(mine);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kAll, before, o);
      if (lane >= o) before += v;
    }
    n = __shfl_sync(kAll, before, 31);
    before -= __popc(mine);
  };
  count();
  if (n > 32) {  // many choices of many lanes, or ties: a higher bound that still leaves K keys
    uint32_t low = bound, high = largest;
    while (low < high) {  // K keys are not under low
      const uint32_t mid = low + (high - low + 1) / 2;
      int not_under = 0;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) not_under += key[i] >= mid;
      not_under = __reduce_add_sync(kAll, not_under);
      if (not_under < c.K) {
        high = mid - 1;
      } else {
        low = mid;
        if (not_under == c.K) break;
      }
    }
    bound = low;
    count();
    if (n > 32) return false;
  }
  *reinterpret_cast<float4*>(&cand.key[lane * kSlots]) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(&cand.key[lane * kSlots + 4]) = make_float4(v[4], v[5], v[6], v[7]);
#pragma unroll
  for (int i = 0; i < kSlots; ++i)
    if ((mine >> i) & 1u) cand.at[before + __popc(mine & ((1u << i) - 1u))] = lane * kSlots + i;
  __syncwarp();
  const bool is = lane < n;
  const int at = is ? cand.at[lane] : 0;
  const float mv = cand.key[at];
  expert = (at / kSlots) * per + at % kSlots;
  logit = load_logit(row + expert);
  cand.cand[lane] = is ? mv : -INFINITY;
  __syncwarp();
  rank = 0;
  int near = 0;  // itself counts
  for (int i = 0; i < n; i += 4) {
    const float4 o4 = *reinterpret_cast<const float4*>(&cand.cand[i]);
    const float o[4] = {o4.x, o4.y, o4.z, o4.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      rank += o[j] > mv || (o[j] == mv && i + j < lane);
      near += fabsf(o[j] - mv) <= margin;
    }
  }
  if (margin > 0.f && __any_sync(kAll, is && near > 1 && rank < c.K)) {
    double sum = 1.0;
    if (c.scoring == MOE_GATING_SOFTMAX) {
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < kSlots; ++i) sum += score_term<false, false, double>(l[i], m);
      sum = warp_add(sum);
    }
    double exact = c.scoring == MOE_GATING_SOFTMAX ? score_term<false, false, double>(logit, m) / sum
                                                   : score_term<true, false, double>(logit, m);
    exact = deciding<double>(logit, exact, true, bias[expert]);
    const unsigned long long mine64 = Keys<double>::of(exact);
    rank = 0;
    for (int i = 0; i < n; ++i) {
      const unsigned long long o = __shfl_sync(kAll, mine64, i);
      rank += o > mine64 || (o == mine64 && i < lane);
    }
  }
  if (!is) rank = 32;
  return true;
}

template <typename LT>
__global__ void __launch_bounds__(32 * kWarpsPerCta)
    select_kernel(const LT* logits, long long stride, const float* bias, SelectCfg c,
                  int32_t* ids, float* w, float* scores) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  const long long t = static_cast<long long>(blockIdx.x) * kWarpsPerCta + warp;
  if (t >= c.T) return;
  __shared__ Candidates cand[kWarpsPerCta];
  const int E = c.E, K = c.K, per = (E + 31) / 32, first = lane * per;
  const LT* row = logits + t * stride;
  float l[kSlots], s[kSlots];
  load_run(row, first, per, E, l);
#pragma unroll
  for (int i = 0; i < kSlots; ++i) s[i] = 0.f;
  const bool softmax = c.scoring == MOE_GATING_SOFTMAX;
  const float m = softmax ? row_max(l) : 0.f;
  if (scores) {
    scores_of<float, false>(l, m, c.scoring, s);
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
      if (i < per && first + i < E) scores[t * E + first + i] = s[i];
  } else if (bias || (c.n_groups > 1 && c.group_score == MOE_GROUP_TOP2)) {
    scores_of<float, true>(l, m, c.scoring, s);
  }
  int e, place;
  float x;
  if (!choose32(row, l, s, m, first, per, bias, c, cand[warp], e, x, place)) {
    e = choose64(row, bias, c);
    place = lane;
    x = lane < K ? load_logit(row + e) : 0.f;
  }
  // the chosen scores again, from their logits: over their sum, or a softmax's own
  float sum = 0.f, v = 0.f;
  if (c.renorm) {
    v = shifted_score(x, place < K, softmax);
    sum = warp_add(v);
  } else {
    if (softmax) {
#pragma unroll
      for (int i = 0; i < kSlots; ++i)
        if (!(l[i] == -INFINITY)) sum += expf(l[i] - m);
      sum = warp_add(sum);
    }
    if (place < K) v = x == -INFINITY ? 0.f : softmax ? expf(x - m) : 1.f / (1.f + expf(-x));
  }
  if (place < K) {
    ids[t * K + place] = e;
    if (softmax || c.renorm) v = sum == 0.f ? 0.f : v / sum;
    w[t * K + place] = c.scale * v;
  }
}

template <typename LT>
__global__ void __launch_bounds__(32 * kWarpsPerCta)
    select_backward_kernel(const LT* logits, long long stride, const int32_t* ids,
                           const float* d_w, const float* d_scores, SelectCfg c,
                           LT* d_logits, int* status) {
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
  const bool softmax = c.scoring == MOE_GATING_SOFTMAX;
  scores_of<float, false>(l, softmax ? row_max(l) : 0.f, c.scoring, s);
  bool far = false;  // of the chosen scores one is too small for what follows in f32 (or masked)
  if (c.renorm) {
    float my_s = 0.f;
    for (int k = 0; k < K; ++k) {
      const int id = __shfl_sync(kAll, my_id, k);
      const float v = of_expert(s, max(id, 0));
      if (lane == k && id >= 0) my_s = v;
    }
    far = __any_sync(kAll, my_id >= 0 && my_s < 0x1p-60f);
    if (!far) {
      const float sum = warp_add(my_s);
      const float mean = warp_add(my_id >= 0 ? my_dw * my_s : 0.f);
      my_dw = sum == 0.f ? 0.f : (my_dw - mean / sum) / sum;
    } else {  // my_dw becomes the slot's n_k (dw_k - sum_j dw_j n_j), the product s_k ds_k
      float my_l = 0.f;
      for (int k = 0; k < K; ++k) {
        const int id = __shfl_sync(kAll, my_id, k);
        const float v = of_expert(l, max(id, 0));
        if (lane == k) my_l = v;
      }
      float n = shifted_score(my_l, my_id >= 0, softmax);
      const float sum = warp_add(n);
      n = sum == 0.f ? 0.f : n / sum;
      const float mean = warp_add(my_id >= 0 ? my_dw * n : 0.f);
      my_dw = n * (my_dw - mean);
    }
  }
  float part[kSlots];  // far: the weights' part of s_e ds_e
#pragma unroll
  for (int i = 0; i < kSlots; ++i) part[i] = 0.f;
  for (int k = 0; k < K; ++k) {  // in slot order, so that an expert named twice sums the same way every time
    const int id = __shfl_sync(kAll, my_id, k);
    const float d = __shfl_sync(kAll, my_dw, k);
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
      if (lane + 32 * i == id) {
        if (far)
          part[i] += d;
        else
          ds[i] += d;
      }
  }
  float dot = 0.f;  // (far: the weights' part of it is 0)
  if (softmax) {
#pragma unroll
    for (int i = 0; i < kSlots; ++i) dot += ds[i] * s[i];
    dot = warp_add(dot);
  }
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int e = lane + 32 * i;
    if (e < E)  // (1 - s_e with the precision of s_e: the difference of f32 numbers has none left for logits above 16)
      store_grad(d_logits + t * E + e,
                 softmax ? part[i] + s[i] * (ds[i] - dot) : (part[i] + ds[i] * s[i]) * (1.f / (1.f + expf(l[i]))));
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
