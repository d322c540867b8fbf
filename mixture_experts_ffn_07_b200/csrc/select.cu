// Expert selection from router logits, and its gradient.
//
// Forward, per token (a warp): scores s_e = softmax(l)_e or 1 / (1 + e^-l_e); the keys that decide are the
// logits when there is no balance bias (the scores' own order) and s_e + b_e otherwise; optional groups of
// experts scored by their largest key or by the sum of their two largest s_e + b_e, the best groups kept; the
// top_k largest keys in order, lower index on ties; weights scale * s_e (/ their sum).  The bias moves the
// choice and never the weights (the selection rule of auxiliary-loss-free balancing).
//
// Keys with a bias are compared in 64 bits: with thousands of tokens and hundreds of experts, scores that f32
// cannot tell apart do occur next to the border, and the choice must not depend on rounding.
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

// Order-preserving integer keys (a > b as numbers iff key(a) > key(b), -0 as +0); NaN counts as -inf.  Zero is
// below the key of -inf.
__device__ __forceinline__ unsigned long long key_of(double v) {
  if (!(v == v)) v = -INFINITY;
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(v == 0.0 ? 0.0 : v));
  return (u >> 63) ? ~u : (u | (1ull << 63));
}

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
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

__device__ __forceinline__ float exp_of(float v) { return expf(v); }
__device__ __forceinline__ double exp_of(double v) { return exp(v); }

// Scores of the lane's experts from its logits (entries beyond E: -inf).  A row of -inf alone scores 0.
template <typename F>
__device__ __forceinline__ void scores_of(const float (&l)[kSlots], int E, int scoring, F (&s)[kSlots]) {
  const int lane = threadIdx.x & 31;
  if (scoring == MOE_GATING_SIGMOID) {
#pragma unroll
    for (int i = 0; i < kSlots; ++i) s[i] = lane + 32 * i < E ? F(1) / (F(1) + exp_of(-static_cast<F>(l[i]))) : F(0);
    return;
  }
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) m = fmaxf(m, l[i]);
  m = warp_max(m);
  F sum = 0;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    s[i] = lane + 32 * i < E && !(l[i] == -INFINITY) ? exp_of(static_cast<F>(l[i]) - static_cast<F>(m)) : F(0);
    sum += s[i];
  }
  sum = warp_add(sum);
  const F inv = sum == F(0) ? F(0) : F(1) / sum;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) s[i] *= inv;
}

// Value that lane `expert % 32` holds for `expert`, in every lane.
template <typename F>
__device__ __forceinline__ F of_expert(const F (&v)[kSlots], int expert) {
  F mine = v[0];
#pragma unroll
  for (int i = 1; i < kSlots; ++i)
    if (expert >> 5 == i) mine = v[i];
  return __shfl_sync(kAll, mine, expert & 31);
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
  float l[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int e = lane + 32 * i;
    l[i] = e < E ? load_logit(logits + t * stride + e) : -INFINITY;
  }
  double s[kSlots];
  scores_of<double>(l, E, c.scoring, s);
  if (scores) {
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
      if (lane + 32 * i < E) scores[t * E + lane + 32 * i] = static_cast<float>(s[i]);
  }
  unsigned long long key[kSlots];  // 0: not eligible
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int e = lane + 32 * i;
    const bool masked = l[i] == -INFINITY;
    const double v = masked ? -INFINITY : (bias && e < E ? s[i] + static_cast<double>(bias[e]) : static_cast<double>(l[i]));
    key[i] = e < E ? key_of(v) : 0ull;
  }
  if (c.n_groups > 1) {
    const int gs = E / c.n_groups;
    unsigned long long mine = 0;  // lane g: the key of group g's score
    for (int g = 0; g < c.n_groups; ++g) {
      unsigned long long gk;
      if (c.group_score == MOE_GROUP_TOP2) {
        double a = -INFINITY, b = -INFINITY;  // the two largest s_e + b_e
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
          const int e = lane + 32 * i;
          if (e < E && e / gs == g && !(l[i] == -INFINITY)) {
            double v = s[i] + (bias ? static_cast<double>(bias[e]) : 0.0);
            if (!(v == v)) v = -INFINITY;
            if (v > a) {
              b = a;
              a = v;
            } else if (v > b) {
              b = v;
            }
          }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const double oa = __shfl_xor_sync(kAll, a, o), ob = __shfl_xor_sync(kAll, b, o);
          const double lo = fmin(a, oa);
          a = fmax(a, oa);
          b = fmax(lo, fmax(b, ob));
        }
        gk = key_of(gs > 1 ? (b == -INFINITY ? a : a + b) : a);
      } else {
        gk = 0;
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
          const int e = lane + 32 * i;
          if (e < E && e / gs == g) gk = max(gk, key[i]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) gk = max(gk, __shfl_xor_sync(kAll, gk, o));
      }
      if (lane == g) mine = gk;
    }
    // rank of lane g's group: the groups that score more, and the equal ones before it
    int rank = 0;
    for (int g = 0; g < c.n_groups; ++g) {
      const unsigned long long o = __shfl_sync(kAll, mine, g);
      rank += o > mine || (o == mine && g < lane);
    }
    const unsigned kept = __ballot_sync(kAll, lane < c.n_groups && rank < c.topk_groups);
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const int e = lane + 32 * i;
      if (e < E && !((kept >> (e / gs)) & 1u)) key[i] = 0;
    }
  }
  int my_e = 0;
  double my_s = 0;
  for (int k = 0; k < K; ++k) {
    unsigned long long bk = 0;
    int bi = 0;
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
      if (key[i] > bk) {
        bk = key[i];
        bi = i;
      }
    int be = lane + 32 * bi;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long ok = __shfl_xor_sync(kAll, bk, o);
      const int oe = __shfl_xor_sync(kAll, be, o);
      if (ok > bk || (ok == bk && oe < be)) {
        bk = ok;
        be = oe;
      }
    }
    const double v = of_expert(s, be);
    if (lane == k) {
      my_e = be;
      my_s = v;
    }
    if (lane == (be & 31)) {
#pragma unroll
      for (int i = 0; i < kSlots; ++i)
        if (i == be >> 5) key[i] = 0;
    }
  }
  const double sum = c.renorm ? warp_add(lane < K ? my_s : 0.0) : 1.0;
  if (lane < K) {
    ids[t * K + lane] = my_e;
    w[t * K + lane] = sum == 0.0 ? 0.f : static_cast<float>(static_cast<double>(c.scale) * my_s / sum);
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
  scores_of<float>(l, E, c.scoring, s);
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
    if (id >= 0 && lane == (id & 31)) {
#pragma unroll
      for (int i = 0; i < kSlots; ++i)
        if (i == id >> 5) ds[i] += d;
    }
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
