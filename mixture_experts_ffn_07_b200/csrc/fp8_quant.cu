// Quantisation to block-scaled 8-bit floats (fp8.cuh): activation rows with one scale per 128 values, weight
// matrices with one scale per 128 x 128 block, and the combine of the 8-bit experts' slot rows.
#include <type_traits>

#include "fp8.cuh"

namespace moe {

namespace {

constexpr int kRowThreads = 256;
constexpr int kTileBlocks = 8;   // blocks of 128 along a row per CTA
// Rows per CTA: one batch of loads, and scales in whole sectors.  Tiles of 32 rows, whose scales fill whole lines, measured
// slower at every size (8192 x 7168: 33.7 us against 30.4; scattered to the experts, 144 x 2816: 15.7 against 7.7).
constexpr int kTileRows = 8;
constexpr int kHalfWarps = kRowThreads / 16;
constexpr int kRowsPerPass = kHalfWarps / kTileBlocks;
constexpr int kMaxSlots = 32;

// Eight values as loaded.
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float4 a, b;
};
template <>
struct Raw<__nv_bfloat16> {
  uint4 a;
};
__device__ __forceinline__ Raw<float> load8(const float* p, int left) {
  Raw<float> r;
  r.a = left > 0 ? *reinterpret_cast<const float4*>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
  r.b = left > 4 ? *(reinterpret_cast<const float4*>(p) + 1) : make_float4(0.f, 0.f, 0.f, 0.f);
  return r;
}
__device__ __forceinline__ Raw<__nv_bfloat16> load8(const __nv_bfloat16* p, int left) {
  Raw<__nv_bfloat16> r;
  r.a = left > 0 ? *reinterpret_cast<const uint4*>(p) : make_uint4(0u, 0u, 0u, 0u);
  return r;
}
__device__ __forceinline__ void values(const Raw<float>& r, float (&v)[8]) {
  v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
  v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
}
__device__ __forceinline__ void values(const Raw<__nv_bfloat16>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_bits_to_f32(w[i] & 0xFFFFu);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
// Largest |x| as f32 bits (NaN is largest).
__device__ __forceinline__ uint32_t amax_bits(const Raw<float>& r) {
  float v[8];
  values(r, v);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}
__device__ __forceinline__ uint32_t amax_bits(const Raw<__nv_bfloat16>& r) {
  // |bf16| patterns order like the numbers: two 16-bit maxima at a time
  const uint32_t m = __vmaxu2(__vmaxu2(r.a.x & 0x7fff7fffu, r.a.y & 0x7fff7fffu),
                              __vmaxu2(r.a.z & 0x7fff7fffu, r.a.w & 0x7fff7fffu));
  return max(m & 0xffff0000u, m << 16);
}
template <typename T>
__device__ __forceinline__ uint2 codes8(const Raw<T>& r, float inv, int fmt) {
  float v[8];
  values(r, v);
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = fp8_pack2(v[2 * i] * inv, v[2 * i + 1] * inv, fmt);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// A CTA codes kTileRows rows x kTileBlocks blocks; a half-warp holds one block (eight values a lane) of four
// rows.  The four maxima are found together (each step over the lanes halves the rows that a lane keeps: five shuffles
// for four rows), then each quarter of the half-warp makes one row's scale, so the divisions are done once for four
// rows, and hands its inverse to the others.  Scales go through shared memory: the output is [block, row], and a CTA
// writes runs of kTileRows.  C is a multiple of 32, so eight values are all inside the row or all outside.
// `sc`: [kTileBlocks][kTileRows + 1] floats of shared memory.  Copies of each row's codes go out too, to rows
// dest[row of the tile][0, copies) of to (-1: none).
constexpr int kBatch = kTileRows / kRowsPerPass;
static_assert(kBatch == 4, "one row per quarter of a half-warp");
template <typename XT>
struct Coding {  // a thread's values, and the inverse scale of row hl / 4 of its half-warp
  Raw<XT> v[kBatch];
  float inv;
};
template <typename XT>
__device__ __forceinline__ Coding<XT> load_rows(const XT* x, long long stride, int R, int C, int fmt,
                                                int pow2, long long row_tile, int block_tile, float* sc) {
  const int hw = threadIdx.x >> 4, hl = threadIdx.x & 15;
  const int bl = hw % kTileBlocks;
  const int col = (block_tile * kTileBlocks + bl) * kFp8Block + hl * 8;
  const int left = C - col;
  const long long row0 = row_tile * kTileRows;
  Coding<XT> k;
  uint32_t m[kBatch];
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const long long r = row0 + u * kRowsPerPass + hw / kTileBlocks;
    k.v[u] = load8(x + (r < R ? r * stride + col : 0), r < R ? left : 0);
  }
#pragma unroll
  for (int u = 0; u < kBatch; ++u) m[u] = amax_bits(k.v[u]);
  const bool up8 = hl & 8, up4 = hl & 4;  // lane hl ends with row hl / 4
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint32_t give = up8 ? m[u] : m[u + 2], keep = up8 ? m[u + 2] : m[u];
    m[u] = max(keep, __shfl_xor_sync(0xffffffffu, give, 8));
  }
  uint32_t top = max(up4 ? m[1] : m[0], __shfl_xor_sync(0xffffffffu, up4 ? m[0] : m[1], 4));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  float scale;
  fp8_scale(top, fmt, pow2 != 0, scale, k.inv);
  if ((hl & 3) == 0) sc[bl * (kTileRows + 1) + (hl >> 2) * kRowsPerPass + hw / kTileBlocks] = scale;
  return k;
}
template <typename XT>
__device__ __forceinline__ void store_rows(const Coding<XT>& k, int R, int C, int fmt, uint8_t* q,
                                           float* scales, long long row_tile, int block_tile,
                                           const float* sc, uint8_t* to = nullptr, const int* dest = nullptr,
                                           int copies = 0) {
  const int hw = threadIdx.x >> 4, hl = threadIdx.x & 15;
  const int col = (block_tile * kTileBlocks + hw % kTileBlocks) * kFp8Block + hl * 8;
  const long long row0 = row_tile * kTileRows;
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const float my_inv = __shfl_sync(0xffffffffu, k.inv, (threadIdx.x & 16) + 4 * u);
    const long long r = row0 + u * kRowsPerPass + hw / kTileBlocks;
    if (r < R && col < C) {
      const uint2 code = codes8(k.v[u], my_inv, fmt);
      if (q) *reinterpret_cast<uint2*>(q + r * C + col) = code;
      const int* d = dest + static_cast<int>(r - row0) * copies;
      for (int c = 0; c < copies; ++c)
        if (d[c] >= 0) *reinterpret_cast<uint2*>(to + static_cast<long long>(d[c]) * C + col) = code;
    }
  }
  __syncthreads();
  const int nkb = (C + kFp8Block - 1) / kFp8Block;
  for (int i = threadIdx.x; i < kTileBlocks * kTileRows; i += kRowThreads) {
    const int b = i / kTileRows, r = i % kTileRows;
    if (block_tile * kTileBlocks + b < nkb && row0 + r < R)
      scales[static_cast<long long>(block_tile * kTileBlocks + b) * R + row0 + r] = sc[b * (kTileRows + 1) + r];
  }
}

// early: the launch before this one (the permutation) waited for everything before it, and nothing here depends on it:
// the coding runs beside it and ends after it (a pass of 100 tokens on 64 experts of 2816 x 704: 88.8 -> 86.8 us).
template <typename XT>
__global__ void __launch_bounds__(kRowThreads)
    fp8_rows_kernel(const XT* x, long long stride, int R, int C, int fmt, int pow2,
                    uint8_t* q, float* scales, bool early) {
  __shared__ float sc[kTileBlocks * (kTileRows + 1)];
  pdl_trigger();
  if (!early) pdl_wait();
  const Coding<XT> k = load_rows(x, stride, R, C, fmt, pow2, blockIdx.x, blockIdx.y, sc);
  store_rows(k, R, C, fmt, q, scales, blockIdx.x, blockIdx.y, sc);
  if (early) pdl_wait();
}

// The activations of a large batch in expert order: x is read once, and each token's codes written to the rows of its
// pairs (coding first and copying rows after read them back K times: 181 us for 8192 tokens of 7168, 8 experts each).
// The places are read ahead of the rows, all at once (one by one behind each row they took most of the time of a batch
// of a few hundred tokens).  ids, pos: [R, K], the pairs' experts (a copy exists for those in [0, E)) and rows.
template <typename XT>
__global__ void __launch_bounds__(kRowThreads)
    fp8_scatter_kernel(const XT* x, int R, int C, uint8_t* q, float* scales,
                       uint8_t* to, const int32_t* ids, const int32_t* pos, int K,
                       int E) {
  __shared__ float sc[kTileBlocks * (kTileRows + 1)];
  __shared__ int dest[kTileRows * kMaxSlots];
  pdl_trigger();
  // x was complete before the permutation let this launch start; only the places have to be waited for
  const Coding<XT> coding = load_rows(x, static_cast<long long>(C), R, C, MOE_E4M3, 0, blockIdx.x, blockIdx.y, sc);
  pdl_wait();
  const long long first = static_cast<long long>(blockIdx.x) * kTileRows * K;
  const int n = static_cast<int>(min(static_cast<long long>(kTileRows) * K, static_cast<long long>(R) * K - first));
  for (int i = threadIdx.x; i < n; i += kRowThreads) {
    const int id = ids[first + i], at = pos[first + i];  // (a pair of no expert has no row: nothing wrote its place)
    dest[i] = id >= 0 && id < E ? at : -1;
  }
  __syncthreads();
  store_rows(coding, R, C, MOE_E4M3, q, scales, blockIdx.x, blockIdx.y, sc, to, dest, K);
}

// Small batches of the 8-bit experts in one launch: CTA 0 sorts the (at most 256) pairs by expert, the others code x.
// The sort is permute.cu's stable counting sort with one pair a thread: a warp ranks equal experts with
// __match_any_sync, warps and experts are scanned through shared memory.
constexpr int kFrontPairs = kRowThreads;
constexpr int kFrontExperts = 256;
template <typename XT>
__global__ void __launch_bounds__(kRowThreads)
    fp8_front_kernel(const XT* x, int R, int C, uint8_t* q, float* scales,
                     int row_tiles, const int32_t* ids, int P, int E, int32_t* counts,
                     int32_t* offsets, int32_t* sorted_pairs,
                     int32_t* pair_pos, int* status) {
  __shared__ union {
    float sc[kTileBlocks * (kTileRows + 1)];
    int hist[kRowThreads / 32][kFrontExperts];
  } sm;
  __shared__ int warp_sum_[kRowThreads / 32];
  pdl_trigger();
  if (blockIdx.x > 0) {
    pdl_wait();
    const int b = blockIdx.x - 1;
    const Coding<XT> k = load_rows(x, static_cast<long long>(C), R, C, MOE_E4M3, 0, b % row_tiles, b / row_tiles, sm.sc);
    store_rows(k, R, C, MOE_E4M3, q, scales, b % row_tiles, b / row_tiles, sm.sc);
    return;
  }
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
#pragma unroll
  for (int w = 0; w < kRowThreads / 32; ++w) sm.hist[w][t] = 0;
  pdl_wait();
  int e = t < P ? ids[t] : -1;
  if (t < P && (e < 0 || e >= E)) {
    record_status(status, MOE_ERR_DEVICE_INDEX);
    e = -1;
  }
  __syncthreads();
  const unsigned peers = __match_any_sync(0xffffffffu, e);
  const int rank = __popc(peers & ((1u << lane) - 1u));
  if (e >= 0 && rank == 0) sm.hist[warp][e] = __popc(peers);
  __syncthreads();
  int total = 0;  // thread t: expert t's pairs, and where each warp's begin among them
#pragma unroll
  for (int w = 0; w < kRowThreads / 32; ++w) {
    const int c = sm.hist[w][t];
    sm.hist[w][t] = total;
    total += c;
  }
  int incl = total;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) warp_sum_[warp] = incl;
  __syncthreads();
  int base = incl - total;
  for (int w = 0; w < warp; ++w) base += warp_sum_[w];
#pragma unroll
  for (int w = 0; w < kRowThreads / 32; ++w) sm.hist[w][t] += base;
  if (t < E) {
    counts[t] = total;
    offsets[t] = base;
    if (t == E - 1) offsets[E] = base + total;
  }
  __syncthreads();
  if (e >= 0) {
    const int pos = sm.hist[warp][e] + rank;
    sorted_pairs[pos] = t;
    pair_pos[t] = pos;
  }
}

// One CTA per 128 x 128 block of a [G, N, K] stack, its values held in registers between the maximum and the
// codes, so that they are read once.
template <typename XT>
__global__ void __launch_bounds__(kRowThreads)
    fp8_blocks_kernel(const XT* w, int N, int K, int fmt, int pow2, uint8_t* q,
                      float* scales) {
  __shared__ uint32_t part[kRowThreads / 32];
  const int hw = threadIdx.x >> 4, hl = threadIdx.x & 15;
  const int kb = blockIdx.x, nb = blockIdx.y;
  const long long g = blockIdx.z;
  const int col = kb * kFp8Block + hl * 8;
  const int left = K - col;
  pdl_trigger();
  pdl_wait();
  constexpr int kRows = kFp8Block / kHalfWarps;
  Raw<XT> v[kRows];
  uint32_t m = 0;
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int n = nb * kFp8Block + u * kHalfWarps + hw;
    v[u] = load8(w + (n < N ? (g * N + n) * K + col : 0), n < N ? left : 0);
  }
#pragma unroll
  for (int u = 0; u < kRows; ++u) m = max(m, amax_bits(v[u]));
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kRowThreads / 32; ++i) m = max(m, part[i]);
  float scale, inv;
  fp8_scale(m, fmt, pow2 != 0, scale, inv);
  if (threadIdx.x == 0) scales[(g * gridDim.y + nb) * gridDim.x + kb] = scale;
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int n = nb * kFp8Block + u * kHalfWarps + hw;
    if (n < N && left > 0) *reinterpret_cast<uint2*>(q + (g * N + n) * K + col) = codes8(v[u], inv, fmt);
  }
}

// 16 bytes of a slot row, as floats, and of an output row.
template <typename T>
struct Slots;
template <>
struct Slots<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void values(const uint4& r, float (&v)[N]) {
    v[0] = __uint_as_float(r.x); v[1] = __uint_as_float(r.y); v[2] = __uint_as_float(r.z); v[3] = __uint_as_float(r.w);
  }
};
template <>
struct Slots<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void values(const uint4& r, float (&v)[N]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
template <>
struct Slots<__half> {  // kSlotsF16, without the power of two
  static constexpr int N = 8;
  static __device__ __forceinline__ void values(const uint4& r, float (&v)[N]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
};
template <int N>
__device__ __forceinline__ void store_row(float* p, const float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
template <int N>
__device__ __forceinline__ void store_row(__nv_bfloat16* p, const float (&v)[N]) {
  uint32_t w[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&a);
  }
#pragma unroll
  for (int i = 0; i < N / 2; i += 2) *reinterpret_cast<uint2*>(p + 2 * i) = make_uint2(w[i], w[i + 1]);
}

// out[t] = sum_k w[t,k] y[t*K+k] in slot order in f32 (w == nullptr: 1; slots whose expert id is outside [0, E)
// hold no row and count nothing), + y_shared[t].  A CTA has one token and 256 threads' worth of its outputs, 16 bytes
// of each slot row a thread; the rows are loaded beside the ids and weights, not after them (one of no expert is
// memory that nobody wrote, and is dropped).  Of f16 rows the powers of two are asked for before the rows, each by one
// thread of the CTA, and multiplied into the weight: asked for after them, and into every value, 8192 tokens of 7168 with
// 8 slots took 285 us, this takes 220 (bf16 rows, without them, 188).
constexpr int kCombineThreads = 256;
template <typename T, typename OT>
__global__ void __launch_bounds__(kCombineThreads)
    combine_ids_kernel(const T* y, const float* w, const int32_t* ids,
                       const float* y_shared, int K, int E, int H, OT* out) {
  constexpr int N = Slots<T>::N;
  constexpr bool kScaled = std::is_same<T, __half>::value;
  constexpr int kAcross = kCombineThreads * N / kFp8Block;  // blocks of 128 outputs
  __shared__ float weight[kMaxSlots];
  __shared__ int valid[kMaxSlots];
  __shared__ float scale[kScaled ? kMaxSlots : 1][kAcross];
  const long long t = blockIdx.x;
  const int c = (blockIdx.y * kCombineThreads + threadIdx.x) * N;
  const bool in = c < H;
  pdl_trigger();
  pdl_wait();
  const T* row = y + t * K * H + (in ? c : 0);
  float s[2] = {0.f, 0.f}, my_w = 1.f;
  int id = -1;
  if (threadIdx.x < K) {
    id = ids[t * K + threadIdx.x];
    if (w) my_w = w[t * K + threadIdx.x];
  }
  const int blocks = (H + kFp8Block - 1) / kFp8Block;
  if (kScaled) {  // the powers of two of the CTA's columns
    const float* from = reinterpret_cast<const float*>(y + static_cast<long long>(gridDim.x) * K * H) + t * K * blocks;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = threadIdx.x + j * kCombineThreads, b = blockIdx.y * kAcross + i % kAcross;
      if (i < K * kAcross && b < blocks) s[j] = from[i / kAcross * blocks + b];
    }
  }
  uint4 r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < K) r[j] = *reinterpret_cast<const uint4*>(row + static_cast<long long>(j) * H);
  if (threadIdx.x < K) {
    valid[threadIdx.x] = id >= 0 && id < E;
    weight[threadIdx.x] = my_w;
  }
  if (kScaled)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = threadIdx.x + j * kCombineThreads;
      if (i < K * kAcross) scale[i / kAcross][i % kAcross] = s[j];
    }
  float acc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;
  __syncthreads();
  if (!in) return;
  for (int k0 = 0; k0 < K; k0 += 8) {
    if (k0 > 0)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (k0 + j < K) r[j] = *reinterpret_cast<const uint4*>(row + static_cast<long long>(k0 + j) * H);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (k0 + j < K && valid[k0 + j]) {
        float v[N];
        Slots<T>::values(r[j], v);
        const float ww = kScaled ? weight[k0 + j] * scale[k0 + j][threadIdx.x * N / kFp8Block] : weight[k0 + j];
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += ww * v[i];
      }
  }
  if (y_shared) {
    const float* ys = y_shared + t * H + c;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(ys + i);
      acc[i] += v.x;
      acc[i + 1] += v.y;
      acc[i + 2] += v.z;
      acc[i + 3] += v.w;
    }
  }
  store_row<N>(out + t * H + c, acc);
}

}  // namespace

static dim3 row_grid(int64_t R, int C) {
  constexpr int kAcross = kFp8Block * kTileBlocks;
  return dim3(static_cast<unsigned>((R + kTileRows - 1) / kTileRows), (C + kAcross - 1) / kAcross);
}

cudaError_t launch_fp8_rows(const Ctx& c, const void* x, int x_dtype, int64_t stride, int64_t R, int C, int fmt,
                            bool pow2, void* q, float* scales, bool early) {
  KernelScope ks(c, "fp8_quantize");
  if (x_dtype == MOE_F32)
    return launch_kernel(c, fp8_rows_kernel<float>, row_grid(R, C), dim3(kRowThreads), 0, static_cast<const float*>(x),
                         static_cast<long long>(stride), static_cast<int>(R), C, fmt, pow2 ? 1 : 0,
                         static_cast<uint8_t*>(q), scales, early);
  return launch_kernel(c, fp8_rows_kernel<__nv_bfloat16>, row_grid(R, C), dim3(kRowThreads), 0,
                       static_cast<const __nv_bfloat16*>(x), static_cast<long long>(stride), static_cast<int>(R), C,
                       fmt, pow2 ? 1 : 0, static_cast<uint8_t*>(q), scales, early);
}

cudaError_t launch_fp8_scatter(const Ctx& c, const void* x, int x_dtype, int R, int C, void* q, float* scales,
                               const int32_t* ids, const int32_t* pair_pos, int K, int E, void* x_perm) {
  if (K > kMaxSlots) return cudaErrorInvalidValue;
  KernelScope ks(c, "fp8_scatter");
  if (x_dtype == MOE_F32)
    return launch_kernel(c, fp8_scatter_kernel<float>, row_grid(R, C), dim3(kRowThreads), 0,
                         static_cast<const float*>(x), R, C, static_cast<uint8_t*>(q), scales,
                         static_cast<uint8_t*>(x_perm), ids, pair_pos, K, E);
  return launch_kernel(c, fp8_scatter_kernel<__nv_bfloat16>, row_grid(R, C), dim3(kRowThreads), 0,
                       static_cast<const __nv_bfloat16*>(x), R, C, static_cast<uint8_t*>(q), scales,
                       static_cast<uint8_t*>(x_perm), ids, pair_pos, K, E);
}

bool fp8_front_fits(int P, int E) { return P <= kFrontPairs && E <= kFrontExperts; }

cudaError_t launch_fp8_front(const Ctx& c, const void* x, int x_dtype, int R, int C, void* q, float* scales,
                             const int32_t* ids, int P, int E, int32_t* counts, int32_t* offsets,
                             int32_t* sorted_pairs, int32_t* pair_pos) {
  const int nkb = (C + kFp8Block - 1) / kFp8Block;
  const int row_tiles = (R + kTileRows - 1) / kTileRows;
  const dim3 grid(1 + row_tiles * ((nkb + kTileBlocks - 1) / kTileBlocks));
  KernelScope ks(c, "fp8_front");
  if (x_dtype == MOE_F32)
    return launch_kernel(c, fp8_front_kernel<float>, grid, dim3(kRowThreads), 0, static_cast<const float*>(x), R, C,
                         static_cast<uint8_t*>(q), scales, row_tiles, ids, P, E, counts, offsets, sorted_pairs, pair_pos,
                         c.status);
  return launch_kernel(c, fp8_front_kernel<__nv_bfloat16>, grid, dim3(kRowThreads), 0,
                       static_cast<const __nv_bfloat16*>(x), R, C, static_cast<uint8_t*>(q), scales, row_tiles, ids, P,
                       E, counts, offsets, sorted_pairs, pair_pos, c.status);
}

cudaError_t launch_fp8_blocks(const Ctx& c, const void* w, int w_dtype, int G, int N, int K, int fmt, bool pow2,
                              void* q, float* scales) {
  const dim3 grid((K + kFp8Block - 1) / kFp8Block, (N + kFp8Block - 1) / kFp8Block, G);
  KernelScope ks(c, "fp8_quantize_weights");
  if (w_dtype == MOE_F32)
    return launch_kernel(c, fp8_blocks_kernel<float>, grid, dim3(kRowThreads), 0, static_cast<const float*>(w), N, K,
                         fmt, pow2 ? 1 : 0, static_cast<uint8_t*>(q), scales);
  return launch_kernel(c, fp8_blocks_kernel<__nv_bfloat16>, grid, dim3(kRowThreads), 0,
                       static_cast<const __nv_bfloat16*>(w), N, K, fmt, pow2 ? 1 : 0, static_cast<uint8_t*>(q),
                       scales);
}

template <typename T, typename OT>
static cudaError_t combine_ids_typed(const Ctx& c, const void* y, const float* w, const int32_t* ids, const float* ys,
                                     int T_, int K, int E, int H, void* out) {
  const int per = kCombineThreads * Slots<T>::N;
  KernelScope ks(c, "combine");
  return launch_kernel(c, combine_ids_kernel<T, OT>, dim3(T_, (H + per - 1) / per), dim3(kCombineThreads), 0,
                       static_cast<const T*>(y), w, ids, ys, K, E, H, static_cast<OT*>(out));
}

cudaError_t launch_combine_ids(const Ctx& c, const void* y_slots, int y_dtype, const float* w, const int32_t* ids,
                               const float* y_shared, int T, int K, int E, int H, void* out, int dtype) {
  if (K > kMaxSlots) return cudaErrorInvalidValue;
  if (dtype == MOE_F32) return combine_ids_typed<float, float>(c, y_slots, w, ids, y_shared, T, K, E, H, out);
  if (y_dtype == MOE_F32)
    return combine_ids_typed<float, __nv_bfloat16>(c, y_slots, w, ids, y_shared, T, K, E, H, out);
  if (y_dtype == kSlotsF16) return combine_ids_typed<__half, __nv_bfloat16>(c, y_slots, w, ids, y_shared, T, K, E, H, out);
  return combine_ids_typed<__nv_bfloat16, __nv_bfloat16>(c, y_slots, w, ids, y_shared, T, K, E, H, out);
}

}  // namespace moe
