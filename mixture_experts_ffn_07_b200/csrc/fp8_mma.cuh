// Pieces shared by the two kernels of the block-scaled 8-bit product (fp8_gemm.cu, fp8_gemm_rows.cu): launch
// parameters, copies and matrix instructions, packed f32 arithmetic, tensor maps.
#pragma once

#include "fp8.cuh"

namespace moe {
namespace {

constexpr int WM = 128;            // weight rows that share a scale block
constexpr int KB = 128;            // k-block: values that share a scale, and bytes per shared-memory row
constexpr int W_BYTES = WM * KB;
constexpr int MAX_G = 256;
constexpr int THREADS = 384;       // four warps of copies, matrix instructions and scales, eight of the epilogue
constexpr int EPI_WARPS = 8;
constexpr int SMEM_MAX = 232448;
constexpr int TILE_ROWS = 128;     // rows of a tile of fp8_gemm_rows.cu

struct Params {
  const int32_t* offsets;
  int G, rows, N, K, n_tiles;
  const float* a_scale;         // [nkb, a_ld]
  long long a_ld;
  const int32_t* a_scale_map;   // row r uses scale column a_scale_map[r] / a_scale_div
  int a_scale_div;
  bool gather;                  // row r of A is row a_scale_map[r] / a_scale_div of the tensor (a_ld rows)
  bool early;                   // weights and offsets were complete before the launch before this one began
  int split, kb_per;            // CTAs of a cluster that share an item's k-blocks, and k-blocks of each
  const float* s0;
  const float* s1;
  uint32_t idesc;               // without N
  int act;
  uint8_t* out_q;
  float* out_qs;                // [ceil(N/128), rows]
  float* out_f32;
  __nv_bfloat16* out_bf16;
  __half* out_f16;              // with out_f16_scale [rows, n_tiles]: kSlotsF16
  float* out_f16_scale;
  const int32_t* row_map;
  const float* row_scale;
  bool wide;                    // outputs allow 32-byte stores
  int* status;
  long long wait_limit;
  int skip_stage;
};

__device__ __forceinline__ bool wait_cycles(uint64_t* bar, uint32_t parity, long long limit) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > limit) return false;
  return true;
}

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1,
                                            int c2, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_addr(smem_dst)),
      "l"(map), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// acc pair += value pair * scale pair (two f32 FMAs)
__device__ __forceinline__ void fma2(unsigned long long& acc, uint32_t v0, uint32_t v1, unsigned long long s) {
  unsigned long long v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(v0), "r"(v1));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(v), "l"(s));
}
__device__ __forceinline__ void split2(unsigned long long v, float& lo, float& hi) {
  uint32_t a, b;
  asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
  lo = __uint_as_float(a);
  hi = __uint_as_float(b);
}

__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(a) : "l"(b));
  return a;
}
__device__ __forceinline__ unsigned long long join2(float lo, float hi) {
  return static_cast<unsigned long long>(__float_as_uint(lo)) |
         (static_cast<unsigned long long>(__float_as_uint(hi)) << 32);
}

__device__ __forceinline__ void named_barrier(int id, int threads) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Every one of `threads` threads says ok.
__device__ __forceinline__ bool named_barrier_and(int id, int threads, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"(ok ? 1u : 0u)
      : "memory");
  return r != 0;
}

// act(g) = g / (1 + 2^(g (c0 + c1 g^2))) for both activations: SiLU has c0 = -log2(e), c1 = 0; GELU_TANH, since
// (1 + tanh z) / 2 = 1 / (1 + e^-2z), c0 = -2 log2(e) sqrt(2/pi), c1 = 0.044715 c0.  One form without a branch, in the
// fast exponential and quotient (a few ulp of f32: h is coded to 4 bits of precision next); with tanhf and a branch
// per value this took 6500 cycles a tile, a tenth of the time of 56 k-blocks.
struct ActCoef {
  float c0, c1;
};
__device__ __forceinline__ ActCoef act_coef(int act) {
  if (act == MOE_ACT_SILU) return {-1.4426950408889634f, 0.f};
  return {-2.f * 1.4426950408889634f * 0.7978845608028654f, -2.f * 1.4426950408889634f * 0.7978845608028654f * 0.044715f};
}
__device__ __forceinline__ float act_fast(ActCoef c, float g) {
  const float y = g * (c.c0 + c.c1 * fminf(g * g, 1e30f));  // the minimum: no 0 * infinity
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(y));
  return __fdividef(g, 1.0f + e);
}

// 32 bytes to one place: one store where the tensor allows it (a whole sector per lane).
__device__ __forceinline__ void store32(void* at, uint4 a, uint4 b, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(at)[0] = a;
    reinterpret_cast<uint4*>(at)[1] = b;
  }
}

// ------------------------------------------------------------------ host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (!fn) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  }
  return fn;
}

// Bytes [groups, rows, cols] read in boxes of box_rows x 128 bytes, 128-byte swizzle; what lies outside a group's
// rows or columns reads as zero.
bool make_map(CUtensorMap* m, const void* base, uint64_t groups, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {cols, rows, groups};
  const cuuint64_t strides[2] = {cols, rows * cols};
  const cuuint32_t box[3] = {static_cast<cuuint32_t>(KB), box_rows, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, groups ? 3 : 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor maps of the rows (boxes of a_box) and of one or two weight stacks (boxes of 128 rows).
bool make_maps(const Fp8GemmArgs& a, uint32_t a_box, CUtensorMap* mA, CUtensorMap* m0, CUtensorMap* m1) {
  const uint64_t G = a.G, N = a.N, K = a.K;
  if (!make_map(mA, a.A, 0, static_cast<uint64_t>(a.gather ? a.a_ld : a.rows), K, a_box) || !make_map(m0, a.B0, G, N, K, WM))
    return false;
  if (a.dual) return make_map(m1, a.B1, G, N, K, WM);
  *m1 = *m0;  // not read
  return true;
}

// `m_fmt`, `n_fmt`: formats of the MMA's M and N operands; M its rows (N is set per tile by the kernel).
Params make_params(const Ctx& c, const Fp8GemmArgs& a, int m_fmt, int n_fmt, int M) {
  Params p{};
  p.offsets = a.offsets;
  p.G = a.G;
  p.rows = a.rows;
  p.N = a.N;
  p.K = a.K;
  p.n_tiles = (a.N + WM - 1) / WM;
  p.a_scale = a.a_scale;
  p.a_ld = a.a_ld;
  p.a_scale_map = a.a_scale_map;
  p.a_scale_div = a.a_scale_div > 0 ? a.a_scale_div : 1;
  p.gather = a.gather;
  p.split = 1;
  p.kb_per = (a.K + KB - 1) / KB;
  p.s0 = a.s0;
  p.s1 = a.s1;
  // kind::f8f6f4 instruction descriptor: D f32, the operands' formats, M
  p.idesc = (1u << 4) | (static_cast<uint32_t>(m_fmt == MOE_E5M2) << 7) |
            (static_cast<uint32_t>(n_fmt == MOE_E5M2) << 10) | (static_cast<uint32_t>(M >> 4) << 24);
  p.act = a.act;
  p.out_q = static_cast<uint8_t*>(a.out_q);
  p.out_qs = a.out_qs;
  p.out_f32 = a.out_f32;
  p.out_bf16 = a.out_bf16;
  p.out_f16 = a.out_f16;
  p.out_f16_scale = a.out_f16_scale;
  p.row_map = a.row_map;
  p.row_scale = a.row_scale;
  const void* out = a.dual ? a.out_q : a.out_bf16 ? static_cast<const void*>(a.out_bf16)
                    : a.out_f16 ? static_cast<const void*>(a.out_f16) : a.out_f32;
  p.wide = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
  p.status = c.status;
  p.wait_limit = c.wait_limit;
  p.skip_stage = c.skip_stage;
  return p;
}

}  // namespace

// The kernel for groups of many rows.
cudaError_t launch_fp8_rows_gemm(const Ctx& c, const Fp8GemmArgs& a);

}  // namespace moe
