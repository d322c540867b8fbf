// Grouped matrix product of block-scaled 8-bit floats on the tensor cores.
//
//   out[r, n] = sum_kb sa[kb, r] sb[g, n / 128, kb] sum_{k in block kb} a[r, k] b[g, n, k]
//
// a: activation rows, one scale per 128 values; b: weight stacks [G, N, K], one scale per 128 x 128 block;
// group g holds rows [offsets[g], offsets[g+1]).  Dual mode multiplies the rows with W_gate and W_up and
// returns h = act(g) * u coded again with one scale per 128 outputs.
//
// The MMA runs with the weights as its M operand (128 weight rows = one scale block) and the rows of a group as
// its N operand, so that a group of any size costs its rows rounded up to 16, not to 128: experts hold from one
// row (decode) to a few hundred.  A weight tile's scale is then one number per k-block, a row's scale one number
// per accumulator column, and 128 outputs that share an h scale are the 128 TMEM lanes of one tile.
//
// A k-block of 128 is four MMAs of K = 32 into one of two TMEM accumulators; the epilogue warps read each
// finished k-block out of TMEM and add it, scaled, to f32 registers while the next one runs.
//  * warp 0: TMA producer (weight tiles 128 x 128 bytes, token tiles in boxes of 32 rows, 128-byte swizzle);
//  * warp 1: allocates TMEM, issues tcgen05.mma kind::f8f6f4 from one lane;
//  * warp 2: loads the scales of each k-block, multiplies row and tile scale, into a ring of its own;
//  * warps 4-11: epilogue; warp w reads TMEM lanes 32 (w % 4) and one half of the columns.
// Every wait is bounded; on expiry the CTA records MOE_ERR_TIMEOUT, drains and exits.
#include <cstring>

#include "fp8.cuh"

namespace moe {

namespace {

constexpr int WM = 128;            // weight rows per tile
constexpr int KB = 128;            // k-block: values that share a scale, and bytes per shared-memory row
constexpr int W_BYTES = WM * KB;
constexpr int BOX = 32;            // token rows per TMA box
constexpr int MAX_G = 256;
constexpr int THREADS = 384;
constexpr int EPI_WARPS = 8;
constexpr int SLOTS = 8;           // k-blocks of scales in flight

template <bool DUAL, int NT>
struct Cfg {
  static constexpr int MATS = DUAL ? 2 : 1;
  static constexpr int STAGE_BYTES = MATS * W_BYTES + NT * KB;
  static constexpr int STAGES = NT == 32 ? (DUAL ? 5 : 9) : (NT == 128 && !DUAL ? 6 : 4);
  static constexpr int ACC = MATS * NT;                      // TMEM columns of one accumulator
  static constexpr uint32_t TMEM_COLS = 2 * ACC < 32 ? 32 : 2 * ACC;
  static constexpr int HALF = NT / 2;                        // columns per epilogue warp
};

template <bool DUAL, int NT>
struct Aux {
  alignas(16) float sc[SLOTS][Cfg<DUAL, NT>::MATS][NT];  // row scale x tile scale
  alignas(16) float inv[NT];                             // dual: 1 / h scale of each column
  float red[EPI_WARPS][NT / 2];                          // dual: largest |h| of each warp's columns
  int dest[2][NT];                                       // single: output row of each column (-1: none)
  float rscale[2][NT];
  uint64_t full[Cfg<DUAL, NT>::STAGES];
  uint64_t empty[Cfg<DUAL, NT>::STAGES];
  uint64_t sfull[SLOTS];
  uint64_t sempty[SLOTS];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t done;
  uint32_t tmem_base;
  int abort;
  int item_off[MAX_G + 1];
  int row_off[MAX_G];
  int cnt[MAX_G];
};

template <bool DUAL, int NT>
constexpr size_t smem_bytes() {
  return 1024 + static_cast<size_t>(Cfg<DUAL, NT>::STAGES) * Cfg<DUAL, NT>::STAGE_BYTES + sizeof(Aux<DUAL, NT>);
}

struct Params {
  const int32_t* offsets;
  int G, rows, N, K, n_tiles;
  const float* a_scale;         // [nkb, a_ld]
  long long a_ld;
  const int32_t* a_scale_map;   // row r uses scale column a_scale_map[r] / a_scale_div
  int a_scale_div;
  const float* s0;
  const float* s1;
  uint32_t idesc;               // without N
  int act;
  uint8_t* out_q;
  float* out_qs;                // [ceil(N/128), rows]
  float* out_f32;
  __nv_bfloat16* out_bf16;
  const int32_t* row_map;
  const float* row_scale;
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

__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
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

// Rows per tile of a group of cnt rows: the fewest tiles of at most NT rows, evened out to multiples of 16.
template <int NT>
__device__ __forceinline__ int rows_per_tile(int cnt) {
  const int tiles = (cnt + NT - 1) / NT;
  const int per = ((cnt + tiles - 1) / max(tiles, 1) + 15) & ~15;
  return min(NT, max(per, 16));
}

struct Item {
  int g, wt, row0, n;  // group, weight tile, first row, rows
  bool alone;          // the group has one token tile: its weights are read once
};
template <int NT, typename AuxT>
__device__ __forceinline__ Item decode_item(const AuxT& aux, int G, int w) {
  int lo = 0, hi = G - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (aux.item_off[mid] <= w)
      lo = mid;
    else
      hi = mid - 1;
  }
  Item it;
  it.g = lo;
  const int cnt = aux.cnt[lo];
  const int per = rows_per_tile<NT>(cnt);
  const int tiles = (cnt + per - 1) / per;
  const int local = w - aux.item_off[lo];
  it.wt = local / tiles;
  const int tt = local - it.wt * tiles;
  it.row0 = aux.row_off[lo] + tt * per;
  it.n = min(per, cnt - tt * per);
  it.alone = tiles == 1;
  return it;
}

__device__ __forceinline__ float act_fast(int act, float g) {
  // e^-g and the quotient in the fast forms (a few ulp of f32): h is coded to 4 bits of precision next
  if (act == MOE_ACT_SILU) return __fdividef(g, 1.0f + __expf(-g));
  const float z = 0.7978845608028654f * (g + 0.044715f * g * g * g);
  return 0.5f * g * (1.0f + tanhf(z));
}

template <bool DUAL, int NT>
__global__ void __launch_bounds__(THREADS, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapW0,
                    const __grid_constant__ CUtensorMap mapW1, const Params p) {
  using C = Cfg<DUAL, NT>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Aux<DUAL, NT>& aux = *reinterpret_cast<Aux<DUAL, NT>*>(smem + STAGES * C::STAGE_BYTES);
  volatile int* abort_flag = &aux.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&aux.full[s], 1);
      mbar_init(&aux.empty[s], 1);
    }
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(&aux.sfull[s], 1);
      mbar_init(&aux.sempty[s], EPI_WARPS);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&aux.tfull[b], 1);
      mbar_init(&aux.tempty[b], EPI_WARPS);
    }
    mbar_init(&aux.done, 1);
    aux.abort = 0;
    fence_mbar_init();
  } else if (threadIdx.x == 64) {
    prefetch_tensormap(&mapA);
    prefetch_tensormap(&mapW0);
    if (DUAL) prefetch_tensormap(&mapW1);
  }
  if (warp == 1) {
    tmem_alloc(&aux.tmem_base, C::TMEM_COLS);
    tmem_relinquish();
  }
  pdl_trigger();
  pdl_wait();
  for (int g = threadIdx.x; g < p.G; g += THREADS) {
    const int o0 = p.offsets ? p.offsets[g] : 0;
    const int o1 = p.offsets ? p.offsets[g + 1] : p.rows;
    // a group's rows stay inside the tensor, whatever the offsets hold
    const int r0 = min(max(o0, 0), p.rows), r1 = min(max(o1, r0), p.rows);
    if (r0 != o0 || r1 != o1) record_status(p.status, MOE_ERR_DEVICE_INDEX);
    aux.row_off[g] = r0;
    aux.cnt[g] = r1 - r0;
  }
  __syncthreads();
  if (warp == 0) {  // exclusive scan of the work items per group; lane owns groups [8 lane, 8 lane + 8)
    int v[8], local = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int g = lane * 8 + i;
      const int cnt = g < p.G ? aux.cnt[g] : 0;
      const int per = rows_per_tile<NT>(cnt);
      v[i] = (cnt + per - 1) / per * p.n_tiles;
      local += v[i];
    }
    int incl = local;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += n;
    }
    int run = incl - local;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int g = lane * 8 + i;
      if (g < p.G) aux.item_off[g] = run;
      run += v[i];
    }
    if (lane == 31) aux.item_off[p.G] = incl;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem_base = aux.tmem_base;
  const int total = aux.item_off[p.G];
  const int nkb = (p.K + KB - 1) / KB;
  const long long limit = p.wait_limit;

  if (warp < 4) {
    // 128 x 56 + 256 x 224 = 384 x 168 registers, what the CTA was launched with
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 0) {
      if (lane == 0) {
        // -------------------------------------------------------- TMA producer
        uint32_t kbg = 0, outstanding = 0, out_phase = 0;
        bool skipped = false;
        const uint64_t pol_first = l2_policy_evict_first(), pol_normal = l2_policy_evict_normal(),
                       pol_last = l2_policy_evict_last();
        for (int w = blockIdx.x; w < total && !*abort_flag; w += gridDim.x) {
          const Item it = decode_item<NT>(aux, p.G, w);
          const int boxes = (it.n + BOX - 1) / BOX;
          const uint64_t pol_w = it.alone ? pol_first : pol_normal;
          for (int kb = 0; kb < nkb; ++kb, ++kbg) {
            const int s = kbg % STAGES;
            const uint32_t ph = (kbg / STAGES) & 1u;
            if (!mbar_wait_bounded(&aux.empty[s], ph ^ 1u, limit, abort_flag)) break;
            outstanding &= ~(1u << s);
            if (p.skip_stage && !skipped && blockIdx.x == 0) {  // debug: leave this stage unfilled
              skipped = true;
              continue;
            }
            uint8_t* st = smem + s * C::STAGE_BYTES;
            mbar_arrive_expect_tx(&aux.full[s], C::MATS * W_BYTES + boxes * BOX * KB);
            tma_load_3d(st, &mapW0, &aux.full[s], kb * KB, it.wt * WM, it.g, pol_w);
            if (DUAL) tma_load_3d(st + W_BYTES, &mapW1, &aux.full[s], kb * KB, it.wt * WM, it.g, pol_w);
            for (int b = 0; b < boxes; ++b)
              tma_load_2d_hint(st + C::MATS * W_BYTES + b * BOX * KB, &mapA, &aux.full[s], kb * KB, it.row0 + b * BOX,
                               pol_last);
            outstanding |= 1u << s;
            out_phase = (out_phase & ~(1u << s)) | (ph << s);
          }
        }
        if (*abort_flag)  // let issued copies land before the CTA exits
          for (int s = 0; s < STAGES; ++s)
            if (outstanding & (1u << s)) wait_cycles(&aux.full[s], (out_phase >> s) & 1u, limit);
      }
    } else if (warp == 1) {
      if (lane == 0) {
        // -------------------------------------------------------- MMA issuer
        uint32_t kbg = 0;
        bool ok = true;
        for (int w = blockIdx.x; w < total && ok; w += gridDim.x) {
          const Item it = decode_item<NT>(aux, p.G, w);
          const uint32_t n16 = (it.n + 15) & ~15;
          const uint32_t idesc = p.idesc | ((n16 >> 3) << 17);
          for (int kb = 0; kb < nkb; ++kb, ++kbg) {
            const int s = kbg % STAGES;
            const int buf = kbg & 1;
            if (!mbar_wait_bounded(&aux.tempty[buf], ((kbg >> 1) & 1u) ^ 1u, limit, abort_flag) ||
                !mbar_wait_bounded(&aux.full[s], (kbg / STAGES) & 1u, limit, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t st = smem_addr(smem + s * C::STAGE_BYTES);
            const uint64_t tdesc = sw128_kmajor_desc(st + C::MATS * W_BYTES);
#pragma unroll
            for (int m = 0; m < C::MATS; ++m) {
              const uint64_t wdesc = sw128_kmajor_desc(st + m * W_BYTES);
              const uint32_t d = tmem_base + buf * C::ACC + m * NT;
#pragma unroll
              for (int kk = 0; kk < KB / 32; ++kk)
                umma_f8(d, wdesc + static_cast<uint64_t>(kk * 2), tdesc + static_cast<uint64_t>(kk * 2), idesc,
                        kk > 0 ? 1u : 0u);
            }
            umma_commit(&aux.empty[s]);
            umma_commit(&aux.tfull[buf]);
          }
        }
        umma_commit(&aux.done);  // every MMA issued above completes before TMEM is released
        wait_cycles(&aux.done, 0, limit);
      }
    } else if (warp == 2) {
      // ---------------------------------------------------------- scales
      constexpr int PER = NT / 32;
      uint32_t kbg = 0;
      bool ok = true;
      for (int w = blockIdx.x; w < total && ok; w += gridDim.x) {
        const Item it = decode_item<NT>(aux, p.G, w);
        int at[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const int r = it.row0 + min(lane + 32 * j, it.n - 1);
          int col = p.a_scale_map ? p.a_scale_map[r] / p.a_scale_div : r;
          col = min(max(col, 0), static_cast<int>(p.a_ld) - 1);
          at[j] = col;
        }
        const long long sb = (static_cast<long long>(it.g) * p.n_tiles + it.wt) * nkb;
        float v[2][PER], t0[2], t1[2];
        auto load = [&](int kb, int b) {
          const int k = min(kb, nkb - 1);
#pragma unroll
          for (int j = 0; j < PER; ++j) v[b][j] = __ldg(p.a_scale + k * p.a_ld + at[j]);
          t0[b] = __ldg(p.s0 + sb + k);
          t1[b] = DUAL ? __ldg(p.s1 + sb + k) : 0.f;
        };
        load(0, 0);
        load(1, 1);
        for (int kb0 = 0; kb0 < nkb && ok; kb0 += 2) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            if (kb0 + b >= nkb) break;
            const int slot = kbg % SLOTS;
            const bool got = mbar_wait_bounded(&aux.sempty[slot], ((kbg / SLOTS) & 1u) ^ 1u, limit, abort_flag);
            if (!__all_sync(0xffffffffu, got)) {
              ok = false;
              break;
            }
#pragma unroll
            for (int j = 0; j < PER; ++j) {
              aux.sc[slot][0][lane + 32 * j] = v[b][j] * t0[b];
              if (DUAL) aux.sc[slot][C::MATS - 1][lane + 32 * j] = v[b][j] * t1[b];
            }
            load(kb0 + b + 2, b);
            __syncwarp();
            if (lane == 0) mbar_arrive(&aux.sfull[slot]);
            ++kbg;
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    // -------------------------------------------------------------- epilogue
    constexpr int HALF = C::HALF;
    constexpr int CH = 16;  // columns per TMEM load
    const int ew = warp - 4;
    const int q = warp & 3, half = ew >> 2;
    const int et = threadIdx.x - 128;  // thread of the epilogue
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    uint32_t kbg = 0;
    int parity = 0;
    for (int w = blockIdx.x; w < total; w += gridDim.x, parity ^= 1) {
      const Item it = decode_item<NT>(aux, p.G, w);
      const int n16 = (it.n + 15) & ~15;
      if (!DUAL) {  // output row and scale of each column
        for (int c = et; c < NT; c += EPI_WARPS * 32) {
          int d = -1;
          float rs = 1.f;
          if (c < it.n) {
            d = p.row_map ? p.row_map[it.row0 + c] : it.row0 + c;
            if (d < 0 || d >= p.rows) {
              record_status(p.status, MOE_ERR_DEVICE_INDEX);
              d = -1;
            } else if (p.row_scale) {
              rs = p.row_scale[d];
            }
          }
          aux.dest[parity][c] = d;
          aux.rscale[parity][c] = rs;
        }
      }
      unsigned long long acc[C::MATS][HALF / 2];
#pragma unroll
      for (int m = 0; m < C::MATS; ++m)
#pragma unroll
        for (int j = 0; j < HALF / 2; ++j) acc[m][j] = 0ull;
      bool ok = true;
      for (int kb = 0; kb < nkb; ++kb, ++kbg) {
        const int slot = kbg % SLOTS, buf = kbg & 1;
        const bool got = mbar_wait_bounded(&aux.sfull[slot], (kbg / SLOTS) & 1u, limit, abort_flag) &&
                         mbar_wait_bounded(&aux.tfull[buf], (kbg >> 1) & 1u, limit, abort_flag);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t tb = tmem_base + lane_base + buf * C::ACC + half * HALF;
#pragma unroll
        for (int c = 0; c < HALF; c += CH) {
          if (half * HALF + c >= n16) break;  // warp-uniform
          uint32_t v[C::MATS][CH];
#pragma unroll
          for (int m = 0; m < C::MATS; ++m) tmem_ld_32x32b_x16(tb + m * NT + c, v[m]);
          tmem_ld_wait();
#pragma unroll
          for (int m = 0; m < C::MATS; ++m) {
            const ulonglong2* s2 = reinterpret_cast<const ulonglong2*>(&aux.sc[slot][m][half * HALF + c]);
#pragma unroll
            for (int j = 0; j < CH / 4; ++j) {
              const ulonglong2 s = s2[j];
              fma2(acc[m][c / 2 + 2 * j], v[m][4 * j], v[m][4 * j + 1], s.x);
              fma2(acc[m][c / 2 + 2 * j + 1], v[m][4 * j + 2], v[m][4 * j + 3], s.y);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&aux.tempty[buf]);
          mbar_arrive(&aux.sempty[slot]);
        }
      }
      // uniform over the epilogue: either every warp has all k-blocks or the tile is dropped; also orders dest
      if (!named_barrier_and(1, EPI_WARPS * 32, ok)) break;
      const int n = it.wt * WM + q * 32 + lane;  // this thread's weight row
      if (DUAL) {
        float mx = 0.f;
        uint32_t keep = 0;
#pragma unroll
        for (int j = 0; j < HALF; j += 2) {
          float g0, g1, u0, u1;
          split2(acc[0][j / 2], g0, g1);
          split2(acc[C::MATS - 1][j / 2], u0, u1);
          const float h0 = act_fast(p.act, g0) * u0, h1 = act_fast(p.act, g1) * u1;
          acc[0][j / 2] = static_cast<unsigned long long>(__float_as_uint(h0)) |
                          (static_cast<unsigned long long>(__float_as_uint(h1)) << 32);
          const uint32_t m0 = __reduce_max_sync(0xffffffffu, __float_as_uint(h0) & 0x7fffffffu);
          const uint32_t m1 = __reduce_max_sync(0xffffffffu, __float_as_uint(h1) & 0x7fffffffu);
          if (lane == (j & 31)) keep = m0;
          if (lane == (j & 31) + 1) keep = m1;
          if ((j & 31) == 30 || j == HALF - 2)
            if (lane <= (j & 31) + 1) aux.red[ew][(j & ~31) + lane] = __uint_as_float(keep);
        }
        (void)mx;
        named_barrier(2 + half, 128);
        if (et - half * 128 < HALF) {
          const int c = et - half * 128;
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(aux.red[half * 4 + i][c]));
          float scale, inv;
          fp8_scale(m, MOE_E4M3, false, scale, inv);
          const int col = half * HALF + c;
          aux.inv[col] = inv;
          if (col < it.n) p.out_qs[static_cast<long long>(it.wt) * p.rows + it.row0 + col] = scale;
        }
        named_barrier(2 + half, 128);
        if (n < p.N) {
          uint8_t* o = p.out_q + static_cast<long long>(it.row0 + half * HALF) * p.N + n;
#pragma unroll
          for (int j = 0; j < HALF; j += 2) {
            if (half * HALF + j < it.n) {
              float h0, h1;
              split2(acc[0][j / 2], h0, h1);
              const uint32_t code = fp8_pack2(h0 * aux.inv[half * HALF + j], h1 * aux.inv[half * HALF + j + 1], MOE_E4M3);
              o[static_cast<long long>(j) * p.N] = static_cast<uint8_t>(code);
              if (half * HALF + j + 1 < it.n) o[static_cast<long long>(j + 1) * p.N] = static_cast<uint8_t>(code >> 8);
            }
          }
        }
      } else if (n < p.N) {
#pragma unroll
        for (int j = 0; j < HALF; j += 2) {
          float y0, y1;
          split2(acc[0][j / 2], y0, y1);
          const int c = half * HALF + j;
          const int d0 = aux.dest[parity][c], d1 = aux.dest[parity][c + 1];
          y0 *= aux.rscale[parity][c];
          y1 *= aux.rscale[parity][c + 1];
          if (p.out_bf16) {
            if (d0 >= 0) p.out_bf16[static_cast<long long>(d0) * p.N + n] = __float2bfloat16_rn(y0);
            if (d1 >= 0) p.out_bf16[static_cast<long long>(d1) * p.N + n] = __float2bfloat16_rn(y1);
          } else {
            if (d0 >= 0) p.out_f32[static_cast<long long>(d0) * p.N + n] = y0;
            if (d1 >= 0) p.out_f32[static_cast<long long>(d1) * p.N + n] = y1;
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
  if (threadIdx.x == 0 && aux.abort) record_status(p.status, MOE_ERR_TIMEOUT);
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

template <bool DUAL, int NT>
cudaError_t launch_typed(const Ctx& c, const Fp8GemmArgs& a) {
  CUtensorMap mA, m0, m1;
  if (!make_map(&mA, a.A, 0, static_cast<uint64_t>(a.rows), static_cast<uint64_t>(a.K), BOX) ||
      !make_map(&m0, a.B0, static_cast<uint64_t>(a.G), static_cast<uint64_t>(a.N), static_cast<uint64_t>(a.K), WM))
    return cudaErrorInvalidValue;
  if (DUAL) {
    if (!make_map(&m1, a.B1, static_cast<uint64_t>(a.G), static_cast<uint64_t>(a.N), static_cast<uint64_t>(a.K), WM))
      return cudaErrorInvalidValue;
  } else {
    m1 = m0;
  }
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
  p.s0 = a.s0;
  p.s1 = a.s1;
  // kind::f8f6f4 instruction descriptor: D f32, formats of the M operand (weights) and the N operand (rows), M
  p.idesc = (1u << 4) | (static_cast<uint32_t>(a.b_fmt == MOE_E5M2) << 7) |
            (static_cast<uint32_t>(a.a_fmt == MOE_E5M2) << 10) | (static_cast<uint32_t>(WM >> 4) << 24);
  p.act = a.act;
  p.out_q = static_cast<uint8_t*>(a.out_q);
  p.out_qs = a.out_qs;
  p.out_f32 = a.out_f32;
  p.out_bf16 = a.out_bf16;
  p.row_map = a.row_map;
  p.row_scale = a.row_scale;
  p.status = c.status;
  p.wait_limit = c.wait_limit;
  p.skip_stage = c.skip_stage;
  const long long tiles = a.rows / 16 < a.G ? a.rows : a.rows / 16 + a.G;  // no fewer than there can be
  const int grid = static_cast<int>(std::max(1LL, std::min<long long>(c.num_sms, tiles * p.n_tiles)));
  auto kern = fp8_gemm_kernel<DUAL, NT>;
  constexpr size_t smem = smem_bytes<DUAL, NT>();
  static_assert(smem <= 232448, "shared memory of one block");
  const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(kern), static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  KernelScope ks(c, a.name ? a.name : "fp8_gemm");
  return launch_kernel(c, kern, dim3(grid), dim3(THREADS), smem, mA, m0, m1, p);
}

}  // namespace

cudaError_t launch_fp8_gemm(const Ctx& c, const Fp8GemmArgs& a) {
  if (a.rows <= 0 || a.G <= 0) return cudaSuccess;
  if (a.G > MAX_G || a.N % 32 || a.K % 32 || a.N <= 0 || a.K <= 0) return cudaErrorInvalidValue;
  const double per_group = static_cast<double>(a.rows) / std::min(a.G, a.rows);
  const bool small = per_group <= 16.0;
  if (a.dual) return small ? launch_typed<true, 32>(c, a) : launch_typed<true, 128>(c, a);
  return small ? launch_typed<false, 32>(c, a) : launch_typed<false, 256>(c, a);
}

}  // namespace moe
