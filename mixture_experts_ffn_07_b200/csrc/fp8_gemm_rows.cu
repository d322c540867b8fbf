// The block-scaled 8-bit product for groups of many rows.
//
// A tile is 128 rows (the MMA's M operand) x 256 weight rows (N; dual mode: 128 of W_gate and the same 128 of W_up).
// A thread of the epilogue owns one row, whose scale in a k-block is one number for the 128 columns of a weight tile:
// adding a finished k-block to the f32 registers is a TMEM load in the fast 32-lane shape and packed FMAs with one
// scalar, 340 cycles for 128 x 256 values against 512 for the MMA (650 when every column has a scale of its own, the
// form of fp8_gemm.cu).  A tile costs 128 rows whatever it holds, so launches of small groups take that form.
//
// One CTA per tile: pairs of CTAs sharing the weights (cta_group::2, 32 KB copied per k-block instead of 48) measured
// slower, 1080 cycles a k-block: an accumulator is free for the next MMA only when both CTAs' epilogues have read it,
// and the signals between the two CTAs took about 600 cycles of that.
// What bounds it: the copies from L2.  48 KB a k-block at the 48 bytes a clock that an SM takes in are 1000 cycles (1030
// measured: 1024 tokens, 32 experts of 7168 x 2048), twice the MMA's time; neither the rows' share of the copies (boxes of
// 32 or 64 rows for part tiles) nor output through bulk stores changed the times.  8192 x 7168 x 2048: 134 us, 1.8 PFLOP/s;
// 163 us in a loop of seconds, where the 1000 W cap holds the clock at 1.6 GHz.
//  * warp 0: TMA producer; warp 1: TMEM and the MMAs, from one lane, into two accumulators;
//  * warps 2 and 3: the scales of each k-block, row times weight tile, into a ring in shared memory;
//  * warps 4-11: epilogue; warp w has the rows of TMEM lanes 32 (w % 4) and one half of the columns.
// Every wait is bounded; on expiry the CTA records MOE_ERR_TIMEOUT, drains and exits.
#include "fp8_mma.cuh"

namespace moe {

namespace {

constexpr int STAGES = 4;
constexpr int STAGE_BYTES = 3 * W_BYTES;  // 128 rows and 256 weight rows of 128 bytes
constexpr int NBUF = 2;
constexpr int ACC = 256;
constexpr uint32_t TMEM_COLS = NBUF * ACC;
constexpr int AHEAD = 4;                  // k-blocks of scales in flight per scale warp
// Ring of scales.  The scale warps write a k-block's slot after its stage came free, that is after the MMA STAGES
// k-blocks earlier, which the epilogue's reads of the k-block two before that one (values and scales) precede: a slot
// that is STAGES + 2 k-blocks old is read, and the ring needs no barriers of its own.
constexpr int SLOTS = 8;
static_assert(SLOTS >= STAGES + NBUF, "ring of scales");

struct Aux {
  alignas(8) float2 sc[SLOTS][TILE_ROWS];  // row scale times the scales of the two weight tiles
  uint64_t full[STAGES];
  uint64_t empty[STAGES];
  uint64_t tfull[NBUF];
  uint64_t tempty[NBUF];
  uint64_t done;
  uint32_t tmem_base;
  int abort;
  uint32_t red[2][128];  // dual: largest |h| of each row over one half of the columns, as bits
  int item_off[MAX_G + 1];
  int row_off[MAX_G];
  int cnt[MAX_G];
};
constexpr size_t SMEM = 1024 + static_cast<size_t>(STAGES) * STAGE_BYTES + sizeof(Aux);
static_assert(SMEM <= SMEM_MAX, "shared memory");

struct Item {
  int g, wt, row0, n;  // group, weight tile (of 128, or 256 in single mode), first row, rows
};
// All lanes of a warp: lane l looks at group 8 l, then lanes 0-7 at the eight groups found (a binary search took a
// dozen dependent shared loads, about 1000 cycles a tile with the divisions).
__device__ __forceinline__ Item decode_item(const Aux& aux, int G, int w) {
  const int lane = threadIdx.x & 31;
  const unsigned coarse = __ballot_sync(0xffffffffu, 8 * lane < G && aux.item_off[min(8 * lane, G)] <= w);
  const int g0 = 8 * (31 - __clz(coarse));  // item_off[0] == 0: lane 0 always says yes
  const int mine = min(g0 + (lane & 7), G);
  const int off = aux.item_off[mine];
  const unsigned fine = __ballot_sync(0xffffffffu, lane < 8 && mine < G && off <= w);
  const int k = 31 - __clz(fine);
  Item it;
  it.g = g0 + k;
  const int local = w - __shfl_sync(0xffffffffu, off, k);
  const int cnt = aux.cnt[it.g];
  const int tiles = (cnt + TILE_ROWS - 1) / TILE_ROWS;
  it.wt = tiles == 1 ? local : local / tiles;
  const int tt = local - it.wt * tiles;
  it.row0 = aux.row_off[it.g] + tt * TILE_ROWS;
  it.n = min(TILE_ROWS, cnt - tt * TILE_ROWS);
  return it;
}

__device__ __forceinline__ void tmem_ld_16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Waits for the thread's TMEM loads; names the registers, so that nothing reads them earlier.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 ::"memory");
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t f16_pair(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// The power of two that brings 128 outputs of a row into f16, and its inverse, from the sum of their k-blocks' |scale|:
// a block of 128 products of two e4m3 codes is at most 128 * 448^2 in size, so the outputs are below `top`, and
// 2^e > top brings them below 2^15 (f32 roundings on the way are far from the factor 2 that is left).  The values lie a
// few hundred times below the bound, where f16 has 11 significant bits down to 2^-29 of it: 2^-11 relative, 8 times
// finer than bf16 rows, for the same bytes.
__device__ __forceinline__ float f16_scale(float scales, float& back) {
  const float top = fminf(scales * (128.f * 448.f * 448.f), 3.4028235e38f);  // (a NaN counts as the largest)
  const int e = max(static_cast<int>(__float_as_uint(top) >> 23) - 126, -110);
  back = __uint_as_float(static_cast<uint32_t>(127 + e - 15) << 23);
  return __uint_as_float(static_cast<uint32_t>(127 + 15 - e) << 23);
}

__device__ __forceinline__ uint4 f32x4(float a, float b, float c, float d) {
  return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c), __float_as_uint(d));
}

template <bool DUAL>
__global__ void __launch_bounds__(THREADS, 1)
    fp8_rows_gemm_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapW0,
                    const __grid_constant__ CUtensorMap mapW1, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Aux& aux = *reinterpret_cast<Aux*>(smem + STAGES * STAGE_BYTES);
  volatile int* abort_flag = &aux.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&aux.full[s], 3);  // the producer and the two scale warps
      mbar_init(&aux.empty[s], 1);
    }
    for (int b = 0; b < NBUF; ++b) {
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
    tmem_alloc(&aux.tmem_base, TMEM_COLS);
    tmem_relinquish();
  }
  // p.early: as in fp8_gemm.cu, the weights' copies start before the launch before has ended
  if (!p.early) pdl_wait();
  pdl_trigger();
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
  const int w_items = DUAL ? p.n_tiles : (p.n_tiles + 1) / 2;
  if (warp == 0) {  // exclusive scan of the work items per group; lane owns groups [8 lane, 8 lane + 8)
    int v[8], local = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int g = lane * 8 + i;
      v[i] = g < p.G ? (aux.cnt[g] + TILE_ROWS - 1) / TILE_ROWS * w_items : 0;
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
    // 128 x 88 + 256 x 208 = 384 x 168 registers, what the CTA was launched with
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0) {
      // ---------------------------------------------------------- TMA producer (lane 0; the warp finds the items)
      uint32_t kbg = 0, outstanding = 0, out_phase = 0;
      bool skipped = false;
      const uint64_t pol_a = l2_policy_evict_last();    // rows: read by every weight tile
      const uint64_t pol_w = l2_policy_evict_normal();  // weights: read by every row tile of the group
      auto weights = [&](const Item& it, int n0, int kb, int s) {  // and the bytes of the whole stage
        uint8_t* st = smem + s * STAGE_BYTES;
        mbar_arrive_expect_tx(&aux.full[s], STAGE_BYTES);
        tma_load_3d(st + W_BYTES, &mapW0, &aux.full[s], kb * KB, n0, it.g, pol_w);
        tma_load_3d(st + 2 * W_BYTES, DUAL ? &mapW1 : &mapW0, &aux.full[s], kb * KB, DUAL ? n0 : n0 + WM, it.g, pol_w);
      };
      for (int w = blockIdx.x; w < total; w += gridDim.x) {
        if (__shfl_sync(0xffffffffu, *abort_flag, 0)) break;
        const Item it = decode_item(aux, p.G, w);
        const int n0 = DUAL ? it.wt * WM : 2 * it.wt * WM;
        int filled = 0;  // k-blocks whose weights are on their way
        if (p.early && w == static_cast<int>(blockIdx.x)) {
          filled = min(STAGES, nkb);
          if (lane == 0)
            for (int kb = 0; kb < filled; ++kb) {
              if (p.skip_stage && kb == 0 && blockIdx.x == 0) continue;  // debug: leave this stage unfilled
              weights(it, n0, kb, kb);
            }
          pdl_wait();
        }
        if (lane == 0)
          for (int kb = 0; kb < nkb; ++kb, ++kbg) {
            const int s = kbg % STAGES;
            const uint32_t ph = (kbg / STAGES) & 1u;
            // (every stage whose weights are on their way gets its rows too, so that its copies are waited for)
            if (kb >= filled && !mbar_wait_bounded(&aux.empty[s], ph ^ 1u, limit, abort_flag)) break;
            outstanding &= ~(1u << s);
            if (p.skip_stage && !skipped && blockIdx.x == 0) {  // debug: leave this stage unfilled
              skipped = true;
              continue;
            }
            if (kb >= filled) weights(it, n0, kb, s);
            tma_load_2d_hint(smem + s * STAGE_BYTES, &mapA, &aux.full[s], kb * KB, it.row0, pol_a);
            outstanding |= 1u << s;
            out_phase = (out_phase & ~(1u << s)) | (ph << s);
          }
        __syncwarp();
      }
      if (lane == 0 && *abort_flag)  // let issued copies land before the CTA exits
        for (int s = 0; s < STAGES; ++s)
          if (outstanding & (1u << s)) wait_cycles(&aux.full[s], (out_phase >> s) & 1u, limit);
    } else if (warp == 1) {
      if (lane == 0) {
        // -------------------------------------------------------- MMA issuer
        const uint32_t idesc = p.idesc | (static_cast<uint32_t>(ACC) >> 3 << 17);
        uint32_t kbg = 0;
        bool ok = true;
        for (int w = blockIdx.x; w < total && ok; w += gridDim.x) {
          for (int kb = 0; kb < nkb; ++kb, ++kbg) {
            const int s = kbg % STAGES;
            const int buf = kbg % NBUF;
            if (!mbar_wait_bounded(&aux.full[s], (kbg / STAGES) & 1u, limit, abort_flag) ||
                !mbar_wait_bounded(&aux.tempty[buf], ((kbg / NBUF) & 1u) ^ 1u, limit, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t st = smem_addr(smem + s * STAGE_BYTES);
            const uint64_t adesc = sw128_kmajor_desc(st), wdesc = sw128_kmajor_desc(st + W_BYTES);
#pragma unroll
            for (int kk = 0; kk < KB / 32; ++kk)
              umma_f8(tmem_base + buf * ACC, adesc + static_cast<uint64_t>(kk * 2),
                      wdesc + static_cast<uint64_t>(kk * 2), idesc, kk > 0 ? 1u : 0u);
            umma_commit(&aux.tfull[buf]);
            umma_commit(&aux.empty[s]);
          }
        }
        umma_commit(&aux.done);  // every MMA issued above completes before TMEM is released
        wait_cycles(&aux.done, 0, limit);
      }
    } else {
      // ---------------------------------------------------------- scales: warp 2 + i has rows 64 i .. 64 i + 63
      const int r0 = (warp - 2) * 64 + lane;
      if (p.early) pdl_wait();
      uint32_t kbg = 0;
      bool ok = true;
      for (int w = blockIdx.x; w < total && ok; w += gridDim.x) {
        const Item it = decode_item(aux, p.G, w);
        int at[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int row = it.row0 + min(r0 + 32 * j, it.n - 1);
          const int col = p.a_scale_map ? p.a_scale_map[row] / p.a_scale_div : row;
          at[j] = min(max(col, 0), static_cast<int>(p.a_ld) - 1);
        }
        const long long tiles = static_cast<long long>(it.g) * p.n_tiles;
        const float* t0 = p.s0 + (tiles + (DUAL ? it.wt : 2 * it.wt)) * nkb;
        const float* t1 = DUAL ? p.s1 + (tiles + it.wt) * nkb : p.s0 + (tiles + min(2 * it.wt + 1, p.n_tiles - 1)) * nkb;
        float va[AHEAD][2], v0[AHEAD], v1[AHEAD];
        auto load = [&](int kb, int b) {
          const int k = min(kb, nkb - 1);
#pragma unroll
          for (int j = 0; j < 2; ++j) va[b][j] = p.a_scale[k * p.a_ld + at[j]];
          v0[b] = t0[k];
          v1[b] = t1[k];
        };
#pragma unroll
        for (int b = 0; b < AHEAD; ++b) load(b, b);
        for (int kb0 = 0; kb0 < nkb && ok; kb0 += AHEAD) {
#pragma unroll
          for (int b = 0; b < AHEAD; ++b) {  // unrolled, so that a scale in flight is never moved between registers
            if (kb0 + b >= nkb) break;
            const int s = kbg % STAGES;
            const bool got = mbar_wait_bounded(&aux.empty[s], ((kbg / STAGES) & 1u) ^ 1u, limit, abort_flag);
            if (!__all_sync(0xffffffffu, got)) {
              ok = false;
              break;
            }
            float2* slot = aux.sc[kbg % SLOTS];
#pragma unroll
            for (int j = 0; j < 2; ++j) slot[r0 + 32 * j] = make_float2(va[b][j] * v0[b], va[b][j] * v1[b]);
            load(kb0 + b + AHEAD, b);
            __syncwarp();
            if (lane == 0) mbar_arrive(&aux.full[s]);
            ++kbg;
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // -------------------------------------------------------------- epilogue
    const int ew = warp - 4;
    const int q = warp & 3, half = ew >> 2;
    const int r = q * 32 + lane;       // this thread's row of the CTA's 128
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    // First column of each part of 32: dual: gate [64 half, + 64), then up of the same outputs, 128 further;
    // single: [128 half, + 128)
    auto load_col = [&](int st) { return DUAL ? (st >> 1) * 128 + half * 64 + (st & 1) * 32 : half * 128 + st * 32; };
    const float2* my_sc = &aux.sc[0][r];
    if (p.early) pdl_wait();
    uint32_t kbg = 0;
    for (int w = blockIdx.x; w < total; w += gridDim.x) {
      const Item it = decode_item(aux, p.G, w);
      const int valid = it.n, row_base = it.row0;
      const bool live = q * 32 < valid;  // warp-uniform
      // single: this row's output row, first looked at after the k-blocks, so that they do not wait for it
      int dest = row_base + r;
      if (!DUAL && r < valid && p.row_map) dest = p.row_map[row_base + r];
      unsigned long long acc[4][16];  // 32 columns each
#pragma unroll
      for (int st = 0; st < 4; ++st)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[st][j] = 0ull;
      float scales = 0.f;  // single: sum of the k-blocks' |scale|
      bool ok = true;
      for (int kb = 0; kb < nkb; ++kb, ++kbg) {
        const int buf = kbg % NBUF;
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(&aux.tfull[buf], (kbg / NBUF) & 1u, limit, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (live) {
          const float2 f = my_sc[(kbg % SLOTS) * TILE_ROWS];  // written before the MMA was issued
          const unsigned long long s0 = DUAL ? join2(f.x, f.x) : (half ? join2(f.y, f.y) : join2(f.x, f.x));
          const unsigned long long s1 = DUAL ? join2(f.y, f.y) : s0;
          if (!DUAL) scales += fabsf(half ? f.y : f.x);
          // 16 columns at a time and one load in flight: the other warp of the scheduler fills the wait, and no
          // accumulator spills (two loads of 16 in flight, or one of 32 consecutive registers, spilled a few registers
          // in this loop and cost a fifth of the time)
          const uint32_t tb = lane_base + buf * ACC;
#pragma unroll
          for (int st = 0; st < 8; ++st) {
            uint32_t v[16];
            tmem_ld_16(tb + load_col(st >> 1) + (st & 1) * 16, v);
            tmem_wait(v);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              fma2(acc[st >> 1][8 * (st & 1) + i], v[2 * i], v[2 * i + 1], DUAL && st >= 4 ? s1 : s0);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&aux.tempty[buf]);
      }
      // uniform over the epilogue: either every warp has all k-blocks or the tile is dropped
      if (!named_barrier_and(1, EPI_WARPS * 32, ok)) break;
      float rs = 1.f;
      if (!DUAL) {
        if (r >= valid) {
          dest = -1;
        } else if (dest < 0 || dest >= p.rows) {
          record_status(p.status, MOE_ERR_DEVICE_INDEX);
          dest = -1;
        } else if (p.row_scale) {
          rs = p.row_scale[dest];
        }
      }
      if (DUAL) {
        // h = act(g) * u in place of g, its largest value over the row's 128 outputs, codes
        const ActCoef ac = act_coef(p.act);
        uint32_t mx = 0;
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float g0, g1, u0, u1;
            split2(acc[st][j], g0, g1);
            split2(acc[st + 2][j], u0, u1);
            const float h0 = act_fast(ac, g0) * u0, h1 = act_fast(ac, g1) * u1;
            acc[st][j] = join2(h0, h1);
            mx = max(mx, max(__float_as_uint(h0) & 0x7fffffffu, __float_as_uint(h1) & 0x7fffffffu));
          }
        aux.red[half][r] = mx;
        named_barrier(2, EPI_WARPS * 32);
        float scale, inv;
        fp8_scale(max(aux.red[0][r], aux.red[1][r]), MOE_E4M3, false, scale, inv);
        if (r < valid) {
          if (half == 0) p.out_qs[static_cast<long long>(it.wt) * p.rows + row_base + r] = scale;
          const int col = it.wt * WM + half * 64;
          uint8_t* o = p.out_q + static_cast<long long>(row_base + r) * p.N + col;
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            uint32_t c[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              float a0, a1, b0, b1;
              split2(acc[st][2 * e], a0, a1);
              split2(acc[st][2 * e + 1], b0, b1);
              c[e] = fp8_pack2(a0 * inv, a1 * inv, MOE_E4M3) | (fp8_pack2(b0 * inv, b1 * inv, MOE_E4M3) << 16);
            }
            if (col + 32 * st < p.N)  // N is a multiple of 32
              store32(o + 32 * st, make_uint4(c[0], c[1], c[2], c[3]), make_uint4(c[4], c[5], c[6], c[7]), p.wide);
          }
        }
      } else if (dest >= 0) {
        const int col = (2 * it.wt + half) * WM;
        if (p.out_f16) {
          float back;
          rs = f16_scale(scales, back);
          if (col < p.N) p.out_f16_scale[static_cast<long long>(dest) * p.n_tiles + 2 * it.wt + half] = back;
        }
#pragma unroll
        for (int st = 0; st < 4; ++st) {
          if (col + 32 * st >= p.N) break;
          const long long at = static_cast<long long>(dest) * p.N + col + 32 * st;
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // 16 columns
            float y[16];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              split2(acc[st][8 * h + j], y[2 * j], y[2 * j + 1]);
              y[2 * j] *= rs;
              y[2 * j + 1] *= rs;
            }
            if (p.out_f16) {
              store32(p.out_f16 + at + 16 * h,
                      make_uint4(f16_pair(y[0], y[1]), f16_pair(y[2], y[3]), f16_pair(y[4], y[5]), f16_pair(y[6], y[7])),
                      make_uint4(f16_pair(y[8], y[9]), f16_pair(y[10], y[11]), f16_pair(y[12], y[13]),
                                 f16_pair(y[14], y[15])),
                      p.wide);
            } else if (p.out_bf16) {
              store32(p.out_bf16 + at + 16 * h,
                      make_uint4(bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3]), bf16_pair(y[4], y[5]), bf16_pair(y[6], y[7])),
                      make_uint4(bf16_pair(y[8], y[9]), bf16_pair(y[10], y[11]), bf16_pair(y[12], y[13]),
                                 bf16_pair(y[14], y[15])),
                      p.wide);
            } else {
#pragma unroll
              for (int e = 0; e < 2; ++e)
                store32(p.out_f32 + at + 16 * h + 8 * e, f32x4(y[8 * e], y[8 * e + 1], y[8 * e + 2], y[8 * e + 3]),
                        f32x4(y[8 * e + 4], y[8 * e + 5], y[8 * e + 6], y[8 * e + 7]), p.wide);
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
  if (threadIdx.x == 0 && aux.abort) record_status(p.status, MOE_ERR_TIMEOUT);
  if (p.early) pdl_wait();  // complete only after the launch before
}

template <bool DUAL>
cudaError_t launch_typed(const Ctx& c, const Fp8GemmArgs& a) {
  CUtensorMap mA, m0, m1;
  if (!make_maps(a, TILE_ROWS, &mA, &m0, &m1)) return cudaErrorInvalidValue;
  Params p = make_params(c, a, a.a_fmt, a.b_fmt, TILE_ROWS);
  p.early = a.early;
  const long long tiles = (a.rows + static_cast<long long>(std::min(a.G, a.rows)) * (TILE_ROWS - 1)) / TILE_ROWS;
  const long long items = tiles * (DUAL ? p.n_tiles : (p.n_tiles + 1) / 2);
  auto kern = fp8_rows_gemm_kernel<DUAL>;
  const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(kern), static_cast<int>(SMEM));
  if (e != cudaSuccess) return e;
  KernelScope ks(c, a.rows_name);
  return launch_kernel(c, kern, dim3(static_cast<unsigned>(std::min<long long>(c.num_sms, items))), dim3(THREADS), SMEM,
                       mA, m0, m1, p);
}

}  // namespace

cudaError_t launch_fp8_rows_gemm(const Ctx& c, const Fp8GemmArgs& a) {
  return a.dual ? launch_typed<true>(c, a) : launch_typed<false>(c, a);
}

}  // namespace moe
