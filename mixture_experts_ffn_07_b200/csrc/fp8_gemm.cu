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
#include "fp8_mma.cuh"

namespace moe {

namespace {

constexpr int BOX = 32;            // token rows per TMA box
constexpr int SLOTS = 8;           // k-blocks of scales in flight
constexpr int PITCH8 = 144;        // dual: staged bytes per row of codes (128 used)
constexpr int PITCH16 = 80;        // single: staged bytes per row of 32 bf16 outputs (64 used)

template <bool DUAL, int NT>
struct Cfg {
  static constexpr int MATS = DUAL ? 2 : 1;
  static constexpr int STAGE_BYTES = MATS * W_BYTES + NT * KB;
  static constexpr int ACC = MATS * NT;                      // TMEM columns of one accumulator
  static constexpr int NBUF = 512 / ACC < 8 ? 512 / ACC : 8; // accumulators
  static constexpr uint32_t TMEM_COLS = NBUF * ACC;
  static constexpr int HALF = NT / 2;                        // columns per epilogue warp
  static constexpr int X = HALF / 8 < 8 ? HALF / 8 : 8;      // 8-column groups per TMEM load
  static constexpr int CHUNKS = HALF / (8 * X);
  static constexpr int SCALE_WARPS = NT > 32 ? 2 : 1;
  static constexpr int OUT_STAGE = DUAL ? NT * PITCH8 : EPI_WARPS * 16 * PITCH16;
};

template <bool DUAL, int NT, int STAGES>
struct Aux {
  alignas(16) float sc[SLOTS][DUAL ? 2 : 1][NT];  // row scale x tile scale
  alignas(16) float inv[DUAL ? NT : 4];           // dual: 1 / h scale of each column
  uint32_t red[DUAL ? EPI_WARPS : 1][NT / 2];     // dual: largest |h| of each warp's columns, as bits
  int dest[2][DUAL ? 4 : NT];                     // single: output row of each column (-1: none)
  float rscale[2][DUAL ? 4 : NT];
  uint64_t full[STAGES];
  uint64_t empty[STAGES];
  uint64_t sfull[SLOTS];
  uint64_t sempty[SLOTS];
  uint64_t tfull[8];
  uint64_t tempty[8];
  uint64_t done;
  uint32_t tmem_base;
  int abort;
  int item_off[MAX_G + 1];
  int row_off[MAX_G];
  int cnt[MAX_G];
};

// As many stages as fit beside the rest.
template <bool DUAL, int NT>
constexpr int kStages = (SMEM_MAX - 1024 - static_cast<int>(sizeof(Aux<DUAL, NT, 16>)) - Cfg<DUAL, NT>::OUT_STAGE) /
                        Cfg<DUAL, NT>::STAGE_BYTES;
template <bool DUAL, int NT>
constexpr size_t kSmem = 1024 + static_cast<size_t>(kStages<DUAL, NT>) * Cfg<DUAL, NT>::STAGE_BYTES +
                         Cfg<DUAL, NT>::OUT_STAGE + sizeof(Aux<DUAL, NT, kStages<DUAL, NT>>);

// 16 TMEM lanes x 8 X columns.  Group i of 8 columns: registers 4 i, 4 i + 1 hold columns 2 (lane % 4), + 1 of row
// lane / 4, registers 4 i + 2, 4 i + 3 the same columns of row lane / 4 + 8.  So a thread needs two of the eight
// column scales, not all of them (reading 32 lanes x 1 column instead cost one shared load per four products).
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
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
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])::"memory");
}

// Four 8 x 8 matrices of 16-bit values, transposed: lane l gives the address of column l % 8 of matrix l / 8.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
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

template <bool DUAL, int NT>
__global__ void __launch_bounds__(THREADS, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapW0,
                    const __grid_constant__ CUtensorMap mapW1, const Params p) {
  using C = Cfg<DUAL, NT>;
  constexpr int STAGES = kStages<DUAL, NT>;
  constexpr int NBUF = C::NBUF;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* out_stage = smem + STAGES * C::STAGE_BYTES;
  Aux<DUAL, NT, STAGES>& aux = *reinterpret_cast<Aux<DUAL, NT, STAGES>*>(out_stage + C::OUT_STAGE);
  volatile int* abort_flag = &aux.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&aux.full[s], 1);
      mbar_init(&aux.empty[s], 1);
    }
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(&aux.sfull[s], C::SCALE_WARPS);
      mbar_init(&aux.sempty[s], EPI_WARPS);
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
            const int bytes = C::MATS * W_BYTES + boxes * BOX * KB;
            mbar_arrive_expect_tx(&aux.full[s], bytes);
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
            const int buf = kbg % NBUF;
            if (!mbar_wait_bounded(&aux.tempty[buf], ((kbg / NBUF) & 1u) ^ 1u, limit, abort_flag) ||
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
    } else if (warp - 2 < C::SCALE_WARPS) {
      // ---------------------------------------------------------- scales: warp 2 + i has the i-th part of the columns.
      // AHEAD k-blocks are in flight per warp (a load takes about 1000 cycles, a k-block about 500).
      constexpr int PER = NT / 32 / C::SCALE_WARPS, AHEAD = 4;
      const int col0 = (warp - 2) * 32 * PER + lane;
      uint32_t kbg = 0;
      bool ok = true;
      for (int w = blockIdx.x; w < total && ok; w += gridDim.x) {
        const Item it = decode_item<NT>(aux, p.G, w);
        int at[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const int r = it.row0 + min(col0 + 32 * j, it.n - 1);
          int col = p.a_scale_map ? p.a_scale_map[r] / p.a_scale_div : r;
          col = min(max(col, 0), static_cast<int>(p.a_ld) - 1);
          at[j] = col;
        }
        const long long sb = (static_cast<long long>(it.g) * p.n_tiles + it.wt) * nkb;
        float v[AHEAD][PER], t0[AHEAD], t1[AHEAD];
        auto load = [&](int kb, int b) {
          const int k = min(kb, nkb - 1);
#pragma unroll
          for (int j = 0; j < PER; ++j) v[b][j] = __ldg(p.a_scale + k * p.a_ld + at[j]);
          t0[b] = __ldg(p.s0 + sb + k);
          t1[b] = DUAL ? __ldg(p.s1 + sb + k) : 0.f;
        };
#pragma unroll
        for (int b = 0; b < AHEAD; ++b) load(b, b);
        for (int kb0 = 0; kb0 < nkb && ok; kb0 += AHEAD) {
#pragma unroll
          for (int b = 0; b < AHEAD; ++b) {
            if (kb0 + b >= nkb) break;
            const int slot = kbg % SLOTS;
            const bool got = mbar_wait_bounded(&aux.sempty[slot], ((kbg / SLOTS) & 1u) ^ 1u, limit, abort_flag);
            if (!__all_sync(0xffffffffu, got)) {
              ok = false;
              break;
            }
#pragma unroll
            for (int j = 0; j < PER; ++j) {
              aux.sc[slot][0][col0 + 32 * j] = v[b][j] * t0[b];
              if (DUAL) aux.sc[slot][C::MATS - 1][col0 + 32 * j] = v[b][j] * t1[b];
            }
            load(kb0 + b + AHEAD, b);
            __syncwarp();
            if (lane == 0) mbar_arrive(&aux.sfull[slot]);
            ++kbg;
          }
        }
      }
    }
  } else {
    // -------------------------------------------------------------- epilogue
    constexpr int HALF = C::HALF, X = C::X, CHUNKS = C::CHUNKS, MATS = C::MATS;
    constexpr int STEPS = MATS * CHUNKS * 2;  // TMEM loads per k-block: (matrix, column chunk, 16-lane half)
    const int ew = warp - 4;
    const int q = warp & 3, half = ew >> 2;
    const int et = threadIdx.x - 128;  // thread of the epilogue
    const int lr = lane >> 2, lc = 2 * (lane & 3);  // row and column inside an 8 x 8 block
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    uint32_t kbg = 0;
    int parity = 0;
    for (int w = blockIdx.x; w < total; w += gridDim.x, parity ^= 1) {
      const Item it = decode_item<NT>(aux, p.G, w);
      const int wt = it.wt;
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
      // acc[m][chunk][half of the lanes][2 i + b]: columns 8 (chunk X + i) + lc, + 1 of row 16 half + 8 b + lr
      unsigned long long acc[MATS][CHUNKS][2][2 * X];
#pragma unroll
      for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
          for (int j = 0; j < 2 * X; ++j) acc[m][c][0][j] = acc[m][c][1][j] = 0ull;
      bool ok = true;
      for (int kb = 0; kb < nkb; ++kb, ++kbg) {
        const int slot = kbg % SLOTS, buf = kbg % NBUF;
        const bool got = mbar_wait_bounded(&aux.sfull[slot], (kbg / SLOTS) & 1u, limit, abort_flag) &&
                         mbar_wait_bounded(&aux.tfull[buf], (kbg / NBUF) & 1u, limit, abort_flag);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (half * HALF < n16) {  // warp-uniform
          const uint32_t tb = tmem_base + lane_base + buf * C::ACC + half * HALF;
          unsigned long long sc[X];
#pragma unroll
          for (int st = 0; st < STEPS; ++st) {
            const int m = st / (2 * CHUNKS), c = st / 2 % CHUNKS, r = st & 1;
            uint32_t v[4 * X];
            tmem_ld_16x256b(tb + (static_cast<uint32_t>(16 * r) << 16) + m * NT + c * 8 * X, v);
            if (r == 0) {
#pragma unroll
              for (int i = 0; i < X; ++i)
                sc[i] = *reinterpret_cast<const unsigned long long*>(&aux.sc[slot][m][half * HALF + 8 * (c * X + i) + lc]);
            }
            tmem_wait(v);
#pragma unroll
            for (int i = 0; i < X; ++i) {
              fma2(acc[m][c][r][2 * i], v[4 * i], v[4 * i + 1], sc[i]);
              fma2(acc[m][c][r][2 * i + 1], v[4 * i + 2], v[4 * i + 3], sc[i]);
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
      if (DUAL) {
        // h = act(g) * u in place of g, and the largest |h| of each of the thread's 2 X columns over its four rows
        const ActCoef ac = act_coef(p.act);
        uint32_t mx[2 * X];
#pragma unroll
        for (int i = 0; i < X; ++i) {
          mx[2 * i] = mx[2 * i + 1] = 0;
#pragma unroll
          for (int rb = 0; rb < 4; ++rb) {
            float g0, g1, u0, u1;
            split2(acc[0][0][rb >> 1][2 * i + (rb & 1)], g0, g1);
            split2(acc[MATS - 1][0][rb >> 1][2 * i + (rb & 1)], u0, u1);
            const float h0 = act_fast(ac, g0) * u0, h1 = act_fast(ac, g1) * u1;
            acc[0][0][rb >> 1][2 * i + (rb & 1)] = join2(h0, h1);
            mx[2 * i] = max(mx[2 * i], __float_as_uint(h0) & 0x7fffffffu);
            mx[2 * i + 1] = max(mx[2 * i + 1], __float_as_uint(h1) & 0x7fffffffu);
          }
        }
        // over the warp's 32 rows: halve the columns a lane keeps while exchanging with lanes 16, 8, 4 away
        int base = 0;
#pragma unroll
        for (int b = 0; b < 3; ++b) {
          constexpr int N0 = 2 * X;
          const int keep = N0 >> (b + 1);
          const int o = 16 >> b;
          const bool upper = lane & o;
          if (keep > 0) {
#pragma unroll
            for (int j = 0; j < keep; ++j) {
              const uint32_t give = upper ? mx[j] : mx[j + keep], take = upper ? mx[j + keep] : mx[j];
              mx[j] = max(take, __shfl_xor_sync(0xffffffffu, give, o));
            }
            base += upper ? keep : 0;
          } else {
            mx[0] = max(mx[0], __shfl_xor_sync(0xffffffffu, mx[0], o));
          }
        }
        constexpr int LEFT = 2 * X / 8 > 1 ? 2 * X / 8 : 1;
#pragma unroll
        for (int j = 0; j < LEFT; ++j) {
          const int k = base + j;  // the thread's column k: group k / 2, parity k % 2
          aux.red[ew][8 * (k >> 1) + lc + (k & 1)] = mx[j];
        }
        named_barrier(2 + half, 128);
        if (et - half * 128 < HALF) {
          const int c = et - half * 128;
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) m = max(m, aux.red[half * 4 + i][c]);
          float scale, inv;
          fp8_scale(m, MOE_E4M3, false, scale, inv);
          const int col = half * HALF + c;
          aux.inv[col] = inv;
          if (col < it.n) p.out_qs[static_cast<long long>(wt) * p.rows + it.row0 + col] = scale;
        }
        named_barrier(2 + half, 128);
        uint8_t* stage = out_stage + half * HALF * PITCH8;
#pragma unroll
        for (int i = 0; i < X; ++i) {
          const float2 inv = *reinterpret_cast<const float2*>(&aux.inv[half * HALF + 8 * i + lc]);
          uint8_t* o = stage + (8 * i + lc) * PITCH8 + q * 32 + lr;
#pragma unroll
          for (int rb = 0; rb < 4; ++rb) {
            float h0, h1;
            split2(acc[0][0][rb >> 1][2 * i + (rb & 1)], h0, h1);
            const uint32_t code = fp8_pack2(h0 * inv.x, h1 * inv.y, MOE_E4M3);
            o[8 * rb] = static_cast<uint8_t>(code);
            o[8 * rb + PITCH8] = static_cast<uint8_t>(code >> 8);
          }
        }
        named_barrier(2 + half, 128);
        // whole rows of 128 codes: eight lanes a row
        const int ch = et & 7;
        if (wt * WM + ch * 16 < p.N) {
#pragma unroll
          for (int c0 = 0; c0 < HALF; c0 += 16) {
            const int c = c0 + ((et & 127) >> 3);
            const int col = half * HALF + c;
            if (col < it.n)
              *reinterpret_cast<uint4*>(p.out_q + static_cast<long long>(it.row0 + col) * p.N + wt * WM + ch * 16) =
                  *reinterpret_cast<const uint4*>(stage + c * PITCH8 + ch * 16);
          }
        }
      } else if (wt * WM + q * 32 < p.N) {  // N is a multiple of 32: the warp's rows are all inside or all outside
        if (p.out_bf16) {
          // 16 columns at a time through the warp's staging rows: [column][32 rows] bf16
          uint8_t* stage = out_stage + ew * 16 * PITCH16;
          const uint32_t st_addr = smem_addr(stage) + (lane & 7) * PITCH16 + (lane >> 3) * 16;
          const int ch = lane & 3;
#pragma unroll
          for (int i = 0; i < CHUNKS * X; i += 2) {
            if (half * HALF + 8 * i >= it.n) break;  // warp-uniform
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              uint32_t pk[4];
              const int col = half * HALF + 8 * (i + e) + lc;
              const float s0 = aux.rscale[parity][col], s1 = aux.rscale[parity][col + 1];
#pragma unroll
              for (int rb = 0; rb < 4; ++rb) {
                float y0, y1;
                split2(acc[0][(i + e) / X][rb >> 1][2 * ((i + e) % X) + (rb & 1)], y0, y1);
                const __nv_bfloat162 t = __floats2bfloat162_rn(y0 * s0, y1 * s1);
                pk[rb] = *reinterpret_cast<const uint32_t*>(&t);
              }
              stmatrix_x4_trans(st_addr + e * 8 * PITCH16, pk[0], pk[1], pk[2], pk[3]);
            }
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int c = 8 * e + lr;
              const int d = aux.dest[parity][half * HALF + 8 * i + c];
              const uint4 v = *reinterpret_cast<const uint4*>(stage + c * PITCH16 + ch * 16);
              if (d >= 0)
                *reinterpret_cast<uint4*>(p.out_bf16 + static_cast<long long>(d) * p.N + wt * WM + q * 32 + ch * 8) = v;
            }
            __syncwarp();
          }
        } else {
#pragma unroll
          for (int i = 0; i < CHUNKS * X; ++i) {
            const int col = half * HALF + 8 * i + lc;
            const int d0 = aux.dest[parity][col], d1 = aux.dest[parity][col + 1];
            const float s0 = aux.rscale[parity][col], s1 = aux.rscale[parity][col + 1];
            float* o = p.out_f32 + wt * WM + q * 32 + lr;
#pragma unroll
            for (int rb = 0; rb < 4; ++rb) {
              float y0, y1;
              split2(acc[0][i / X][rb >> 1][2 * (i % X) + (rb & 1)], y0, y1);
              if (d0 >= 0) o[static_cast<long long>(d0) * p.N + 8 * rb] = y0 * s0;
              if (d1 >= 0) o[static_cast<long long>(d1) * p.N + 8 * rb] = y1 * s1;
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
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
  if (threadIdx.x == 0 && aux.abort) record_status(p.status, MOE_ERR_TIMEOUT);
}

// ------------------------------------------------------------------ host side
template <bool DUAL, int NT>
cudaError_t launch_typed(const Ctx& c, const Fp8GemmArgs& a) {
  CUtensorMap mA, m0, m1;
  if (!make_maps(a, BOX, &mA, &m0, &m1)) return cudaErrorInvalidValue;
  const Params p = make_params(c, a, a.b_fmt, a.a_fmt, WM);
  const long long tiles = a.rows / 16 < a.G ? a.rows : a.rows / 16 + a.G;  // no fewer than there can be
  const int grid = static_cast<int>(std::max(1LL, std::min<long long>(c.num_sms, tiles * p.n_tiles)));
  auto kern = fp8_gemm_kernel<DUAL, NT>;
  constexpr size_t smem = kSmem<DUAL, NT>;
  static_assert(smem <= SMEM_MAX && kStages<DUAL, NT> >= 3 && kStages<DUAL, NT> <= 16, "stages");
  const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(kern), static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  KernelScope ks(c, a.name ? a.name : "fp8_gemm");
  return launch_kernel(c, kern, dim3(grid), dim3(THREADS), smem, mA, m0, m1, p);
}

}  // namespace

cudaError_t launch_fp8_gemm(const Ctx& c, const Fp8GemmArgs& a) {
  if (a.rows <= 0 || a.G <= 0) return cudaSuccess;
  if (a.G > MAX_G || a.N % 32 || a.K % 32 || a.N <= 0 || a.K <= 0) return cudaErrorInvalidValue;
  // Mean rows of a group, of the groups that can hold any.  Measured crossovers with fp8_gemm_rows.cu (64 experts, K and N
  // of 1024 and 2048): gate/up 62 us here and 71 us there at 48 rows, 76 and 72 us at 64; down 37 and 35 us at 16,
  // 41 and 35 us at 24.
  const double rows = static_cast<double>(a.rows) / std::min(a.G, a.rows);
  if (rows > (a.dual ? 48.0 : 16.0)) return launch_fp8_rows_gemm(c, a);
  if (!a.dual) return launch_typed<false, 32>(c, a);
  return rows > 16.0 ? launch_typed<true, 64>(c, a) : launch_typed<true, 32>(c, a);
}

}  // namespace moe
