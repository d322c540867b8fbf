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
// A k-block of 128 is four MMAs of K = 32 into one of the TMEM accumulators; the epilogue warps read each finished
// k-block out of TMEM and add it, scaled, to f32 registers while the next ones run.
//  * warp 0: TMA producer (weight tiles 128 x 128 bytes; token rows in boxes of 32, 128-byte swizzle, or, for the
//    routed gate/up, gathered row by row straight from the tokens with tile::gather4);
//  * warp 1: allocates TMEM, issues tcgen05.mma kind::f8f6f4 from one lane; warp 3 issues every second k-block: each
//    has an accumulator of its own, and a k-block costs its issuer two barrier waits, four
//    instructions and a commit, 600-800 cycles, more than its copies take;
//  * warp 2: loads the scales of each k-block, multiplies row and tile scale, into a ring;
//  * warps 4-11: epilogue; warp w reads TMEM lanes 32 (w % 4), and one half of the columns, or, with at most 16 rows,
//    every second k-block.
// A k-block's stage and accumulator have the same number, and one commit frees the stage and fills the accumulator.
//
// Few items (one decoded token: experts x weight tiles, fewer than SMs) split K over a cluster of up to eight CTAs:
// each sums its k-blocks, leaves the sums in its shared memory, and the first CTA adds them in rank order.
// What bounds it: HBM with many experts touched (16 tokens, 128 experts of 2816 x 704: 490 MB in 80 us, 0.95 of the copy
// rate), latency with few (16 x 2048 x 7168: 11 us, 2.3 of them for its 15 MB).
// Every wait is bounded; on expiry the CTA records MOE_ERR_TIMEOUT, drains and exits.
#include <atomic>

#include "fp8_mma.cuh"

namespace moe {

namespace {

constexpr int NT = 32;             // token rows of a tile, one TMA box
constexpr int HALF = NT / 2;       // columns per epilogue warp
constexpr int X = HALF / 8;        // 8-column groups per TMEM load
constexpr int MMA_WARPS = 2;
constexpr int PITCH8 = 144;        // dual: staged bytes per row of codes (128 used)
constexpr int PITCH16 = 80;        // single: staged bytes per row of 32 bf16 outputs (64 used)

template <bool DUAL>
struct Cfg {
  static constexpr int MATS = DUAL ? 2 : 1;
  static constexpr int STAGE_BYTES = MATS * W_BYTES + NT * KB;
  static constexpr int ACC = MATS * NT;                      // TMEM columns of one accumulator
  // Stages, and accumulators.  An even number: a k-block's stage then always belongs to the same MMA warp and, with at
  // most 16 rows, to the same half of the epilogue, so each of them sees every phase of the barriers that it waits for
  // (waiting for a phase by its parity while the one before is still open would pass at once).
  static constexpr int RING = DUAL ? 4 : 8;
  static_assert(RING % 2 == 0, "phases");
  static constexpr uint32_t TMEM_COLS = 256;
  static_assert(RING * ACC <= 256, "TMEM columns");
  // Ring of scales.  The scale warps write a k-block's slot after its stage came free, that is after the MMA RING
  // k-blocks earlier, which the epilogue's reads of the k-block RING before that one (values and scales) precede: a
  // slot 2 RING k-blocks old is read, and the ring needs no barriers of its own.
  static constexpr int SLOTS = 16;
  static_assert(SLOTS >= 2 * RING, "ring of scales");
  static constexpr int OUT_STAGE = DUAL ? NT * PITCH8 : EPI_WARPS * 16 * PITCH16;
};

struct Item {
  int g, wt, row0, n;  // group, weight tile, first row, rows
  bool alone;          // the group has one token tile: its weights are read once
};

template <bool DUAL>
struct Aux {
  alignas(16) float sc[Cfg<DUAL>::SLOTS][DUAL ? 2 : 1][NT];  // row scale x tile scale
  alignas(16) float inv[DUAL ? NT : 4];           // dual: 1 / h scale of each column
  uint32_t red[DUAL ? EPI_WARPS : 1][NT / 2];     // dual: largest |h| of each warp's columns, as bits
  int dest[2][DUAL ? 4 : NT];                     // single: output row of each column (-1: none)
  float rscale[2][DUAL ? 4 : NT];
  unsigned long long alt[Cfg<DUAL>::MATS * 8][EPI_WARPS * 16];  // at most 16 rows: the second half's sums
  uint64_t full[Cfg<DUAL>::RING];
  uint64_t done[Cfg<DUAL>::RING];    // the k-block's MMAs: its stage is free and its accumulator full
  uint64_t tempty[Cfg<DUAL>::RING];
  uint64_t all_done;
  uint32_t tmem_base;
  int abort;
  int item_off[MAX_G + 1];
  int row_off[MAX_G];
  int cnt[MAX_G];
  Item first;  // this CTA's first item
};

template <bool DUAL>
constexpr size_t kSmem = 1024 + static_cast<size_t>(Cfg<DUAL>::RING) * Cfg<DUAL>::STAGE_BYTES +
                         Cfg<DUAL>::OUT_STAGE + sizeof(Aux<DUAL>);

// 16 TMEM lanes x 8 X columns.  Group i of 8 columns: registers 4 i, 4 i + 1 hold columns 2 (lane % 4), + 1 of row
// lane / 4, registers 4 i + 2, 4 i + 3 the same columns of row lane / 4 + 8.  So a thread needs two of the eight
// column scales, not all of them (reading 32 lanes x 1 column instead cost one shared load per four products).
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
// Waits for the thread's TMEM loads; names the registers, so that nothing reads them earlier.
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

// Item `local` of group g: its tiles of NT rows, every one against the same weight tile before the next weight tile.
template <typename AuxT>
__device__ __forceinline__ Item item_at(const AuxT& aux, int g, int local) {
  Item it;
  it.g = g;
  const int cnt = aux.cnt[g];
  const int tiles = (cnt + NT - 1) / NT;
  it.alone = tiles == 1;
  it.wt = it.alone ? local : local / tiles;
  const int tt = local - it.wt * tiles;
  it.row0 = aux.row_off[g] + tt * NT;
  it.n = min(NT, cnt - tt * NT);
  return it;
}
template <typename AuxT>
__device__ __forceinline__ Item decode_item(const AuxT& aux, int G, int w) {
  int lo = 0, hi = G - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (aux.item_off[mid] <= w)
      lo = mid;
    else
      hi = mid - 1;
  }
  return item_at(aux, lo, w - aux.item_off[lo]);
}

// The two halves of a barrier over every thread of the cluster (whole warps); they order the shared-memory accesses
// around them.
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// What every role but the epilogue does at the end of an item whose k-blocks a cluster shares.
__device__ __forceinline__ void pass_item(bool split) {
  if (split) {
    cluster_arrive();
    cluster_wait();
    cluster_arrive();
    cluster_wait();
  }
}
__device__ __forceinline__ unsigned long long ld_cluster(uint32_t cluster_address) {
  unsigned long long v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(cluster_address) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t cluster_id() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t clusters() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%nclusterid.x;" : "=r"(r));
  return r;
}

template <bool DUAL>
__global__ void __launch_bounds__(THREADS, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapW0,
                    const __grid_constant__ CUtensorMap mapW1, const Params p) {
  using C = Cfg<DUAL>;
  constexpr int RING = C::RING;
  constexpr int SLOTS = C::SLOTS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* out_stage = smem + RING * C::STAGE_BYTES;
  Aux<DUAL>& aux = *reinterpret_cast<Aux<DUAL>*>(out_stage + C::OUT_STAGE);
  volatile int* abort_flag = &aux.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool split = p.split > 1;
  const int rank = split ? static_cast<int>(cluster_ctarank()) : 0;
  const int first = split ? cluster_id() : blockIdx.x, step = split ? clusters() : gridDim.x;

  if (threadIdx.x == 0) {
    for (int s = 0; s < RING; ++s) {
      mbar_init(&aux.full[s], 2);  // the producer and the scale warp
      mbar_init(&aux.done[s], 1);
      mbar_init(&aux.tempty[s], EPI_WARPS);
    }
    mbar_init(&aux.all_done, MMA_WARPS);
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
  // p.early (the down projection behind its own gate/up, whose launch waited for everything before it before it let
  // this one start): the offsets and the weights are there already, so the weights' copies start at once, while
  // the last CTAs of the launch before still run; what that launch writes is read after pdl_wait.
  if (!p.early) pdl_wait();
  pdl_trigger();
  if (warp == 0) {  // rows and work items of each group; lane owns groups [8 lane, 8 lane + 8)
    int off[9], v[8], local = 0;
#pragma unroll
    for (int i = 0; i < 9; ++i) {
      const int g = lane * 8 + i;
      off[i] = p.offsets && g <= p.G ? p.offsets[g] : (g == 0 ? 0 : p.rows);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int g = lane * 8 + i;
      v[i] = 0;
      if (g < p.G) {
        // a group's rows stay inside the tensor, whatever the offsets hold
        const int r0 = min(max(off[i], 0), p.rows), r1 = min(max(off[i + 1], r0), p.rows);
        if (r0 != off[i] || r1 != off[i + 1]) record_status(p.status, MOE_ERR_DEVICE_INDEX);
        aux.row_off[g] = r0;
        aux.cnt[g] = r1 - r0;
        v[i] = (r1 - r0 + NT - 1) / NT * p.n_tiles;
      }
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
      if (run <= first && first < run + v[i]) aux.first = item_at(aux, g, first - run);
      run += v[i];
    }
    if (lane == 31) aux.item_off[p.G] = incl;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem_base = aux.tmem_base;
  const int total = aux.item_off[p.G];
  const int nkb_all = (p.K + KB - 1) / KB;
  // this CTA's k-blocks
  const int kb_lo = rank * p.kb_per, kb_hi = min(nkb_all, kb_lo + p.kb_per);
  const long long limit = p.wait_limit;
  // With split every role passes two cluster barriers per item (before and after the first CTA's reads), whether its
  // CTA still works or has given up.

  if (warp == 0) {
    // ---------------------------------------------------------- TMA producer (whole warp: lane l gathers rows
    // [4 l, 4 l + 4) of a tile, lane 0 does the rest)
    uint32_t kbg = 0, outstanding = 0, out_phase = 0;
    bool ok = true;
    const uint64_t pol_first = l2_policy_evict_first(), pol_normal = l2_policy_evict_normal(),
                   pol_last = l2_policy_evict_last();
    for (int w = first; w < total; w += step) {
      ok = ok && !__shfl_sync(0xffffffffu, *abort_flag, 0);
      if (ok) {
        const Item it = w == first ? aux.first : decode_item(aux, p.G, w);
        const int quads = (it.n + 3) / 4;
        const uint64_t pol_w = it.alone ? pol_first : pol_normal;
        int tok[4] = {0, 0, 0, 0};
        if (p.gather && lane < quads)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int t = p.a_scale_map[it.row0 + min(4 * lane + j, it.n - 1)] / p.a_scale_div;
            tok[j] = min(max(t, 0), static_cast<int>(p.a_ld) - 1);
          }
        const int bytes = C::MATS * W_BYTES + (p.gather ? quads * 4 : NT) * KB;
        int done = 0;  // k-blocks of this item already requested
        if (w == first) {
          // The first item's first stages are free, and a lane fills each: waiting for and arriving on a barrier takes
          // a lane a few hundred cycles, which one lane would spend stage after stage.  Weights before rows, whose
          // indexes (gathered) or values (early) are still on their way.
          const int fill = min(RING, kb_hi - kb_lo);
          const bool mine = lane < fill && !(p.skip_stage && lane == 0 && blockIdx.x == 0);  // debug: one stage unfilled
          uint8_t* st = smem + lane * C::STAGE_BYTES;
          const int x = (kb_lo + lane) * KB;
          if (mine) {
            mbar_arrive_expect_tx(&aux.full[lane], bytes);
            tma_load_3d(st, &mapW0, &aux.full[lane], x, it.wt * WM, it.g, pol_w);
            if (DUAL) tma_load_3d(st + W_BYTES, &mapW1, &aux.full[lane], x, it.wt * WM, it.g, pol_w);
          }
          if (p.early) pdl_wait();
          if (p.gather) {
            for (int b = 0; b < quads; ++b) {
              int t[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) t[j] = __shfl_sync(0xffffffffu, tok[j], b);
              if (mine)
                tma_gather4(st + C::MATS * W_BYTES + b * 4 * KB, &mapA, &aux.full[lane], x, t[0], t[1], t[2], t[3],
                            pol_last);
            }
          } else if (mine) {
            tma_load_2d_hint(st + C::MATS * W_BYTES, &mapA, &aux.full[lane], x, it.row0, pol_last);
          }
          __syncwarp();
          outstanding = (1u << fill) - 1u;
          done = fill;
        }
        for (int n = done; n < kb_hi - kb_lo; ++n) {
          const int kb = kb_lo + n;
          const uint32_t k = kbg + n;
          const int s = k % RING;
          const uint32_t ph = (k / RING) & 1u;
          int got = 1;
          if (lane == 0) got = mbar_wait_bounded(&aux.done[s], ph ^ 1u, limit, abort_flag);
          if (!__shfl_sync(0xffffffffu, got, 0)) break;
          outstanding &= ~(1u << s);
          uint8_t* st = smem + s * C::STAGE_BYTES;
          uint8_t* sa = st + C::MATS * W_BYTES;
          if (lane == 0) {
            mbar_arrive_expect_tx(&aux.full[s], bytes);
            tma_load_3d(st, &mapW0, &aux.full[s], kb * KB, it.wt * WM, it.g, pol_w);
            if (DUAL) tma_load_3d(st + W_BYTES, &mapW1, &aux.full[s], kb * KB, it.wt * WM, it.g, pol_w);
          }
          __syncwarp();
          if (p.gather) {
            if (lane < quads)
              tma_gather4(sa + lane * 4 * KB, &mapA, &aux.full[s], kb * KB, tok[0], tok[1], tok[2], tok[3], pol_last);
          } else if (lane == 0) {
            tma_load_2d_hint(sa, &mapA, &aux.full[s], kb * KB, it.row0, pol_last);
          }
          outstanding |= 1u << s;
          out_phase = (out_phase & ~(1u << s)) | (ph << s);
        }
        kbg += kb_hi - kb_lo;
      }
      pass_item(split);
    }
    if (lane == 0 && *abort_flag)  // let issued copies land before the CTA exits
      for (int s = 0; s < RING; ++s)
        if (outstanding & (1u << s)) wait_cycles(&aux.full[s], (out_phase >> s) & 1u, limit);
  } else if (warp == 1 || warp == 3) {
    // ---------------------------------------------------------- MMA issuers (one lane; k-blocks in turn)
    const uint32_t mine = warp >> 1;
    uint32_t kbg = 0;
    bool ok = true;
    for (int w = first; w < total; w += step) {
      if (lane == 0 && ok) {
        const Item it = w == first ? aux.first : decode_item(aux, p.G, w);
        const uint32_t n16 = (it.n + 15) & ~15;
        const uint32_t idesc = p.idesc | ((n16 >> 3) << 17);
        for (int kb = kb_lo; kb < kb_hi; ++kb, ++kbg) {
          if ((kbg & 1u) != mine) continue;
          const int s = kbg % RING;
          const uint32_t round = kbg / RING;
          if ((round > 0 && !mbar_wait_bounded(&aux.tempty[s], (round & 1u) ^ 1u, limit, abort_flag)) ||
              !mbar_wait_bounded(&aux.full[s], round & 1u, limit, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = smem_addr(smem + s * C::STAGE_BYTES);
          const uint64_t tdesc = sw128_kmajor_desc(st + C::MATS * W_BYTES);
#pragma unroll
          for (int m = 0; m < C::MATS; ++m) {
            const uint64_t wdesc = sw128_kmajor_desc(st + m * W_BYTES);
            const uint32_t d = tmem_base + s * C::ACC + m * NT;
#pragma unroll
            for (int kk = 0; kk < KB / 32; ++kk)
              umma_f8(d, wdesc + static_cast<uint64_t>(kk * 2), tdesc + static_cast<uint64_t>(kk * 2), idesc,
                      kk > 0 ? 1u : 0u);
          }
          umma_commit(&aux.done[s]);
        }
      }
      pass_item(split);
    }
    if (lane == 0) {
      umma_commit(&aux.all_done);  // every MMA issued completes before TMEM is released
      wait_cycles(&aux.all_done, 0, limit);
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------- scales: AHEAD k-blocks are in flight (a load takes
    // about 1000 cycles)
    constexpr int AHEAD = 4;
    uint32_t kbg = 0;
    bool ok = true;
    if (p.early) pdl_wait();
    for (int w = first; w < total; w += step) {
      if (ok) {
        const Item it = w == first ? aux.first : decode_item(aux, p.G, w);
        const int r = it.row0 + min(lane, it.n - 1);
        const int col = p.a_scale_map ? p.a_scale_map[r] / p.a_scale_div : r;
        const int at = min(max(col, 0), static_cast<int>(p.a_ld) - 1);
        const long long sb = (static_cast<long long>(it.g) * p.n_tiles + it.wt) * nkb_all;
        float v[AHEAD], t0[AHEAD], t1[AHEAD];
        auto load = [&](int kb, int b) {
          const int k = min(kb, nkb_all - 1);
          v[b] = p.a_scale[k * p.a_ld + at];
          t0[b] = p.s0[sb + k];
          t1[b] = DUAL ? p.s1[sb + k] : 0.f;
        };
#pragma unroll
        for (int b = 0; b < AHEAD; ++b) load(kb_lo + b, b);
        for (int kb0 = kb_lo; kb0 < kb_hi && ok; kb0 += AHEAD) {
#pragma unroll
          for (int b = 0; b < AHEAD; ++b) {  // unrolled, so that a scale in flight is never moved between registers
            if (kb0 + b >= kb_hi) break;
            const int s = kbg % RING;
            const bool got = mbar_wait_bounded(&aux.done[s], ((kbg / RING) & 1u) ^ 1u, limit, abort_flag);
            if (!__all_sync(0xffffffffu, got)) {
              ok = false;
              break;
            }
            const int slot = kbg % SLOTS;
            aux.sc[slot][0][lane] = v[b] * t0[b];
            if (DUAL) aux.sc[slot][C::MATS - 1][lane] = v[b] * t1[b];
            load(kb0 + b + AHEAD, b);
            __syncwarp();
            if (lane == 0) mbar_arrive(&aux.full[s]);
            ++kbg;
          }
        }
      }
      pass_item(split);
    }
  } else {
    // ---------------------------------------------------------- epilogue
    constexpr int MATS = C::MATS;
    constexpr int STEPS = MATS * 2;  // TMEM loads per k-block: (matrix, 16-lane half)
    const int ew = warp - 4;
    const int q = warp & 3, half = ew >> 2;
    const int et = threadIdx.x - 128;  // thread of the epilogue
    const int lr = lane >> 2, lc = 2 * (lane & 3);  // row and column inside an 8 x 8 block
    const uint32_t lane_base = static_cast<uint32_t>(q * 32) << 16;
    uint32_t kbg = 0;
    int parity = 0;
    bool alive = true;
    if (p.early) pdl_wait();
    for (int w = first; w < total; w += step, parity ^= 1) {
      const Item it = w == first ? aux.first : decode_item(aux, p.G, w);
      const int wt = it.wt;
      const int n16 = (it.n + 15) & ~15;
      const bool alt = it.n <= 16;  // the halves take k-blocks in turn, both the first 16 columns
      const int col0 = alt ? 0 : half * HALF;
      // single: thread c < NT has column c's output row, first looked at after the k-blocks
      int d = et < it.n ? it.row0 + et : -1;
      if (!DUAL && et < it.n && p.row_map) d = p.row_map[it.row0 + et];
      // acc[m][half of the lanes][2 i + b]: columns 8 i + lc, + 1 of row 16 half + 8 b + lr
      unsigned long long acc[MATS][2][2 * X];
#pragma unroll
      for (int m = 0; m < MATS; ++m)
#pragma unroll
        for (int j = 0; j < 2 * X; ++j) acc[m][0][j] = acc[m][1][j] = 0ull;
      bool ok = alive;
      for (int kb = kb_lo; kb < kb_hi && ok; ++kb, ++kbg) {
        // (the barrier after the item's last k-block closes the phases that the other half has waited for)
        if (alt && (kbg & 1u) != half) continue;
        const int slot = kbg % SLOTS, buf = kbg % RING;
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(&aux.done[buf], (kbg / RING) & 1u, limit, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (col0 < n16) {  // warp-uniform
          const uint32_t tb = tmem_base + lane_base + buf * C::ACC + col0;
          unsigned long long sc[X];
#pragma unroll
          for (int st = 0; st < STEPS; ++st) {
            const int m = st >> 1, r = st & 1;
            uint32_t v[4 * X];
            tmem_ld_16x256b(tb + (static_cast<uint32_t>(16 * r) << 16) + m * NT, v);
            if (r == 0) {
#pragma unroll
              for (int i = 0; i < X; ++i)
                sc[i] = *reinterpret_cast<const unsigned long long*>(&aux.sc[slot][m][col0 + 8 * i + lc]);
            }
            tmem_wait(v);
#pragma unroll
            for (int i = 0; i < X; ++i) {
              fma2(acc[m][r][2 * i], v[4 * i], v[4 * i + 1], sc[i]);
              fma2(acc[m][r][2 * i + 1], v[4 * i + 2], v[4 * i + 3], sc[i]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&aux.tempty[buf]);
          if (alt) mbar_arrive(&aux.tempty[buf]);  // for the other half's warp
        }
      }
      if (!DUAL && et < NT) {
        float rs = 1.f;
        if (et < it.n) {
          if (d < 0 || d >= p.rows) {
            record_status(p.status, MOE_ERR_DEVICE_INDEX);
            d = -1;
          } else if (p.row_scale) {
            rs = p.row_scale[d];
          }
        }
        aux.dest[parity][et] = d;
        aux.rscale[parity][et] = rs;
      }
      // uniform over the epilogue: either every warp has all k-blocks or the tile is dropped; also orders dest
      alive = named_barrier_and(1, EPI_WARPS * 32, ok);
      if (alt) {
        constexpr int VALS = MATS * 4 * X;
        unsigned long long* flat = &acc[0][0][0];
        unsigned long long* at = &aux.alt[0][et & 127];
        if (half)
#pragma unroll
          for (int j = 0; j < VALS; ++j) at[j * 128] = flat[j];
        named_barrier(1, EPI_WARPS * 32);
#pragma unroll
        for (int j = 0; j < VALS; ++j) flat[j] = half ? 0ull : add2(flat[j], at[j * 128]);
      }
      if (split) {
        // The k-ranges' sums, left in each CTA's first stages (every copy into them has been used) and added in rank
        // order.  Distributed shared memory passes about 20 bytes a cycle, so only columns in use are read; a plain
        // product is added and written by all the CTAs, each a part of the values, h by the first one, which needs
        // whole columns for their scales.
        constexpr int VALS = MATS * 4 * X, PITCH = EPI_WARPS * 32;
        static_assert(VALS * PITCH * 8 <= RING * C::STAGE_BYTES, "partial sums");
        unsigned long long* mine = reinterpret_cast<unsigned long long*>(smem) + et;
        unsigned long long* flat = &acc[0][0][0];  // value j: columns 8 ((j / 2) % X) + lc, + 1 of a row
#pragma unroll
        for (int j = 0; j < VALS; ++j) mine[j * PITCH] = flat[j];
        cluster_arrive();
        cluster_wait();
        if (DUAL) {
          if (rank == 0)
            for (int r = 1; r < p.split; ++r) {
              const uint32_t from = cluster_addr(mine, r);
              unsigned long long v[VALS];
#pragma unroll
              for (int j = 0; j < VALS; ++j) {
                v[j] = 0;
                if (half * HALF + 8 * (j / 2 % X) + lc < it.n) v[j] = ld_cluster(from + j * PITCH * 8);
              }
#pragma unroll
              for (int j = 0; j < VALS; ++j) flat[j] = add2(flat[j], v[j]);
            }
        } else if (alive) {
#pragma unroll
          for (int j = 0; j < VALS; ++j) {
            const int col = half * HALF + 8 * (j / 2 % X) + lc;
            const int n = wt * WM + q * 32 + 16 * (j / (2 * X) % 2) + 8 * (j & 1) + lr;
            if (j % p.split != rank || col >= it.n || n >= p.N) continue;
            unsigned long long v[8];
#pragma unroll
            for (int r = 0; r < 8; ++r)
              if (r < p.split) v[r] = ld_cluster(cluster_addr(mine, r) + j * PITCH * 8);
#pragma unroll
            for (int r = 1; r < 8; ++r)
              if (r < p.split) v[0] = add2(v[0], v[r]);
            float y[2];
            split2(v[0], y[0], y[1]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int d = aux.dest[parity][col + e];
              if (d < 0) continue;
              const float o = y[e] * aux.rscale[parity][col + e];
              if (p.out_bf16)
                p.out_bf16[static_cast<long long>(d) * p.N + n] = __float2bfloat16_rn(o);
              else
                p.out_f32[static_cast<long long>(d) * p.N + n] = o;
            }
          }
        }
        // the next item's copies into those stages come after these generic accesses
        fence_proxy_async_smem();
        cluster_arrive();
        if (!DUAL || rank > 0 || !alive) {
          cluster_wait();
          continue;
        }
      }
      if (!alive) break;
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
            split2(acc[0][rb >> 1][2 * i + (rb & 1)], g0, g1);
            split2(acc[MATS - 1][rb >> 1][2 * i + (rb & 1)], u0, u1);
            const float h0 = act_fast(ac, g0) * u0, h1 = act_fast(ac, g1) * u1;
            acc[0][rb >> 1][2 * i + (rb & 1)] = join2(h0, h1);
            mx[2 * i] = max(mx[2 * i], __float_as_uint(h0) & 0x7fffffffu);
            mx[2 * i + 1] = max(mx[2 * i + 1], __float_as_uint(h1) & 0x7fffffffu);
          }
        }
        // over the warp's 32 rows: halve the columns a lane keeps while exchanging with lanes 16 and 8 away
        static_assert(X == 2, "four columns a thread");
        const bool up16 = lane & 16, up8 = lane & 8;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t give = up16 ? mx[j] : mx[j + 2], keep = up16 ? mx[j + 2] : mx[j];
          mx[j] = max(keep, __shfl_xor_sync(0xffffffffu, give, 16));
        }
        uint32_t top = max(up8 ? mx[1] : mx[0], __shfl_xor_sync(0xffffffffu, up8 ? mx[0] : mx[1], 8));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 4));
        aux.red[ew][(up16 ? 8 : 0) + lc + (up8 ? 1 : 0)] = top;
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
            split2(acc[0][rb >> 1][2 * i + (rb & 1)], h0, h1);
            const uint32_t code = fp8_pack2(h0 * inv.x, h1 * inv.y, MOE_E4M3);
            o[8 * rb] = static_cast<uint8_t>(code);
            o[8 * rb + PITCH8] = static_cast<uint8_t>(code >> 8);
          }
        }
        named_barrier(2 + half, 128);
        // whole rows of 128 codes: eight lanes a row
        const int ch = et & 7;
        if (wt * WM + ch * 16 < p.N) {
          const int c = (et & 127) >> 3;
          const int col = half * HALF + c;
          if (col < it.n)
            *reinterpret_cast<uint4*>(p.out_q + static_cast<long long>(it.row0 + col) * p.N + wt * WM + ch * 16) =
                *reinterpret_cast<const uint4*>(stage + c * PITCH8 + ch * 16);
        }
      } else if (wt * WM + q * 32 < p.N) {  // N is a multiple of 32: the warp's rows are all inside or all outside
        if (p.out_bf16) {
          // the 16 columns through the warp's staging rows: [column][32 rows] bf16
          uint8_t* stage = out_stage + ew * 16 * PITCH16;
          const uint32_t st_addr = smem_addr(stage) + (lane & 7) * PITCH16 + (lane >> 3) * 16;
          const int ch = lane & 3;
          if (half * HALF < it.n) {  // warp-uniform
#pragma unroll
            for (int i = 0; i < X; ++i) {
              uint32_t pk[4];
              const int col = half * HALF + 8 * i + lc;
              const float s0 = aux.rscale[parity][col], s1 = aux.rscale[parity][col + 1];
#pragma unroll
              for (int rb = 0; rb < 4; ++rb) {
                float y0, y1;
                split2(acc[0][rb >> 1][2 * i + (rb & 1)], y0, y1);
                const __nv_bfloat162 t = __floats2bfloat162_rn(y0 * s0, y1 * s1);
                pk[rb] = *reinterpret_cast<const uint32_t*>(&t);
              }
              stmatrix_x4_trans(st_addr + i * 8 * PITCH16, pk[0], pk[1], pk[2], pk[3]);
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < X; ++i) {
              const int c = 8 * i + lr;
              const int d = aux.dest[parity][half * HALF + c];
              const uint4 v = *reinterpret_cast<const uint4*>(stage + c * PITCH16 + ch * 16);
              if (d >= 0)
                *reinterpret_cast<uint4*>(p.out_bf16 + static_cast<long long>(d) * p.N + wt * WM + q * 32 + ch * 8) = v;
            }
            __syncwarp();
          }
        } else {
#pragma unroll
          for (int i = 0; i < X; ++i) {
            const int col = half * HALF + 8 * i + lc;
            const int d0 = aux.dest[parity][col], d1 = aux.dest[parity][col + 1];
            const float s0 = aux.rscale[parity][col], s1 = aux.rscale[parity][col + 1];
            float* o = p.out_f32 + wt * WM + q * 32 + lr;
#pragma unroll
            for (int rb = 0; rb < 4; ++rb) {
              float y0, y1;
              split2(acc[0][rb >> 1][2 * i + (rb & 1)], y0, y1);
              if (d0 >= 0) o[static_cast<long long>(d0) * p.N + 8 * rb] = y0 * s0;
              if (d1 >= 0) o[static_cast<long long>(d1) * p.N + 8 * rb] = y1 * s1;
            }
          }
        }
      }
      if (split) {
        __syncwarp();
        cluster_wait();
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
  if (p.early) pdl_wait();  // complete only after the launch before
}

// ------------------------------------------------------------------ host side
// Clusters of `size` CTAs of the kernel that fit on the device at once, asked for once per device.
template <bool DUAL>
int resident_clusters(const Ctx& c, int size) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> cached[kMaxDevices][9];  // 1 + the number
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  if (const int v = cached[dev][size].load()) return v - 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(size * (c.num_sms / size));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = kSmem<DUAL>;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, fp8_gemm_kernel<DUAL>, &cfg) != cudaSuccess) n = 0;
  cudaGetLastError();
  cached[dev][size].store(n + 1);
  return n;
}

// How many CTAs share an item's k-blocks: as many (up to 8, of two k-blocks at least each) as leave every item's
// cluster resident at once.  Clusters do not fill the GPU (148 SMs hold 74 of two CTAs, but 45 of three, 15 of eight),
// and a second wave of them costs more than a wider split gains.
//
// A split itself costs about 2 us (the cluster's launch, its barriers and sums), so it is taken only where it saves the
// CTAs that many k-blocks.  Measured, us without / with a split, rows 1 to 64: one product, 16 to 8 k-blocks 9.1 / 10.8
// (7168 x 2048), 16 to 4 8.4 / 7.5 (2048 x 2048), 28 to 14 12.2 / 12.3, 40 to 20 15.5 / 14.2 (7168 x 5120), 4 to 2 4.8 / 6.6;
// the dual one of a token's experts, 8 to 4 14.8 / 16.8, 8 to 2 14.8 / 12.9, 16 to 8 18.9 / 16.9.
template <bool DUAL>
void set_split(const Ctx& c, Params& p, long long items) {
  constexpr int kSaved = DUAL ? 6 : 12;
  const int nkb = (p.K + KB - 1) / KB;
  for (int want = static_cast<int>(std::min<long long>({8LL, c.num_sms / std::max(1LL, items), nkb / 2})); want > 1; --want) {
    const int kb_per = (nkb + want - 1) / want;
    if (nkb - kb_per < kSaved) return;
    if (resident_clusters<DUAL>(c, want) >= items) {
      p.kb_per = kb_per;
      p.split = (nkb + kb_per - 1) / kb_per;
      return;
    }
  }
}

// Items of a launch, no fewer than there can be: c rows of a group are at most (c + NT - 1) / NT tiles.
long long items_of(int rows, int N, int G) {
  return (rows + static_cast<long long>(std::min(G, rows)) * (NT - 1)) / NT * ((N + WM - 1) / WM);
}

template <bool DUAL>
cudaError_t launch_typed(const Ctx& c, const Fp8GemmArgs& a) {
  CUtensorMap mA, m0, m1;
  if (!make_maps(a, a.gather ? 1 : NT, &mA, &m0, &m1)) return cudaErrorInvalidValue;
  Params p = make_params(c, a, a.b_fmt, a.a_fmt, WM);
  const long long items = items_of(a.rows, a.N, a.G);
  p.early = a.early;
  auto kern = fp8_gemm_kernel<DUAL>;
  constexpr size_t smem = kSmem<DUAL>;
  static_assert(smem <= SMEM_MAX, "shared memory");
  const cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void*>(kern), static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  set_split<DUAL>(c, p, items);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(c.num_sms / p.split, items) * p.split));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = c.stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = c.pdl ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.split > 1 ? 2 : 1;
  KernelScope ks(c, a.name);
  const cudaError_t le = cudaLaunchKernelEx(&cfg, kern, mA, m0, m1, p);
  return le != cudaSuccess ? le : cudaGetLastError();
}

// Mean rows of a group, of the groups that can hold any.
double mean_rows(int rows, int G) { return static_cast<double>(rows) / std::max(1, std::min(G, rows)); }
// Up to how many of them this form is the faster one.  Measured on whole passes of the experts (64 experts of 2816 x 704,
// 64 of 1024 x 2048, 16 of 2048 x 1024, 128 of 2048 x 768; us here / in fp8_gemm_rows.cu): the dual product with 14 rows a
// group 89 / 94, 89 / 90, 32 / 37, 124 / 124 (with 20 rows the other one, by 1 to 5 us); the single one with 6 rows
// 82 / 85, 79 / 81, 34 / 33, 108 / 110, with 10 rows 88 / 88, 82 / 84, 35 / 33, 126 / 123.  Whatever the rows, it is also
// faster while its items do not fill the GPU, since they are smaller and share their k-blocks (one product, 16 x 2048 x
// 7168: 10.4 / 25.8, 128 x 4096 x 7168, 128 items: 21.3 / 31.0, 512 x 512 x 2048: 10.2 / 12.2; but 512 x 2048 x 7168, 256
// items: 37.0 / 31.0, 96 x 7168 x 2048, 168 items: 15.3 / 12.5).  The rule knows the mean of a routing alone, which is what
// the host has: an uneven one's large groups go with the others (a few hundred rows of a mean of 16, in tiles of 32).
constexpr double kSmallRowsDual = 16.0, kSmallRows = 8.0;

}  // namespace

bool fp8_gemm_many(int num_sms, int rows, int N, int G, bool dual) {
  return mean_rows(rows, G) > (dual ? kSmallRowsDual : kSmallRows) && items_of(rows, N, G) > std::min(num_sms, kFp8MaxSms);
}

bool fp8_gemm_gathers(int rows, int G) { return mean_rows(rows, G) <= kSmallRowsDual; }

cudaError_t launch_fp8_gemm(const Ctx& c, const Fp8GemmArgs& a) {
  if (a.rows <= 0 || a.G <= 0) return cudaSuccess;
  if (a.G > MAX_G || a.N % 32 || a.K % 32 || a.N <= 0 || a.K <= 0) return cudaErrorInvalidValue;
  if (a.gather && (!a.dual || mean_rows(a.rows, a.G) > kSmallRowsDual)) return cudaErrorInvalidValue;
  const bool many = fp8_gemm_many(c.num_sms, a.rows, a.N, a.G, a.dual);
  if (a.out_f16 && (!many || a.dual || a.a_fmt != MOE_E4M3 || a.b_fmt != MOE_E4M3 || a.row_scale)) return cudaErrorInvalidValue;
  if (many) return launch_fp8_rows_gemm(c, a);
  return a.dual ? launch_typed<true>(c, a) : launch_typed<false>(c, a);
}

}  // namespace moe
