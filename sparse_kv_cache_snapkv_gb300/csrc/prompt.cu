// The attention weight that every key of a prompt gets from the prompt's queries (sm_103a):
// column sums of a causal softmax, without the attention's outputs.
//
//   s_rj = scale q_r . k_j over the keys j <= lim_r that query row r sees,
//   lse_r = log sum_j exp(s_rj),   weights_j += sum_r exp(s_rj - lse_r),
// r running over the queries of all heads of the KV group. The sums lse_r are needed before the
// first weight, and the scores are far too many to keep (2 GB for one head of a 32K prompt), so
// there are two passes over Q K^T, both on tcgen05:
//   pass 1  256 query rows stay in shared memory, the keys stream by: S = Q K^T, and every lane
//           of the accumulator is one query row with a running maximum and sum of its own;
//   pass 2  256 keys stay, the query rows stream by: S^T = K Q^T, and every lane is one key that
//           adds up 2^(s - lse_r). No value crosses lanes in either pass, and each key has one
//           owner, so nothing depends on the order in which CTAs run.
// Bound: one exponential and one multiply-add per (row, key) and pass beside 256 flops on the
// tensor cores. Stationary tiles of 256 rows halve the streamed bytes per product against 128.
//
// A CTA is persistent over work items (a stationary tile, or one split of its stream), largest
// first. One thread loads (TMA), one issues the products, sixteen warps read the accumulators: two
// of 128 rows, each double-buffered in TMEM (512 columns), so that the exponentials of one tile run
// under the products of the next.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/rkv_testing.h"
#include "common.cuh"
#include "rkv_internal.h"
#include "tensor_core.cuh"

namespace rkv {

constexpr int kPrThreads = 576;   // warp 0: TMA, warp 1: MMA, warps 2..17: accumulators
constexpr int kPrEpi = 512;       // two threads per stationary row, half of a tile's columns each
constexpr int kPrStat = 256;      // stationary rows of an item
constexpr int kPrTile = 128;      // streamed rows of a step
constexpr int kPrStages = 3;
constexpr int kPrStatBytes = kPrStat * kHeadDim * 2;   // 64 KB
constexpr int kPrTileBytes = kPrTile * kHeadDim * 2;   // 32 KB
constexpr uint32_t kPrCols = 512;
// Slots of the streamed rows' log-sum-exps (pass 2). A tile is requested when the product three
// tiles before it is done, which was issued when the accumulator five tiles before it was free: the
// slot of that tile is free too, without a barrier of its own.
constexpr int kPrNlSlots = kPrStages + 2;

// Query rows of a (unit, KV head). With at least 256 queries a tile holds rows of one head (the
// causal limits of a tile are then close together, and most of what it need not see is skipped);
// with fewer, a tile runs on through the heads so that short chunks still fill it.
struct RowMap {
  int gqa, max_q, per_head;  // per_head: tiles of one head (0: the rows run through the heads)
};

__host__ __device__ inline RowMap row_map(int gqa, int max_q, int tile) {
  return RowMap{gqa, max_q, max_q >= kPrStat ? (max_q + tile - 1) / tile : 0};
}
__host__ __device__ inline int row_tiles(const RowMap& m, int tile) {
  return m.per_head ? m.gqa * m.per_head : (m.gqa * m.max_q + tile - 1) / tile;
}
// first row of a tile among the group's gqa * max_q rows as they lie in memory
__device__ __forceinline__ int tile_row0(const RowMap& m, int t, int tile) {
  return m.per_head ? (t / m.per_head) * m.max_q + (t % m.per_head) * tile : t * tile;
}
// query index of row k of a tile; -1: not a row of this tile
__device__ __forceinline__ int tile_query(const RowMap& m, int t, int tile, int k) {
  if (m.per_head) {
    const int i = (t % m.per_head) * tile + k;
    return i < m.max_q ? i : -1;
  }
  const int r = t * tile + k;
  return r < m.gqa * m.max_q ? r % m.max_q : -1;
}
// smallest and largest query index of a tile's rows (rows past q_len count as rows)
__device__ __forceinline__ void tile_span(const RowMap& m, int t, int tile, int* lo, int* hi) {
  if (m.per_head) {
    *lo = (t % m.per_head) * tile;
    *hi = min(*lo + tile, m.max_q) - 1;
  } else {
    *lo = 0;
    *hi = m.max_q - 1;
  }
}

struct PromptParams {
  int n_kv, gqa, max_q, max_len, units;  // units = n * n_kv
  int tiles1, nsplit1;   // pass 1: stationary query tiles per unit, splits of the key stream
  int tiles2, nsplit2;   // pass 2: stationary key tiles per unit, splits of the query stream
  float scale_log2;
  const int32_t* len;
  const int32_t* q_len;
  float* nl;             // [units][tiles1 * 256]: every row's negated log-sum-exp (log2 domain)
  float2* ml;            // [units][nsplit1][tiles1 * 256]: (max, sum) of a split when nsplit1 > 1
  float* part;           // [nsplit2][units][max_len] when nsplit2 > 1
  float* weights;        // [units][max_len]
  uint32_t* status;
  WaitLimit wait_limit;    // bound of every mbarrier wait
  int test_skip;           // testing only: what CTA 0 never requests (RKV_TESTING_PROMPT_*; 0: nothing)
};

struct PrSmem {
  static constexpr size_t stat_off = 0;
  static constexpr size_t tile_off = 2 * (size_t)kPrStatBytes;
  static constexpr size_t bar_off = tile_off + (size_t)kPrStages * kPrTileBytes;
  static constexpr size_t nl_off = bar_off + 256;  // [kPrNlSlots][128]
  static constexpr size_t total = nl_off + (size_t)kPrNlSlots * kPrTile * 4;
};
static_assert(PrSmem::total <= 232448, "shared memory of a CTA");

// -(max + log2 sum) of a row; -1e30 (its weights are 0) for one that sees nothing or is no query
__device__ __forceinline__ float negated_lse(float m, float l) {
  return l > 0.f ? -(m + log2f(l)) : (l == 0.f ? -1e30f : l);
}

struct PromptItem {
  int ukv, u, L, T;   // L = 0: nothing to do
  int tile;           // stationary tile
  int first, count;   // streamed steps [first, first + count)
  int q0, span;       // pass 2, one head per tile: first streamed tile of a head, and how many
};

template <int PASS>
__device__ __forceinline__ PromptItem prompt_item(const PromptParams& p, int i) {
  PromptItem it;
  const int nsplit = PASS == 1 ? p.nsplit1 : p.nsplit2;
  const RowMap m1 = row_map(p.gqa, p.max_q, kPrStat), m2 = row_map(p.gqa, p.max_q, kPrTile);
  const int per = p.units * nsplit;
  int o = i / per;                  // place in the order of decreasing work
  const int rest = i - o * per;
  it.ukv = rest / nsplit;
  const int split = rest - it.ukv * nsplit;
  if (PASS == 1) {
    // the last queries see most keys: tiles from the end of each head, heads side by side
    if (m1.per_head) {
      const int h = o % p.gqa;
      it.tile = h * m1.per_head + (m1.per_head - 1 - o / p.gqa);
    } else {
      it.tile = o;
    }
  } else {
    it.tile = o;  // the first keys are seen by most queries
  }
  it.u = it.ukv / p.n_kv;
  it.L = p.len[it.u];
  it.T = p.q_len[it.u];
  it.first = it.count = it.q0 = it.span = 0;
  if (it.L < 0 || it.L > p.max_len || it.T <= 0 || it.T > p.max_q || it.T > it.L) {
    it.L = 0;
    return it;
  }
  int steps;
  if (PASS == 1) {
    int lo, hi;
    tile_span(m1, it.tile, kPrStat, &lo, &hi);
    if (lo >= it.T) return it;
    const int keys = it.L - it.T + min(hi, it.T - 1) + 1;
    steps = (keys + kPrTile - 1) / kPrTile;
  } else {
    const int k0 = it.tile * kPrStat;
    if (k0 >= it.L) return it;
    if (m2.per_head) {
      it.q0 = max(0, k0 - (it.L - it.T)) / kPrTile;
      it.span = (it.T + kPrTile - 1) / kPrTile - it.q0;
      steps = it.span * p.gqa;
    } else {
      steps = row_tiles(m2, kPrTile);
    }
  }
  const int each = (steps + nsplit - 1) / nsplit;
  it.first = split * each;
  it.count = max(0, min(each, steps - it.first));
  return it;
}

// streamed query tile of a pass-2 step
__device__ __forceinline__ int step_tile(const PromptParams& p, const PromptItem& it, int step) {
  if (it.span == 0) return step;
  const RowMap m2 = row_map(p.gqa, p.max_q, kPrTile);
  const int h = step / it.span;
  return h * m2.per_head + it.q0 + (step - h * it.span);
}

// HEADS: a tile's query rows are of one head (row_map's per_head is not 0).
template <int PASS, bool HEADS>
__global__ void __launch_bounds__(kPrThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap qmap, PromptParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* stat = smem + PrSmem::stat_off;
  uint8_t* tiles = smem + PrSmem::tile_off;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + PrSmem::bar_off);
  uint64_t* empty = full + kPrStages;
  uint64_t* tfull = empty + kPrStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* sfull = tempty + 2;
  uint64_t* sempty = sfull + 2;
  uint64_t* nfull = sempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(nfull + kPrNlSlots);
  float* nl_s = reinterpret_cast<float*>(smem + PrSmem::nl_off);

  if (smem_addr(smem) & 1023u) {  // the swizzled tiles need it; a CTA's dynamic memory has it
    if (threadIdx.x == 0) set_status(p.status, RKV_DEV_SELECT_FAILED);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const RowMap m1 = row_map(p.gqa, p.max_q, kPrStat), m2 = row_map(p.gqa, p.max_q, kPrTile);
  const int items = p.units * (PASS == 1 ? p.tiles1 * p.nsplit1 : p.tiles2 * p.nsplit2);

  // Items come in waves of one per CTA, every second wave from the other end: the CTA that had the
  // largest item of a wave gets the smallest of the next.
  auto wave_item = [&](int w) {
    return w * (int)gridDim.x + ((w & 1) ? (int)(gridDim.x - 1 - blockIdx.x) : (int)blockIdx.x);
  };

  if (tid == 0) {
    for (int i = 0; i < kPrStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], kPrEpi / 32);
      mbar_init(&sfull[i], 1);
      mbar_init(&sempty[i], 1);
    }
    for (int i = 0; i < kPrNlSlots; ++i) mbar_init(&nfull[i], 1);
    fence_barrier_init();
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_addr(tmem_slot)), "r"(kPrCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  bool aborted = false;
  const WaitLimit limit = p.wait_limit;
  const int skip = blockIdx.x == 0 ? p.test_skip : 0;

  if (warp == 0) {
    // ------------------------------------------------------------------ loads
    if (lane == 0) {
      int step = 0, ic = 0, sent = 0;  // sent: stationary tiles requested
      for (int w = 0; w * gridDim.x < items && !aborted; ++w) {
        const int i = wave_item(w);
        if (i >= items) continue;
        const PromptItem it = prompt_item<PASS>(p, i);
        if (it.count == 0) continue;
        const int sb = ic & 1;
        if (ic >= 2 && !mbar_wait(&sempty[sb], (uint32_t)(((ic >> 1) - 1) & 1), limit)) {
          aborted = true;
          break;
        }
        const int qbase = it.ukv * p.gqa * p.max_q, kbase = it.ukv * p.max_len;
        const int srow = PASS == 1 ? qbase + tile_row0(m1, it.tile, kPrStat)
                                   : kbase + it.tile * kPrStat;
        const CUtensorMap* smap = PASS == 1 ? &qmap : &kmap;
        uint8_t* sdst = stat + (size_t)sb * kPrStatBytes;
        mbar_arrive_expect_tx(&sfull[sb], (uint32_t)kPrStatBytes);
        for (int rb = 0; rb < 2; ++rb)
          for (int h = 0; h < 2; ++h)
            tma_load_2d(sdst + (size_t)(rb * 2 + h) * 16384, smap, 64 * h, srow + rb * 128,
                        &sfull[sb]);
        sent = ic + 1;
        for (int t = 0; t < it.count; ++t, ++step) {
          const int s = step % kPrStages;
          if (step >= kPrStages &&
              !mbar_wait(&empty[s], (uint32_t)(((step / kPrStages) - 1) & 1), limit)) {
            aborted = true;
            break;
          }
          int y = kbase + (it.first + t) * kPrTile;
          if (PASS == 2) {
            const int x = step_tile(p, it, it.first + t);
            y = qbase + tile_row0(m2, x, kPrTile);
            // the same rows' log-sum-exps, as pass 1's tiles have them
            const int row = m2.per_head ? (x / m2.per_head) * (m1.per_head * kPrStat) +
                                              (x % m2.per_head) * kPrTile
                                        : x * kPrTile;
            const int ns = step % kPrNlSlots;
            if (skip != RKV_TESTING_PROMPT_SUMS || step > 0) {
              mbar_arrive_expect_tx(&nfull[ns], kPrTile * 4);
              bulk_load(nl_s + ns * kPrTile, p.nl + (size_t)it.ukv * p.tiles1 * kPrStat + row,
                        kPrTile * 4, &nfull[ns]);
            }
          }
          if (skip == (PASS == 1 ? RKV_TESTING_PROMPT_KEYS : RKV_TESTING_PROMPT_QUERIES) && step == 0)
            continue;
          uint8_t* dst = tiles + (size_t)s * kPrTileBytes;
          mbar_arrive_expect_tx(&full[s], (uint32_t)kPrTileBytes);
          tma_load_2d(dst, PASS == 1 ? &kmap : &qmap, 0, y, &full[s]);
          tma_load_2d(dst + 16384, PASS == 1 ? &kmap : &qmap, 64, y, &full[s]);
        }
        ++ic;
      }
      if (aborted) set_status(p.status, RKV_DEV_WAIT_TIMEOUT);
      // every issued load lands before the CTA ends, whoever gave up (else they have, and this is no wait)
      for (int j = max(0, step - kPrStages); j < step; ++j)
        mbar_wait(&full[j % kPrStages], (uint32_t)((j / kPrStages) & 1), drain_limit(limit));
      for (int j = max(0, step - kPrNlSlots); PASS == 2 && j < step; ++j)
        mbar_wait(&nfull[j % kPrNlSlots], (uint32_t)((j / kPrNlSlots) & 1), drain_limit(limit));
      for (int j = max(0, ic - 2); j < sent; ++j)
        mbar_wait(&sfull[j & 1], (uint32_t)((j >> 1) & 1), drain_limit(limit));
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ products
    if (lane == 0) {
      int step = 0, ic = 0;
      for (int w = 0; w * gridDim.x < items && !aborted; ++w) {
        const int i = wave_item(w);
        if (i >= items) continue;
        const PromptItem it = prompt_item<PASS>(p, i);
        if (it.count == 0) continue;
        const int sb = ic & 1;
        if (!mbar_wait(&sfull[sb], (uint32_t)((ic >> 1) & 1), limit)) {
          aborted = true;
          break;
        }
        const uint32_t sbase = smem_addr(stat + (size_t)sb * kPrStatBytes);
        for (int t = 0; t < it.count; ++t, ++step) {
          const int s = step % kPrStages, b = step & 1;
          if (!mbar_wait(&full[s], (uint32_t)((step / kPrStages) & 1), limit) ||
              (step >= 2 && !mbar_wait(&tempty[b], (uint32_t)(((step >> 1) - 1) & 1), limit))) {
            aborted = true;
            break;
          }
          tc_fence_after();
          const uint32_t tbase = smem_addr(tiles + (size_t)s * kPrTileBytes);
          constexpr uint32_t id = idesc_bf16(128, kPrTile);
#pragma unroll
          for (int rb = 0; rb < 2; ++rb) {
            const uint32_t d = tmem + (uint32_t)((b * 2 + rb) * kPrTile);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t off = (uint32_t)((kk >> 2) * 16384 + (kk & 3) * 32);
              umma_bf16(d, desc_sw128(sbase + rb * 32768 + off), desc_sw128(tbase + off), id,
                        kk > 0);
            }
          }
          umma_commit(&empty[s]);
          umma_commit(&tfull[b]);
        }
        if (aborted) break;
        umma_commit(&sempty[sb]);
        ++ic;
      }
      if (aborted) {
        set_status(p.status, RKV_DEV_WAIT_TIMEOUT);
        for (int j = max(0, step - 2); j < step; ++j)  // let issued products end
          mbar_wait(&tfull[j & 1], (uint32_t)((j >> 1) & 1), drain_limit(limit));
      }
    }
  } else {
    // ------------------------------------------------------------------ accumulators
    const int e = warp - 2;
    const int quarter = warp & 3;       // TMEM lanes this warp may read
    const int rb = (e >> 2) & 1, hf = e >> 3;
    const int srow = rb * 128 + quarter * 32 + lane;  // stationary row of this thread
    const int c0 = hf * 64;             // its columns of a tile: c0 .. c0 + 63
    const int etid = tid - 64;
    const uint32_t lane_addr = ((uint32_t)(quarter * 32) << 16) + (uint32_t)(rb * kPrTile + c0);
    // what the second half hands to the first, one item after the other
    float2* xch = reinterpret_cast<float2*>(smem + PrSmem::nl_off);  // (pass 1: no log-sum-exps)
    const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2);
    int step = 0, nslot = 0;
    uint32_t nphase = 0;
    for (int w = 0; w * gridDim.x < items; ++w) {
      const int i = wave_item(w);
      if (i >= items) continue;
      const PromptItem it = prompt_item<PASS>(p, i);
      if (PASS == 1 && it.L == 0 && it.tile == 0 && it.ukv == it.u * p.n_kv && etid == 0) {
        const int L = p.len[it.u], T = p.q_len[it.u];
        if (L < 0 || L > p.max_len)
          set_status(p.status, RKV_DEV_LEN_OVER_CAP);
        else if (T != 0)
          set_status(p.status, RKV_DEV_BAD_WINDOW);
      }
      if (PASS == 1) {
        const int qi = tile_query(m1, it.tile, kPrStat, srow);
        const int lim = (qi >= 0 && qi < it.T) ? it.L - it.T + qi : -1;  // last visible key
        float m = -1e30f, l = 0.f;
        // one half of the columns after the other, the second's load under the first's work
        uint32_t r[2][32];
        auto chunk = [&](uint32_t (&x)[32], int key0) {
          if (__any_sync(0xffffffffu, key0 + 31 > lim)) {  // (no divergence at the loads)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (key0 + j > lim) x[j] = 0xff800000u;
          }
          // Terms relative to a reference m that need not be the maximum: it is set by the first
          // keys, and again by a chunk whose terms come out huge. So most chunks look for no
          // maximum; a sum stays below 2^60 of its reference, far inside fp32.
          float sum;
          auto terms = [&]() {
            const uint64_t off = pack2(-m, -m);
            uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const float2 y = unpack2(
                  fma2(pack2(__uint_as_float(x[j]), __uint_as_float(x[j + 1])), scale2, off));
              acc[(j >> 1) & 1] = add2(acc[(j >> 1) & 1], pack2(fast_exp2(y.x), fast_exp2(y.y)));
            }
            const float2 s = unpack2(add2(acc[0], acc[1]));
            sum = s.x + s.y;
          };
          terms();
          if (__any_sync(0xffffffffu, !(sum < 1.152921504606847e18f))) {  // 2^60; NaN too
            float mt[2] = {__uint_as_float(x[0]), __uint_as_float(x[1])};
#pragma unroll
            for (int j = 2; j < 32; ++j) mt[j & 1] = fmaxf(mt[j & 1], __uint_as_float(x[j]));
            const float mn = fmaxf(m, fmaxf(mt[0], mt[1]) * p.scale_log2);
            l *= fast_exp2(m - mn);
            m = mn;
            terms();
          }
          l += sum;
        };
        // waits for a tile's product (the whole warp goes on or none of it: `aborted` is the same in all
        // lanes) and starts its first half (started under the half before it, instead of after that, the
        // loads made the 8K prompt take 513 us instead of 447)
        auto start_tile = [&](int st) {
          if (!mbar_wait_warp(&tfull[st & 1], (uint32_t)((st >> 1) & 1), limit)) {
            aborted = true;
            return false;
          }
          tc_fence_after();
          tmem_ld32_start(tmem + lane_addr + (uint32_t)((st & 1) * 2 * kPrTile), r[0]);
          return true;
        };
        for (int t = 0; t < it.count; ++t, ++step) {
          if (aborted || !start_tile(step)) continue;
          const int b = step & 1, k0 = (it.first + t) * kPrTile + c0;
          tmem_ld_wait(r[0]);
          tmem_ld32_start(tmem + lane_addr + (uint32_t)(b * 2 * kPrTile) + 32, r[1]);
          chunk(r[0], k0);
          tmem_ld_wait(r[1]);
          tc_fence_before();  // the accumulator is free once both halves are in registers
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[b]);
          chunk(r[1], k0 + 32);
        }
        if (hf == 1) xch[srow] = make_float2(m, l);
        named_bar_sync(1, kPrEpi);
        if (hf == 0) {
          const float2 o = xch[srow];
          const float mn = fmaxf(m, o.x);
          l = l * fast_exp2(m - mn) + o.y * fast_exp2(o.x - mn);
          m = mn;
          // every row of every item is written, so that pass 2 never meets an old workspace
          const size_t row = (size_t)it.tile * kPrStat + srow, rows = (size_t)p.tiles1 * kPrStat;
          if (p.nsplit1 == 1) {
            p.nl[it.ukv * rows + row] = negated_lse(m, l);
          } else {
            const int split = (i % (p.units * p.nsplit1)) % p.nsplit1;
            p.ml[((size_t)it.ukv * p.nsplit1 + split) * rows + row] = make_float2(m, l);
          }
        }
        named_bar_sync(1, kPrEpi);  // xch is rewritten by the next item
      } else {
        const int key = it.tile * kPrStat + srow;
        // A key's sum over many tiles is a compensated one (sum - lost): an early key of a long prompt
        // has tens of thousands of weights added, each of which a plain sum would round at its size.
        const uint64_t minus = pack2(-1.f, -1.f);
        uint64_t acc[2], sum = 0ull, lost = 0ull;
        uint32_t r[2][32];
        auto chunk = [&](uint32_t (&x)[32], int tile, bool mask, int base, const float* nl) {
          if (mask) {
            // row j of this half is query q + j of its head (wrapping at max_q where the rows run
            // through the heads), and sees this key from query `from` on
            const int from = key - (it.L - it.T);
            uint32_t sees;  // a bit for each row
            if (HEADS) {
              const int q = tile * kPrTile + base, b0 = from - q, b1 = it.T - q;
              sees = b0 >= 32 ? 0u : (0xffffffffu << max(b0, 0));
              sees &= b1 >= 32 ? 0xffffffffu : (b1 <= 0 ? 0u : (1u << b1) - 1u);
            } else {
              const int row = tile * kPrTile + base, rows = p.gqa * p.max_q;
              int q = row % p.max_q;
              sees = 0u;
              for (int j = 0; j < 32; ++j) {
                if (q >= from && q < it.T && row + j < rows) sees |= 1u << j;
                q = q + 1 == p.max_q ? 0 : q + 1;
              }
            }
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!((sees >> j) & 1u)) x[j] = 0xff800000u;
          }
          const ulonglong2* n2 = reinterpret_cast<const ulonglong2*>(nl + base);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const ulonglong2 v = n2[j];  // negated log-sum-exps of four rows
            const float2 y0 = unpack2(fma2(pack2(__uint_as_float(x[4 * j]),
                                                 __uint_as_float(x[4 * j + 1])), scale2, v.x));
            const float2 y1 = unpack2(fma2(pack2(__uint_as_float(x[4 * j + 2]),
                                                 __uint_as_float(x[4 * j + 3])), scale2, v.y));
            acc[0] = add2(acc[0], pack2(fast_exp2(y0.x), fast_exp2(y0.y)));
            acc[1] = add2(acc[1], pack2(fast_exp2(y1.x), fast_exp2(y1.y)));
          }
        };
        // the streamed tile: its number within its head (or among all rows' tiles), counted along
        int ti = HEADS ? it.q0 + it.first % max(it.span, 1) : it.first;
        for (int t = 0; t < it.count; ++t, ++step, ++ti) {
          if (HEADS && ti == it.q0 + it.span) ti = it.q0;
          if (aborted) continue;
          // the tile's product and its log-sum-exps, both before the first load is started: that would
          // have to be waited for. One vote where both are there (8K prompt: 1.0 % over lanes that
          // decide for themselves, with a vote for each 1.5 %).
          const uint32_t tphase = (uint32_t)((step >> 1) & 1);
          if (!__all_sync(0xffffffffu, mbar_try_wait(smem_addr(&tfull[step & 1]), tphase) &&
                                           mbar_try_wait(smem_addr(&nfull[nslot]), nphase)) &&
              !(mbar_wait_warp(&tfull[step & 1], tphase, limit) && mbar_wait_warp(&nfull[nslot], nphase, limit))) {
            aborted = true;
            continue;
          }
          tc_fence_after();
          tmem_ld32_start(tmem + lane_addr + (uint32_t)((step & 1) * 2 * kPrTile), r[0]);
          const float* nl = nl_s + nslot * kPrTile;
          if (++nslot == kPrNlSlots) {
            nslot = 0;
            nphase ^= 1u;
          }
          const int b = step & 1;
          acc[0] = acc[1] = 0ull;
          // a tile with rows that are no queries, or that do not see all of the stationary keys
          const int x = ti;
          const int last = HEADS ? ti * kPrTile + kPrTile : p.max_q;  // queries below `last`
          const bool mask = last > it.T || (!HEADS && ti * kPrTile + kPrTile > p.gqa * p.max_q) ||
                            it.L - it.T + (HEADS ? ti * kPrTile : 0) < (it.tile + 1) * kPrStat - 1;
          tmem_ld_wait(r[0]);
          tmem_ld32_start(tmem + lane_addr + (uint32_t)(b * 2 * kPrTile) + 32, r[1]);
          chunk(r[0], x, mask, c0, nl);
          tmem_ld_wait(r[1]);
          chunk(r[1], x, mask, c0 + 32, nl);
          const uint64_t y = fma2(lost, minus, add2(acc[0], acc[1])), now = add2(sum, y);
          lost = fma2(y, minus, fma2(sum, minus, now));
          sum = now;
          // (the log-sum-exps are read before this too: their slot is free with the accumulator)
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[b]);
        }
        const float2 s = unpack2(sum);
        // the two threads of a key add to it one after the other (shared memory is full)
        const bool one = p.nsplit2 == 1;
        const int split = (i % (p.units * p.nsplit2)) % p.nsplit2;
        float* dst = one ? p.weights + (size_t)it.ukv * p.max_len + key
                         : p.part + ((size_t)split * p.units + it.ukv) * p.max_len + key;
        const bool mine = key < it.L && (!one || (it.count > 0 && !aborted));
        if (hf == 0 && mine) *dst = (one ? *dst : 0.f) + (s.x + s.y);
        named_bar_sync(1, kPrEpi);
        if (hf == 1 && mine) *dst += s.x + s.y;
      }
    }
    if (aborted) set_status(p.status, RKV_DEV_WAIT_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                 "r"(kPrCols) : "memory");
  }
}

// Joins the splits of pass 1 (grid: units x blocks of 256 rows).
__global__ void __launch_bounds__(256) prompt_lse_kernel(PromptParams p) {
  pdl_wait();
  pdl_trigger();
  const size_t rows = (size_t)p.tiles1 * kPrStat, row = (size_t)blockIdx.y * 256 + threadIdx.x;
  const float2* src = p.ml + (size_t)blockIdx.x * p.nsplit1 * rows + row;
  float m = -1e30f, l = 0.f;
  for (int s = 0; s < p.nsplit1; ++s) {
    const float2 y = src[s * rows];
    const float mn = fmaxf(m, y.x);
    l = l * fast_exp2(m - mn) + y.y * fast_exp2(y.x - mn);
    m = mn;
  }
  p.nl[blockIdx.x * rows + row] = negated_lse(m, l);
}

// Sum of the splits, in their order.
__global__ void __launch_bounds__(256) prompt_sum_kernel(PromptParams p) {
  pdl_wait();
  const int ukv = blockIdx.x, u = ukv / p.n_kv;
  const int L = p.len[u], T = p.q_len[u];
  if (L < 0 || L > p.max_len || T <= 0 || T > p.max_q || T > L) return;
  for (int j = blockIdx.y * 256 + threadIdx.x; j < L; j += gridDim.y * 256) {
    float s = 0.f;
    for (int k = 0; k < p.nsplit2; ++k)
      s += p.part[((size_t)k * p.units + ukv) * p.max_len + j];
    p.weights[(size_t)ukv * p.max_len + j] += s;
  }
}

struct PromptPlan {
  int tiles1, nsplit1, tiles2, nsplit2;
};

// Splits only where the items alone would leave SMs without work (a split costs its own stationary
// load, and partial results that are read back). Pass 2 has few and uneven items (the first keys
// are seen by every query): with fewer than four per SM the largest would outlast the rest.
static PromptPlan prompt_plan(int n, int n_kv, int gqa, int max_q, int max_len) {
  PromptPlan p;
  const long long units = (long long)n * n_kv;
  const int sms = device_sm_count();
  p.tiles1 = row_tiles(row_map(gqa, max_q, kPrStat), kPrStat);
  p.tiles2 = (max_len + kPrStat - 1) / kPrStat;
  auto splits = [](long long items, long long target, int most) {
    const long long want = target / items;
    return (int)(want < 1 ? 1 : (want < most ? want : (most < 1 ? 1 : most)));
  };
  const int steps1 = (max_len + kPrTile - 1) / kPrTile;
  const int steps2 = row_tiles(row_map(gqa, max_q, kPrTile), kPrTile);
  p.nsplit1 = splits(units * p.tiles1, sms, (steps1 + 3) / 4);
  const int fill = splits(units * p.tiles2, sms, (steps2 + 3) / 4);         // an item for every SM
  const int even = splits(units * p.tiles2, 4LL * sms, steps2 / 32);        // of at least 32 steps
  p.nsplit2 = fill > even ? fill : even;
  return p;
}

static size_t nl_bytes(const PromptPlan& p, size_t units) {
  return align_up(units * p.tiles1 * kPrStat * 4, 256);
}
static size_t ml_bytes(const PromptPlan& p, size_t units) {
  return p.nsplit1 > 1 ? align_up(units * p.nsplit1 * p.tiles1 * kPrStat * 8, 256) : 0;
}

// Room for every call of no larger sizes, so that a workspace for the largest shape serves all: splits
// are made until there are `sms` items in pass 1 and 4 sms in pass 2, so their partial results are at
// most that many tiles' (and a split fewer than four steps of the stream is not made), whichever sizes
// bring that about.
size_t prompt_scratch_bytes(int n, int n_kv, int gqa, int max_q, int max_len) {
  const PromptPlan p = prompt_plan(n, n_kv, gqa, max_q, max_len);
  const size_t units = (size_t)n * n_kv, sms = device_sm_count();
  const size_t most1 = (size_t)((max_len + kPrTile - 1) / kPrTile + 3) / 4;
  const size_t most2 = (size_t)(row_tiles(row_map(gqa, max_q, kPrTile), kPrTile) + 3) / 4;
  const size_t items1 = units * p.tiles1 * most1, rows2 = units * most2 * max_len;
  const size_t ml = (items1 < sms ? items1 : sms) * kPrStat * 8;
  const size_t part = (rows2 < 4 * sms * kPrStat ? rows2 : 4 * sms * kPrStat) * 4;
  return nl_bytes(p, units) + align_up(ml, 256) + align_up(part, 256);
}

template <int PASS, bool HEADS>
static cudaError_t launch_prompt_pass(const CUtensorMap& km, const CUtensorMap& qm,
                                      const PromptParams& p, cudaStream_t s) {
  cudaError_t e = ensure_dyn_smem((const void*)prompt_kernel<PASS, HEADS>, PrSmem::total);
  if (e != cudaSuccess) return e;
  const long long items =
      (long long)p.units * (PASS == 1 ? p.tiles1 * p.nsplit1 : p.tiles2 * p.nsplit2);
  if (items > 0x3fffffffll) return cudaErrorInvalidConfiguration;
  const int sms = device_sm_count();
  return launch_pdl_kernel(prompt_kernel<PASS, HEADS>, dim3((unsigned)(items < sms ? items : sms)),
                           dim3(kPrThreads), PrSmem::total, s, km, qm, p);
}

cudaError_t launch_prompt_weights(const PromptArgs& a, cudaStream_t s) {
  CUtensorMap km, qm;
  if (!make_rows_map(&km, a.k, (uint64_t)a.n * a.n_kv * a.max_len) ||
      !make_rows_map(&qm, a.q, (uint64_t)a.n * a.n_kv * a.gqa * a.max_q))
    return cudaErrorInvalidValue;
  const PromptPlan pl = prompt_plan(a.n, a.n_kv, a.gqa, a.max_q, a.max_len);
  PromptParams p{};
  p.n_kv = a.n_kv;
  p.gqa = a.gqa;
  p.max_q = a.max_q;
  p.max_len = a.max_len;
  p.units = a.n * a.n_kv;
  p.tiles1 = pl.tiles1;
  p.nsplit1 = pl.nsplit1;
  p.tiles2 = pl.tiles2;
  p.nsplit2 = pl.nsplit2;
  p.scale_log2 = a.scale_log2;
  p.len = a.len;
  p.q_len = a.q_len;
  unsigned char* w = static_cast<unsigned char*>(a.scratch);
  p.nl = reinterpret_cast<float*>(w);
  w += nl_bytes(pl, p.units);
  p.ml = reinterpret_cast<float2*>(w);
  p.part = reinterpret_cast<float*>(w + ml_bytes(pl, p.units));
  p.weights = a.weights;
  p.status = a.status;
  p.wait_limit = a.wait_limit_ns ? WaitLimit{a.wait_limit_ns} : kWaitLimit;
  p.test_skip = a.test_skip;
  const bool heads = row_map(a.gqa, a.max_q, kPrTile).per_head != 0;
  cudaError_t e = heads ? launch_prompt_pass<1, true>(km, qm, p, s)
                        : launch_prompt_pass<1, false>(km, qm, p, s);
  if (e != cudaSuccess) return e;
  if (p.nsplit1 > 1) {
    e = launch_pdl_kernel(prompt_lse_kernel, dim3(p.units, p.tiles1), dim3(256), 0, s, p);
    if (e != cudaSuccess) return e;
  }
  e = heads ? launch_prompt_pass<2, true>(km, qm, p, s) : launch_prompt_pass<2, false>(km, qm, p, s);
  if (e != cudaSuccess || p.nsplit2 == 1) return e;
  int y = (a.max_len + 255) / 256;
  return launch_pdl_kernel(prompt_sum_kernel, dim3(p.units, y < 1024 ? y : 1024), dim3(256), 0, s,
                           p);
}

}  // namespace rkv
