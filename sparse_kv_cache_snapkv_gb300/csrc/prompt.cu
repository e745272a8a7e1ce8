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
// first. One thread loads (TMA), one issues the products, eight warps read the accumulators: two
// of 128 rows, each double-buffered in TMEM (512 columns), so that the exponentials of one tile run
// under the products of the next.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "common.cuh"
#include "rkv_internal.h"
#include "tensor_core.cuh"

namespace rkv {

constexpr int kPrThreads = 320;   // warp 0: TMA, warp 1: MMA, warps 2..9: accumulators
constexpr int kPrEpi = 256;
constexpr int kPrStat = 256;      // stationary rows of an item
constexpr int kPrTile = 128;      // streamed rows of a step
constexpr int kPrStages = 3;
constexpr int kPrStatBytes = kPrStat * kHeadDim * 2;   // 64 KB
constexpr int kPrTileBytes = kPrTile * kHeadDim * 2;   // 32 KB
constexpr uint32_t kPrCols = 512;

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
  float2* ml;            // [units][nsplit1][tiles1 * 256]: (max, sum) of every row
  float* part;           // [nsplit2][units][max_len] when nsplit2 > 1
  float* weights;        // [units][max_len]
  uint32_t* status;
};

struct PrSmem {
  static constexpr size_t stat_off = 0;
  static constexpr size_t tile_off = 2 * (size_t)kPrStatBytes;
  static constexpr size_t bar_off = tile_off + (size_t)kPrStages * kPrTileBytes;
  static constexpr size_t nl_off = bar_off + 128;          // [2][128] negated log-sum-exp
  static constexpr size_t lim_off = nl_off + 2 * 128 * 4;  // [2][128] last visible key
  static constexpr size_t total = lim_off + 2 * 128 * 4;   // below the 227 KB of a CTA
};
static_assert(PrSmem::total <= 232448, "shared memory of a CTA");

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

template <int PASS>
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
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sempty + 2);
  float* nl_s = reinterpret_cast<float*>(smem + PrSmem::nl_off);
  int* lim_s = reinterpret_cast<int*>(smem + PrSmem::lim_off);

  if (smem_addr(smem) & 1023u) {  // the swizzled tiles need it; a CTA's dynamic memory has it
    if (threadIdx.x == 0) set_status(p.status, RKV_DEV_SELECT_FAILED);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const RowMap m1 = row_map(p.gqa, p.max_q, kPrStat), m2 = row_map(p.gqa, p.max_q, kPrTile);
  const int items = p.units * (PASS == 1 ? p.tiles1 * p.nsplit1 : p.tiles2 * p.nsplit2);

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

  if (warp == 0) {
    // ------------------------------------------------------------------ loads
    if (lane == 0) {
      int step = 0, ic = 0, sent = 0;  // sent: stationary tiles requested
      for (int i = blockIdx.x; i < items && !aborted; i += gridDim.x) {
        const PromptItem it = prompt_item<PASS>(p, i);
        if (it.count == 0) continue;
        const int sb = ic & 1;
        if (ic >= 2 && !mbar_wait(&sempty[sb], (uint32_t)(((ic >> 1) - 1) & 1))) {
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
              !mbar_wait(&empty[s], (uint32_t)(((step / kPrStages) - 1) & 1))) {
            aborted = true;
            break;
          }
          const int y = PASS == 1
                            ? kbase + (it.first + t) * kPrTile
                            : qbase + tile_row0(m2, step_tile(p, it, it.first + t), kPrTile);
          uint8_t* dst = tiles + (size_t)s * kPrTileBytes;
          mbar_arrive_expect_tx(&full[s], (uint32_t)kPrTileBytes);
          tma_load_2d(dst, PASS == 1 ? &kmap : &qmap, 0, y, &full[s]);
          tma_load_2d(dst + 16384, PASS == 1 ? &kmap : &qmap, 64, y, &full[s]);
        }
        ++ic;
      }
      if (aborted) {
        set_status(p.status, RKV_DEV_WAIT_TIMEOUT);
        for (int j = max(0, step - kPrStages); j < step; ++j)  // let issued loads land
          mbar_wait(&full[j % kPrStages], (uint32_t)((j / kPrStages) & 1));
        for (int j = max(0, ic - 2); j < sent; ++j) mbar_wait(&sfull[j & 1], (uint32_t)((j >> 1) & 1));
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ products
    if (lane == 0) {
      int step = 0, ic = 0;
      for (int i = blockIdx.x; i < items && !aborted; i += gridDim.x) {
        const PromptItem it = prompt_item<PASS>(p, i);
        if (it.count == 0) continue;
        const int sb = ic & 1;
        if (!mbar_wait(&sfull[sb], (uint32_t)((ic >> 1) & 1))) {
          aborted = true;
          break;
        }
        const uint32_t sbase = smem_addr(stat + (size_t)sb * kPrStatBytes);
        for (int t = 0; t < it.count; ++t, ++step) {
          const int s = step % kPrStages, b = step & 1;
          if (!mbar_wait(&full[s], (uint32_t)((step / kPrStages) & 1)) ||
              (step >= 2 && !mbar_wait(&tempty[b], (uint32_t)(((step >> 1) - 1) & 1)))) {
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
      if (aborted) set_status(p.status, RKV_DEV_WAIT_TIMEOUT);
    }
  } else {
    // ------------------------------------------------------------------ accumulators
    const int rb = (warp - 2) >> 2;
    const int quarter = warp & 3;       // TMEM lanes this warp may read
    const int srow = rb * 128 + quarter * 32 + lane;  // stationary row of this thread
    const int etid = tid - 64;
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    int step = 0;
    for (int i = blockIdx.x; i < items; i += gridDim.x) {
      const PromptItem it = prompt_item<PASS>(p, i);
      if (PASS == 1 && it.L == 0 && it.tile == 0 && it.ukv == it.u * p.n_kv && etid == 0) {
        // (the first tile's split that comes first in the order reports; repeats do no harm)
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
        for (int t = 0; t < it.count; ++t, ++step) {
          const int b = step & 1;
          if (aborted) continue;
          if (!mbar_wait(&tfull[b], (uint32_t)((step >> 1) & 1))) {
            aborted = true;
            continue;
          }
          tc_fence_after();
          const int k0 = (it.first + t) * kPrTile;
          for (int cc = 0; cc < kPrTile; cc += 32) {
            uint32_t r[32];
            tmem_ld32(tmem + lane_addr + (uint32_t)((b * 2 + rb) * kPrTile + cc), r);
            float mt = -INFINITY;
            if (k0 + cc + 31 <= lim) {
#pragma unroll
              for (int j = 0; j < 32; ++j) mt = fmaxf(mt, __uint_as_float(r[j]));
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const float x = (k0 + cc + j <= lim) ? __uint_as_float(r[j]) : -INFINITY;
                r[j] = __float_as_uint(x);
                mt = fmaxf(mt, x);
              }
            }
            const float mn = fmaxf(m, mt * p.scale_log2);
            float a4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = 0; j < 32; ++j)
              a4[j & 3] += fast_exp2(fmaf(__uint_as_float(r[j]), p.scale_log2, -mn));
            l = l * fast_exp2(m - mn) + ((a4[0] + a4[1]) + (a4[2] + a4[3]));
            m = mn;
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[b]);
        }
        // every row of every item is written, so that pass 2 never meets an old workspace
        const int per = p.units * p.nsplit1, split = (i % per) % p.nsplit1;
        p.ml[((size_t)it.ukv * p.nsplit1 + split) * ((size_t)p.tiles1 * kPrStat) +
             (size_t)it.tile * kPrStat + srow] = make_float2(m, l);
      } else {
        const int key = it.tile * kPrStat + srow;
        // column e of streamed tile x: its negated log-sum-exp and its last visible key (a row
        // without a query sees none)
        auto column = [&](int t, float* nl, int* lim) {
          const int x = step_tile(p, it, it.first + t);
          const int qi = tile_query(m2, x, kPrTile, etid);
          *nl = -1e30f;
          *lim = -1;
          if (qi < 0 || qi >= it.T) return;
          *lim = it.L - it.T + qi;
          // the same row in pass 1's tiles
          const int h = m2.per_head ? x / m2.per_head : 0;
          const int row = m2.per_head
                              ? h * (m1.per_head * kPrStat) + qi
                              : x * kPrTile + etid;
          const float2* src = p.ml + (size_t)it.ukv * p.nsplit1 * p.tiles1 * kPrStat + row;
          float m = -1e30f, l = 0.f;
          for (int s = 0; s < p.nsplit1; ++s) {
            const float2 y = src[(size_t)s * p.tiles1 * kPrStat];
            const float mn = fmaxf(m, y.x);
            l = l * fast_exp2(m - mn) + y.y * fast_exp2(y.x - mn);
            m = mn;
          }
          *nl = l > 0.f ? -(m + log2f(l)) : (l == 0.f ? -1e30f : l);
        };
        float nl = 0.f;
        int lim = 0;
        if (it.count > 0) {
          if (etid < kPrTile) {
            column(0, &nl, &lim);
            nl_s[etid] = nl;
            lim_s[etid] = lim;
          }
          named_bar_sync(1, kPrEpi);
        }
        float acc = 0.f;
        for (int t = 0; t < it.count; ++t, ++step) {
          const int b = step & 1, cb = t & 1;
          const bool more = t + 1 < it.count;
          if (more && etid < kPrTile) column(t + 1, &nl, &lim);
          if (!aborted && !mbar_wait(&tfull[b], (uint32_t)((step >> 1) & 1))) aborted = true;
          if (!aborted) {
            tc_fence_after();
            // rows that are no queries, or that do not see all of the stationary keys
            int lo, hi;
            const int x = step_tile(p, it, it.first + t);
            tile_span(m2, x, kPrTile, &lo, &hi);
            const bool mask = hi >= it.T || tile_query(m2, x, kPrTile, kPrTile - 1) < 0 ||
                              it.L - it.T + lo < (it.tile + 1) * kPrStat - 1;
            float a4[4] = {0.f, 0.f, 0.f, 0.f};
            for (int cc = 0; cc < kPrTile; cc += 32) {
              uint32_t r[32];
              tmem_ld32(tmem + lane_addr + (uint32_t)((b * 2 + rb) * kPrTile + cc), r);
              const float4* n4 = reinterpret_cast<const float4*>(nl_s + cb * kPrTile + cc);
              const int4* l4 = reinterpret_cast<const int4*>(lim_s + cb * kPrTile + cc);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float4 v = n4[j];
                float y0 = fmaf(__uint_as_float(r[4 * j + 0]), p.scale_log2, v.x);
                float y1 = fmaf(__uint_as_float(r[4 * j + 1]), p.scale_log2, v.y);
                float y2 = fmaf(__uint_as_float(r[4 * j + 2]), p.scale_log2, v.z);
                float y3 = fmaf(__uint_as_float(r[4 * j + 3]), p.scale_log2, v.w);
                if (mask) {
                  const int4 q = l4[j];
                  y0 = key <= q.x ? y0 : -INFINITY;
                  y1 = key <= q.y ? y1 : -INFINITY;
                  y2 = key <= q.z ? y2 : -INFINITY;
                  y3 = key <= q.w ? y3 : -INFINITY;
                }
                a4[0] += fast_exp2(y0);
                a4[1] += fast_exp2(y1);
                a4[2] += fast_exp2(y2);
                a4[3] += fast_exp2(y3);
              }
            }
            acc += (a4[0] + a4[1]) + (a4[2] + a4[3]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tempty[b]);
          }
          if (more && etid < kPrTile) {
            nl_s[(cb ^ 1) * kPrTile + etid] = nl;
            lim_s[(cb ^ 1) * kPrTile + etid] = lim;
          }
          named_bar_sync(1, kPrEpi);
        }
        if (key < it.L) {
          if (p.nsplit2 == 1) {
            if (it.count > 0 && !aborted) p.weights[(size_t)it.ukv * p.max_len + key] += acc;
          } else {
            const int per = p.units * p.nsplit2, split = (i % per) % p.nsplit2;
            p.part[((size_t)split * p.units + it.ukv) * p.max_len + key] = acc;
          }
        }
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

// Splits only where the items alone would leave SMs without work: a split costs its own
// stationary load, and partial results that are read back.
static PromptPlan prompt_plan(int n, int n_kv, int gqa, int max_q, int max_len) {
  PromptPlan p;
  const long long units = (long long)n * n_kv;
  const int sms = device_sm_count();
  p.tiles1 = row_tiles(row_map(gqa, max_q, kPrStat), kPrStat);
  p.tiles2 = (max_len + kPrStat - 1) / kPrStat;
  auto splits = [&](long long items, int steps) {
    if (items >= sms) return 1;
    const int want = (int)(sms / items), most = (steps + 3) / 4;  // at least 4 steps a split
    return want < most ? (want > 1 ? want : 1) : most;
  };
  p.nsplit1 = splits(units * p.tiles1, (max_len + kPrTile - 1) / kPrTile);
  p.nsplit2 = splits(units * p.tiles2, row_tiles(row_map(gqa, max_q, kPrTile), kPrTile));
  return p;
}

static size_t ml_bytes(const PromptPlan& p, size_t units) {
  return align_up(units * p.nsplit1 * p.tiles1 * kPrStat * 8, 256);
}

size_t prompt_scratch_bytes(int n, int n_kv, int gqa, int max_q, int max_len) {
  const PromptPlan p = prompt_plan(n, n_kv, gqa, max_q, max_len);
  const size_t units = (size_t)n * n_kv;
  return ml_bytes(p, units) +
         (p.nsplit2 > 1 ? align_up(units * p.nsplit2 * max_len * 4, 256) : 0);
}

template <int PASS>
static cudaError_t launch_prompt_pass(const CUtensorMap& km, const CUtensorMap& qm,
                                      const PromptParams& p, cudaStream_t s) {
  cudaError_t e = ensure_dyn_smem((const void*)prompt_kernel<PASS>, PrSmem::total);
  if (e != cudaSuccess) return e;
  const long long items =
      (long long)p.units * (PASS == 1 ? p.tiles1 * p.nsplit1 : p.tiles2 * p.nsplit2);
  if (items > 0x3fffffffll) return cudaErrorInvalidConfiguration;
  const int sms = device_sm_count();
  return launch_pdl_kernel(prompt_kernel<PASS>, dim3((unsigned)(items < sms ? items : sms)),
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
  p.ml = reinterpret_cast<float2*>(w);
  p.part = reinterpret_cast<float*>(w + ml_bytes(pl, p.units));
  p.weights = a.weights;
  p.status = a.status;
  cudaError_t e = launch_prompt_pass<1>(km, qm, p, s);
  if (e != cudaSuccess) return e;
  e = launch_prompt_pass<2>(km, qm, p, s);
  if (e != cudaSuccess || p.nsplit2 == 1) return e;
  int y = (a.max_len + 255) / 256;
  return launch_pdl_kernel(prompt_sum_kernel, dim3(p.units, y < 1024 ? y : 1024), dim3(256), 0, s,
                           p);
}

}  // namespace rkv
