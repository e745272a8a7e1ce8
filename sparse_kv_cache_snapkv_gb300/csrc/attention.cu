// Attention of packed new tokens over the cache that holds their own rows already (sm_103a): a whole
// prompt or a chunk of one (causal), or a tree of drafted tokens (a bit mask among the newest rows).
//
//   o_r = sum_j p_rj v_j / sum_j p_rj,   p_rj = 2^(scale log2(e) q_r . k_j - m_r),
// over the keys j that query row r sees. m_r is a reference, not the maximum: it is the first keys'
// maximum, and moves up only when a later one passes it by kRaise (in log2); sums and outputs are then
// scaled once. p stays below 2^kRaise of its reference, so bf16 and fp32 hold it and its sums as well.
//
// Rows are (token, query head of the KV group), heads fastest: a tile of 128 rows holds 128 / gqa tokens
// of one (unit, KV head), and an item is two tiles that read each key and value once. The cache streams
// by in steps of 128 rows: S = Q K^T and O += P V on tcgen05, one tile of the pair after the other, so
// that one tile's softmax runs under the other's products. A softmax thread owns one row: no value
// crosses lanes. P goes back to TMEM, over the S it comes from, as the bf16 operand of P V: each p is
// rounded once, by 2^-9 of its value on average less, where a second bf16 part would cost half as many
// tensor operations again; the outputs are bf16 numbers with a rounding of the same size.
//
// Bound: a prompt by the tensor cores (four times 128 flops a (row, key) pair), a tree by reading the
// cache. Items of a prompt go to CTAs as they are, largest first in waves of alternating direction;
// where the longest item would outlast an equal share of all steps, every CTA takes an equal range of
// the steps instead, and a second kernel joins the parts of cut items in their order.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/rkv_testing.h"
#include "common.cuh"
#include "rkv_internal.h"
#include "tensor_core.cuh"

namespace rkv {

constexpr int kAtThreads = 384;  // warp 0 loads, 1 multiplies, 2 and 3 clean; 4..7 and 8..11: a tile's softmax
constexpr int kAtRows = 128;     // rows of a tile
constexpr int kAtTile = 128;     // cache rows of a step
constexpr int kAtStages = 5;     // K and V tiles in flight
constexpr int kAtTileBytes = kAtTile * kHeadDim * 2;  // 32 KB
constexpr uint32_t kAtCols = 512;                     // S or P of both tiles, O of both
constexpr int kPlanThreads = 1024;
constexpr int kPlanBuckets = 1024;
constexpr float kRaise = 16.f;
constexpr float kNoMax = -1e30f;
constexpr int kSplitLeast = 2;   // steps of a CTA's range
constexpr int kSplitGain = 6;    // steps that ranges must save over whole items: what parts and their join cost

struct AtSmem {
  static constexpr size_t q_off = 0;
  static constexpr size_t ring_off = 2 * (size_t)kAtTileBytes;
  static constexpr size_t bar_off = ring_off + (size_t)kAtStages * kAtTileBytes;
  static constexpr size_t total = bar_off + 256;
};
static_assert(AtSmem::total <= 232448, "shared memory of a CTA");

// One pair of tiles of a unit, for every KV head.
struct __align__(16) AtRec {
  int row0;   // packed row of its first token
  int t0;     // that token's number among the unit's new ones
  int T, L;   // the unit's new tokens, and its rows in the cache with theirs
  int u, steps;
  int before;  // steps of one KV head in the pairs before it (in the linear order)
  int pad;
};
static_assert(sizeof(AtRec) == 32, "");

struct AtPlan {
  int split;  // 1: equal ranges of the linear order, 0: whole items in the sorted one
  int count;  // pairs
  int per;    // steps of a CTA's range
  int total;  // steps of all KV heads (split)
};

struct AtFirst {
  int rec, head, off, pad;  // where a CTA's range begins (rec < 0: no range)
};

struct AtParams {
  int n, n_kv, gqa, hq, tokens, cap, words, room, ctas;
  int tile_tokens;  // 128 / gqa
  float scale_log2;
  const int32_t* q_start;
  const int32_t* len;
  const uint32_t* mask;  // nullptr: causal
  PagedMap pm;           // table == nullptr: contiguous
  bf16* out;
  AtPlan* plan;
  AtFirst* first;     // [ctas]
  AtRec* rec;         // [room], linear order
  AtRec* sorted;      // [room]
  int* unit_first;    // [n + 1]
  float2* part_ml;    // [2 ctas][256]
  float* part_o;      // [2 ctas][256][128]
  uint32_t* status;
  WaitLimit wait_limit;
  int test_skip;
};

// ------------------------------------------------------------------------------------------
// plan
// ------------------------------------------------------------------------------------------
// A unit's tokens; false (and its status bit) where the call's arrays make no sense for it.
__device__ __forceinline__ bool at_unit(const AtParams& p, int u, int* row0, int* T, int* L) {
  const int a = p.q_start[u], b = p.q_start[u + 1], l = p.len[u];
  *row0 = a;
  *T = 0;
  *L = l;
  if (l < 0 || l > p.cap) {
    set_status(p.status, RKV_DEV_LEN_OVER_CAP);
    return false;
  }
  if (a < 0 || b < a || b > p.tokens || b - a > l || (p.mask && b - a > 32 * p.words)) {
    set_status(p.status, RKV_DEV_BAD_WINDOW);
    return false;
  }
  *T = b - a;
  return true;
}

__global__ void __launch_bounds__(kPlanThreads) at_plan_kernel(AtParams p) {
  __shared__ unsigned long long scan[33];
  __shared__ int hist[kPlanBuckets];
  __shared__ int longest, sh_split, sh_per;
  const int tid = threadIdx.x, pair = 2 * p.tile_tokens;
  for (int i = tid; i < kPlanBuckets; i += kPlanThreads) hist[i] = 0;
  if (tid == 0) longest = 0;
  pdl_wait();
  pdl_trigger();
  long long carry = 0;
  for (int base = 0; base < p.n; base += kPlanThreads) {
    const int u = base + tid;
    int row0, T = 0, L;
    if (u < p.n) at_unit(p, u, &row0, &T, &L);
    const unsigned long long tiles = (unsigned long long)((T + pair - 1) / pair);
    const unsigned long long at = block_excl_scan64(tiles, scan);
    if (u < p.n) p.unit_first[u] = (int)min((long long)p.room, carry + (long long)at);
    if (tid == kPlanThreads - 1) scan[32] = at + tiles;
    __syncthreads();
    carry += (long long)scan[32];
    __syncthreads();
  }
  // (units that overlap could come to more pairs than there is room for)
  if (carry > p.room && tid == 0) set_status(p.status, RKV_DEV_BAD_WINDOW);
  const int count = (int)min((long long)p.room, carry);
  long long steps_before = 0;
  for (int base = 0; base < count; base += kPlanThreads) {
    const int e = base + tid;
    AtRec r{};
    if (e < count) {
      int lo = 0, hi = p.n;  // the last unit whose pairs begin at or before e
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.unit_first[mid] <= e) lo = mid; else hi = mid;
      }
      const int tile = e - p.unit_first[lo];
      r.u = lo;
      r.L = p.len[lo];
      r.row0 = p.q_start[lo];
      r.T = p.q_start[lo + 1] - r.row0;
      r.t0 = tile * pair;
      r.row0 += r.t0;
      const int keys = p.mask ? r.L : r.L - r.T + min(r.t0 + pair, r.T);
      r.steps = (keys + kAtTile - 1) / kAtTile;
      atomicMax(&longest, r.steps);
      atomicAdd(&hist[kPlanBuckets - 1 - min(r.steps, kPlanBuckets - 1)], 1);
    }
    const unsigned long long at = block_excl_scan64((unsigned long long)r.steps, scan);
    r.before = (int)min(0x7fffffffll, steps_before + (long long)at);
    if (e < count) p.rec[e] = r;
    if (tid == kPlanThreads - 1) scan[32] = at + (unsigned long long)r.steps;
    __syncthreads();
    steps_before += (long long)scan[32];
    __syncthreads();
  }
  const long long total = steps_before * p.n_kv;
  if (tid == 0) {
    const long long each = (total + p.ctas - 1) / p.ctas;
    sh_split = total < (1ll << 30) && longest - each >= kSplitGain && longest * 4ll > each * 5ll;
    sh_per = (int)max((long long)kSplitLeast, min(each, 1ll << 30));
    *p.plan = AtPlan{sh_split, count, sh_per, (int)min(total, 1ll << 30)};
  }
  __syncthreads();
  if (!sh_split) {  // largest first
    const unsigned long long mine = (unsigned long long)hist[tid];
    const unsigned long long at = block_excl_scan64(mine, scan);
    hist[tid] = (int)at;
    __syncthreads();
    for (int e = tid; e < count; e += kPlanThreads) {
      const AtRec r = p.rec[e];
      p.sorted[atomicAdd(&hist[kPlanBuckets - 1 - min(r.steps, kPlanBuckets - 1)], 1)] = r;
    }
    return;
  }
  for (int c = tid; c < p.ctas; c += kPlanThreads) {
    const long long a = (long long)c * sh_per;
    AtFirst f{-1, 0, 0, 0};
    if (a < total) {
      int lo = 0, hi = count;  // the last pair that begins at or before a
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((long long)p.rec[mid].before * p.n_kv <= a) lo = mid; else hi = mid;
      }
      const int r = (int)(a - (long long)p.rec[lo].before * p.n_kv), steps = p.rec[lo].steps;
      f.rec = lo;
      f.head = r / steps;
      f.off = r - f.head * steps;
    }
    p.first[c] = f;
  }
}
static_assert(kPlanBuckets == kPlanThreads, "one bucket per thread in the scan");

// ------------------------------------------------------------------------------------------
// the pieces of a CTA, the same for every warp
// ------------------------------------------------------------------------------------------
struct Piece {
  AtRec r;
  int g, s0;    // KV head, first step
  int cnt[2];   // steps of each tile, from s0
  int steps;    // the larger of the two
  int slot;     // where its part goes; -1: the item is whole
};

struct Pieces {
  int split, count, per, total;
  int wave;                   // whole items
  int rec, head, off, left;   // ranges
  __device__ __forceinline__ void init(const AtParams& p) {
    const AtPlan pl = *p.plan;
    split = pl.split;
    count = pl.count;
    per = pl.per;
    total = pl.total;
    wave = 0;
    left = 0;
    if (split) {
      const AtFirst f = p.first[blockIdx.x];
      rec = f.rec;
      head = f.head;
      off = f.off;
      const long long a = (long long)blockIdx.x * per;
      left = f.rec < 0 ? 0 : (int)min((long long)per, total - a);
    }
  }
  __device__ __forceinline__ bool next(const AtParams& p, Piece& x) {
    int len;
    if (split) {
      if (left <= 0) return false;
      x.r = p.rec[rec];
      x.g = head;
      x.s0 = off;
      len = min(x.r.steps - off, left);
      x.slot = off > 0 ? 2 * (int)blockIdx.x : len < x.r.steps ? 2 * (int)blockIdx.x + 1 : -1;
      left -= len;
      off = 0;
      if (++head == p.n_kv) {
        head = 0;
        ++rec;
      }
    } else {
      const long long items = (long long)count * p.n_kv;
      long long i;
      do {
        i = (long long)wave * gridDim.x + ((wave & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        if ((long long)wave * gridDim.x >= items) return false;
        ++wave;
      } while (i >= items);
      const int e = (int)(i / p.n_kv);
      x.r = p.sorted[e];
      x.g = (int)(i - (long long)e * p.n_kv);
      x.s0 = 0;
      len = x.r.steps;
      x.slot = -1;
    }
    x.steps = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = x.r.t0 + h * p.tile_tokens;  // the tile's first token
      const int keys = p.mask ? x.r.L : x.r.L - x.r.T + min(t + p.tile_tokens, x.r.T);
      const int all = t < x.r.T ? (keys + kAtTile - 1) / kAtTile : 0;
      x.cnt[h] = max(0, min(x.s0 + len, all) - x.s0);
      x.steps = max(x.steps, x.cnt[h]);
    }
    return true;
  }
};

// A warpgroup's registers per thread: the first hands back what the others then take (setmaxnreg; the
// shares add up to what the block was launched with, so that no take can wait for ever).
constexpr int kAtLoadRegs = 88, kAtSoftmaxRegs = 208, kAtLaunchRegs = 168;
static_assert(kAtLoadRegs + 2 * kAtSoftmaxRegs <= 3 * kAtLaunchRegs, "");
static_assert(kAtThreads * kAtLaunchRegs <= 65536 && kAtThreads * (kAtLaunchRegs + 8) > 65536, "");
template <int N>
__device__ __forceinline__ void reg_release() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_take() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// D += A B with A (bf16, 128 x 16) in TMEM.
__device__ __forceinline__ void umma_bf16_ta(uint32_t tmem_d, uint32_t tmem_a, uint64_t b,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(tmem_d), "r"(tmem_a), "l"(b), "r"(idesc), "r"(accumulate));
}

// V as the B operand of P V: rows are the reduction, dimensions contiguous (64 of them in 128 bytes,
// swizzled; the other 64 are 16 KB further, eight rows 1024 bytes).
__device__ __forceinline__ uint64_t desc_rows_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(16384 >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
constexpr uint32_t kIdescS = idesc_bf16(kAtRows, kAtTile);
constexpr uint32_t kIdescO = idesc_bf16(kAtRows, kHeadDim) | (1u << 16);  // B is not K-major

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
      ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// The tile's rows of (token, head), heads fastest.
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(smem_addr(dst)), "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}

struct AtBars {
  uint64_t full[kAtStages], empty[kAtStages];  // the ring of K and V tiles
  uint64_t qfull[2], qempty[2];
  uint64_t sfull[2];   // S of a step is there (and all products before it are done)
  uint64_t pfull[2];   // P of a step is written
  uint64_t ofull[2];   // the item's last product is done
  uint64_t ofree[2];   // O has been read
  uint64_t dirty, clean;      // a V tile with rows behind the last is next; they are zeros
  uint64_t drain;      // everything issued is done (after a wait gave up)
  uint32_t tmem;
};
static_assert(sizeof(AtBars) <= 256, "");

template <bool PAGED, bool TREE>
__global__ void __launch_bounds__(kAtThreads, 1)
    at_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
              const __grid_constant__ CUtensorMap vmap, const __grid_constant__ AtParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* qs = smem + AtSmem::q_off;
  uint8_t* ring = smem + AtSmem::ring_off;
  AtBars& bar = *reinterpret_cast<AtBars*>(smem + AtSmem::bar_off);

  if (smem_addr(smem) & 1023u) {  // the swizzled tiles need it; a CTA's dynamic memory has it
    if (threadIdx.x == 0) set_status(p.status, RKV_DEV_SELECT_FAILED);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kAtStages; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.qfull[i], 1);
      mbar_init(&bar.qempty[i], 1);
      mbar_init(&bar.sfull[i], 1);
      mbar_init(&bar.pfull[i], 4);
      mbar_init(&bar.ofull[i], 1);
      mbar_init(&bar.ofree[i], 4);
    }
    mbar_init(&bar.dirty, 1);
    mbar_init(&bar.clean, 2);
    mbar_init(&bar.drain, 1);
    fence_barrier_init();
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_addr(&bar.tmem)), "r"(kAtCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;
  pdl_wait();
  pdl_trigger();
  const WaitLimit limit = p.wait_limit;
  bool aborted = false;
  Pieces it;
  it.init(p);
  Piece x{};

  if (warp < 4) {
  reg_release<kAtLoadRegs>();
  if (warp == 0) {
    // ------------------------------------------------------------------ loads
    const int skip = blockIdx.x == 0 ? p.test_skip : 0;
    const uint32_t qbytes = (uint32_t)(p.gqa * p.tile_tokens * kHeadDim * 2);
    const int rows = PAGED ? min(p.pm.block, kAtTile) : kAtTile;  // of one copy
    int ld = 0;                  // tiles requested
    int nq[2] = {0, 0};          // Q tiles requested
    auto slot = [&]() {          // waits for the next place of the ring
      const int s = ld % kAtStages;
      if (ld >= kAtStages &&
          !mbar_wait_warp(&bar.empty[s], (uint32_t)((ld / kAtStages - 1) & 1), limit)) {
        aborted = true;
        return -1;
      }
      return s;
    };
    // rows [k0, k0 + 128) of the unit; behind L nothing need be there
    auto tile = [&](const CUtensorMap* map, int s, int k0, int blk) {
      uint8_t* dst = ring + (size_t)s * kAtTileBytes;
      if (PAGED) {
        const int copies = min(kAtTile / rows, (x.r.L - k0 + rows - 1) / rows);
        if (lane == 0) mbar_arrive_expect_tx(&bar.full[s], (uint32_t)(copies * rows * 256));
        __syncwarp();
        for (int c = lane; c < copies; c += 32) {
          const int t = k0 + c * rows;
          const int b = c == lane ? blk : paged_block(p.pm, x.r.u, t, p.status);
          const int y = (b * p.n_kv + x.g) * p.pm.block + (t & (p.pm.block - 1));
          tma_load_2d(dst + c * rows * 128, map, 0, y, &bar.full[s]);
          tma_load_2d(dst + 16384 + c * rows * 128, map, 64, y, &bar.full[s]);
        }
      } else if (lane == 0) {
        const int y = (x.r.u * p.n_kv + x.g) * p.cap + k0;
        mbar_arrive_expect_tx(&bar.full[s], kAtTileBytes);
        tma_load_2d(dst, map, 0, y, &bar.full[s]);
        tma_load_2d(dst + 16384, map, 64, y, &bar.full[s]);
      }
      __syncwarp();
    };
    while (!aborted && it.next(p, x)) {
      for (int j = 0; j < x.steps && !aborted; ++j) {
        const int k0 = (x.s0 + j) * kAtTile;
        int blk = 0;
        if (PAGED && k0 + lane * rows < x.r.L && lane * rows < kAtTile)
          blk = paged_block(p.pm, x.r.u, k0 + lane * rows, p.status);
        int s = slot();
        if (s < 0) break;
        if (!(skip == RKV_TESTING_ATTENTION_KEYS && ld == 0)) tile(&kmap, s, k0, blk);
        ++ld;
        if (j == 0) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (aborted || x.cnt[h] == 0) continue;
            if (nq[h] > 0 && !mbar_wait_warp(&bar.qempty[h], (uint32_t)((nq[h] - 1) & 1), limit)) {
              aborted = true;
              continue;
            }
            if (lane == 0 && !(skip == RKV_TESTING_ATTENTION_QUERIES && nq[h] == 0)) {
              uint8_t* dst = qs + (size_t)h * kAtTileBytes;
              mbar_arrive_expect_tx(&bar.qfull[h], qbytes);
              for (int c = 0; c < 2; ++c)
                tma_load_3d(dst + c * 16384, &qmap, 64 * c, x.g * p.gqa,
                            x.r.row0 + h * p.tile_tokens, &bar.qfull[h]);
            }
            __syncwarp();
            ++nq[h];
          }
          if (aborted) break;
        }
        s = slot();
        if (s < 0) break;
        if (!(skip == RKV_TESTING_ATTENTION_VALUES && ld == 1)) tile(&vmap, s, k0, blk);
        ++ld;
      }
    }
    if (aborted && lane == 0) set_status(p.status, RKV_DEV_WAIT_TIMEOUT);
    // every issued load lands before the CTA ends, whoever gave up (else they have, and this is no wait)
    for (int j = max(0, ld - kAtStages); j < ld; ++j)
      mbar_wait_warp(&bar.full[j % kAtStages], (uint32_t)((j / kAtStages) & 1), drain_limit(limit));
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (nq[h] > 0) mbar_wait_warp(&bar.qfull[h], (uint32_t)((nq[h] - 1) & 1), drain_limit(limit));
  } else if (warp == 1) {
    // ------------------------------------------------------------------ products
    if (lane == 0) {
      int steps = 0;  // steps begun: K tile 2 steps of the ring, V tile 2 steps + 1
      int nq[2] = {0, 0}, np[2] = {0, 0}, no[2] = {0, 0}, nclean = 0;
      bool pend[2] = {false, false}, first[2] = {false, false}, last[2] = {false, false};  // P V products to come
      int vload = 0;
      bool vtail = false, vwaited = false, vboth = false;
      auto wait = [&](uint64_t* b, uint32_t parity) {
        if (!aborted && !mbar_wait(b, parity, limit)) aborted = true;
        return !aborted;
      };
      auto product = [&](int h) {  // O of tile h += P V
        pend[h] = false;
        if (!wait(&bar.pfull[h], (uint32_t)(np[h] & 1))) return;
        ++np[h];
        if (first[h] && no[h] > 0 && !wait(&bar.ofree[h], (uint32_t)((no[h] - 1) & 1))) return;
        const int s = vload % kAtStages;
        if (!vwaited) {
          if (!wait(&bar.full[s], (uint32_t)((vload / kAtStages) & 1))) return;
          if (vtail && !wait(&bar.clean, (uint32_t)(nclean++ & 1))) return;
          vwaited = true;
        }
        tc_fence_after();
        const uint32_t b = smem_addr(ring + (size_t)s * kAtTileBytes);
        const uint32_t d = tmem + 256 + h * 128, a = tmem + h * 128;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_bf16_ta(d, a + 8 * kk, desc_rows_sw128(b + kk * 2048), kIdescO, kk > 0 || !first[h]);
        if (h == 1 || !vboth) umma_commit(&bar.empty[s]);
        if (last[h]) {
          umma_commit(&bar.ofull[h]);
          ++no[h];
        }
      };
      auto scores = [&](int h, bool begin, bool end, bool only, int kload) {  // S of tile h = Q K^T
        if (begin && !wait(&bar.qfull[h], (uint32_t)(nq[h]++ & 1))) return;
        const int s = kload % kAtStages;
        if (!wait(&bar.full[s], (uint32_t)((kload / kAtStages) & 1))) return;
        tc_fence_after();
        const uint32_t a = smem_addr(qs + (size_t)h * kAtTileBytes);
        const uint32_t b = smem_addr(ring + (size_t)s * kAtTileBytes);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = (uint32_t)((kk >> 2) * 16384 + (kk & 3) * 32);
          umma_bf16(tmem + h * 128, desc_sw128(a + off), desc_sw128(b + off), kIdescS, kk > 0);
        }
        umma_commit(&bar.sfull[h]);
        if (end) umma_commit(&bar.qempty[h]);
        if (h == 1 || only) umma_commit(&bar.empty[s]);
      };
      while (!aborted && it.next(p, x)) {
        for (int j = 0; j < x.steps && !aborted; ++j, ++steps) {
          const bool act[2] = {j < x.cnt[0], j < x.cnt[1]};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!aborted && pend[h]) product(h);
            if (!aborted && act[h]) scores(h, j == 0, j == x.cnt[h] - 1, !act[1], 2 * steps);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            pend[h] = act[h];
            first[h] = j == 0;
            last[h] = j == x.cnt[h] - 1;
          }
          vload = 2 * steps + 1;
          vboth = act[1];
          vwaited = false;
          vtail = (x.s0 + j + 1) * kAtTile > x.r.L;
          if (vtail) mbar_arrive(&bar.dirty);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (!aborted && pend[h]) product(h);
      if (aborted) {
        set_status(p.status, RKV_DEV_WAIT_TIMEOUT);
        umma_commit(&bar.drain);  // let issued products end
        mbar_wait(&bar.drain, 0u, drain_limit(limit));
      }
    }
  } else {
    // ------------------------------------------------------------------ rows behind the last
    // p is 0 there, but 0 times what the cache may hold (infinity, NaN) is not. The tile's place in the ring
    // is its own from when its step's scores are issued (they are behind all products that used the place)
    // until its product, so the wait for its load cannot be taken for another one's.
    int steps = 0, ntail = 0;
    while (!aborted && it.next(p, x)) {
      const int at = x.r.L / kAtTile - x.s0, cut = x.r.L % kAtTile;  // the step that the sequence ends in
      if (cut && at >= 0 && at < x.steps) {
        const int load = 2 * (steps + at) + 1, s = load % kAtStages;
        if (!mbar_wait_warp(&bar.dirty, (uint32_t)(ntail++ & 1), limit) ||
            !mbar_wait_warp(&bar.full[s], (uint32_t)((load / kAtStages) & 1), limit)) {
          aborted = true;
          break;
        }
        // (warps 2 and 3: 64 dimensions each)
        uint4* v = reinterpret_cast<uint4*>(ring + (size_t)s * kAtTileBytes + (warp - 2) * 16384 + cut * 128);
        for (int i = lane; i < (kAtTile - cut) * 8; i += 32) v[i] = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.clean);
      }
      steps += x.steps;
    }
  }
  } else {
    reg_take<kAtSoftmaxRegs>();
    // ------------------------------------------------------------------ softmax of a tile
    const int h = (warp >> 2) - 1, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t sp = tmem + lanes + h * 128, od = tmem + lanes + 256 + h * 128;
    const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2);
    const int tok = row / p.gqa, head = row - tok * p.gqa;
    int ns = 0, no = 0;  // waits for S and for the last product
    while (!aborted && it.next(p, x)) {
      const int t = x.r.t0 + h * p.tile_tokens + tok;  // this row's token
      const bool valid = tok < p.tile_tokens && t < x.r.T;
      const int base = x.r.L - x.r.T;
      const int lim = valid ? base + t : -1;  // last key of a causal row
      const bool idle = !__any_sync(0xffffffffu, valid);
      const uint32_t* bits = TREE ? p.mask + (size_t)(x.r.row0 + h * p.tile_tokens + tok) * p.words : nullptr;
      float m = kNoMax, l = 0.f;
      for (int j = 0; j < x.cnt[h] && !aborted; ++j) {
        if (!mbar_wait_warp(&bar.sfull[h], (uint32_t)(ns & 1), limit)) {
          aborted = true;
          break;
        }
        ++ns;
        if (idle) {
          if (lane == 0) mbar_arrive(&bar.pfull[h]);
          continue;
        }
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32_start(sp + 32 * c, s[c]);
        const int k0 = (x.s0 + j) * kAtTile;
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_wait(s[c]);
        // keys that the row does not see
        if (TREE) {
          if (k0 + kAtTile > base) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int d = k0 + 32 * c - base;  // number of the chunk's first key among the new ones
              uint32_t sees = 0xffffffffu;
              if (d > -32) {
                // bits d .. d + 31 of the row, ones where d is below 0, zeros from T on
                sees = 0u;
                if (valid) {
                  const int w = d >> 5, o = d & 31;
                  const uint32_t a = w < 0 ? 0xffffffffu : w * 32 < x.r.T ? bits[w] : 0u;
                  const uint32_t b = (w + 1) * 32 < x.r.T ? bits[w + 1] : 0u;
                  sees = o ? (a >> o) | (b << (32 - o)) : a;
                  const int end = x.r.T - d;
                  if (end < 32) sees &= end <= 0 ? 0u : (1u << end) - 1u;
                }
              }
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((sees >> i) & 1u)) s[c][i] = 0xff800000u;
            }
          }
        } else if (__any_sync(0xffffffffu, k0 + kAtTile - 1 > lim)) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (k0 + 32 * c + i > lim) s[c][i] = 0xff800000u;
        }
        float mt[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mt[c] = __uint_as_float(s[c][0]);
#pragma unroll
          for (int i = 1; i < 32; ++i) mt[c] = fmaxf(mt[c], __uint_as_float(s[c][i]));
        }
        const float mn = fmaxf(fmaxf(mt[0], mt[1]), fmaxf(mt[2], mt[3])) * p.scale_log2;
        if (j == 0) {
          m = fmaxf(mn, kNoMax);
        } else if (__any_sync(0xffffffffu, mn > m + kRaise)) {
          // (the product before this step's S is done: S was issued behind it)
          const float to = fmaxf(m, mn), f = fast_exp2(m - to);
          m = to;
          l *= f;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tmem_ld32(od + 32 * c, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
            tmem_st32(od + 32 * c, o);
          }
        }
        const uint64_t off = pack2(-m, -m);
        uint64_t acc[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t out[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int a = 2 * i + 64 * c;
            const float2 y = unpack2(fma2(pack2(__uint_as_float(s[a >> 5][a & 31]),
                                                __uint_as_float(s[a >> 5][(a & 31) + 1])), scale2, off));
            const float e0 = fast_exp2(y.x), e1 = fast_exp2(y.y);
            acc[i & 1] = add2(acc[i & 1], pack2(e0, e1));
            out[i] = pack_bf16x2(e0, e1);
          }
          tmem_st32(sp + 32 * c, out);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.pfull[h]);
        const float2 sum = unpack2(add2(acc[0], acc[1]));
        l += sum.x + sum.y;
      }
      if (aborted) break;
      if (x.cnt[h] == 0) {  // a part that this tile has no steps in
        if (x.slot >= 0) p.part_ml[(size_t)x.slot * 256 + h * 128 + row] = make_float2(kNoMax, 0.f);
        continue;
      }
      if (!mbar_wait_warp(&bar.ofull[h], (uint32_t)(no & 1), limit)) {
        aborted = true;
        break;
      }
      ++no;
      tc_fence_after();
      if (!idle) {
        const bool none = l == 0.f;  // the row sees nothing: zeros, whatever v holds
        const float f = l > 0.f ? 1.f / l : l;
        bf16* dst = p.out + ((size_t)(x.r.row0 + h * p.tile_tokens + tok) * p.hq + x.g * p.gqa + head) * kHeadDim;
        float* part = p.part_o + ((size_t)max(x.slot, 0) * 256 + h * 128 + row) * kHeadDim;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t o[32];
          tmem_ld32(od + 32 * c, o);
          if (c == 3) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.ofree[h]);
          }
          if (valid && x.slot >= 0) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<uint4*>(part + 32 * c + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          } else if (valid) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = none ? 0u : pack_bf16x2(__uint_as_float(o[i + 2 * k]) * f, __uint_as_float(o[i + 2 * k + 1]) * f);
              *reinterpret_cast<uint4*>(dst + 32 * c + i) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();
        }
      } else if (lane == 0) {
        mbar_arrive(&bar.ofree[h]);
      }
      if (x.slot >= 0) p.part_ml[(size_t)x.slot * 256 + h * 128 + row] = make_float2(m, valid ? l : 0.f);
    }
    if (aborted && lane == 0) set_status(p.status, RKV_DEV_WAIT_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kAtCols)
                 : "memory");
  }
}

// Joins the parts of the items that ranges cut: the item in which CTA x + 1's range begins, unless it was
// cut before already (grid: ranges' borders x groups of rows; a warp per row, four columns a lane).
constexpr int kJoinRows = 32;
__global__ void __launch_bounds__(256) at_join_kernel(AtParams p) {
  pdl_wait();
  const AtPlan pl = *p.plan;
  if (!pl.split) return;
  const int c = blockIdx.x + 1, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const AtFirst f = p.first[c];
  if (f.rec < 0 || f.off == 0) return;
  const long long a = (long long)c * pl.per - f.off;
  const int c0 = (int)(a / pl.per);
  if (c0 != c - 1) return;
  const AtRec r = p.rec[f.rec];
  const int parts = (int)((a + r.steps - 1) / pl.per) - c0 + 1;
  for (int k = warp; k < kJoinRows; k += 8) {
    const int row = blockIdx.y * kJoinRows + k, tok = (row & 127) / p.gqa, t = (row >> 7) * p.tile_tokens + tok;
    if (tok >= p.tile_tokens || r.t0 + t >= r.T) continue;
    float m = kNoMax, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < parts; ++i) {
      const size_t at = (size_t)(i ? 2 * (c0 + i) : 2 * c0 + 1) * 256 + row;
      const float2 y = p.part_ml[at];
      if (y.y == 0.f) continue;
      const float4 v = *reinterpret_cast<const float4*>(p.part_o + at * kHeadDim + 4 * lane);
      const float to = fmaxf(m, y.x), f0 = fast_exp2(m - to), f1 = fast_exp2(y.x - to);
      m = to;
      l = l * f0 + y.y * f1;
      o.x = o.x * f0 + v.x * f1;
      o.y = o.y * f0 + v.y * f1;
      o.z = o.z * f0 + v.z * f1;
      o.w = o.w * f0 + v.w * f1;
    }
    const float s = l > 0.f ? 1.f / l : l;
    bf16* dst = p.out + ((size_t)(r.row0 + t) * p.hq + f.head * p.gqa + (row & 127) - tok * p.gqa) * kHeadDim;
    *reinterpret_cast<uint2*>(dst + 4 * lane) = make_uint2(pack_bf16x2(o.x * s, o.y * s), pack_bf16x2(o.z * s, o.w * s));
  }
}

// ------------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------------
struct AtSizes {
  size_t plan, first, rec, unit, ml, o;
  int room;
};

static AtSizes at_sizes(int n, int gqa, int tokens) {
  AtSizes z;
  const int pair = 2 * (kAtRows / gqa), ctas = device_sm_count();
  z.room = tokens / pair + n;
  z.plan = 256;
  z.first = align_up((size_t)ctas * sizeof(AtFirst), 256);
  z.rec = align_up((size_t)z.room * sizeof(AtRec), 256);
  z.unit = align_up((size_t)(n + 1) * 4, 256);
  z.ml = (size_t)2 * ctas * 256 * sizeof(float2);
  z.o = (size_t)2 * ctas * 256 * kHeadDim * 4;
  return z;
}

size_t attention_scratch_bytes(int n, int gqa, int tokens) {
  const AtSizes z = at_sizes(n, gqa, tokens);
  return z.plan + z.first + 2 * z.rec + z.unit + z.ml + z.o;
}

// tokens x heads x 128 bf16, tokens `stride` elements apart: boxes of 64 columns of a group's heads of as
// many tokens as a tile holds
static bool make_queries_map(CUtensorMap* map, const AttentionArgs& a, int hq, int tile_tokens) {
  EncodeTiledFn enc = get_encoder();
  if (!enc) return false;
  cuuint64_t dims[3] = {(cuuint64_t)kHeadDim, (cuuint64_t)hq, (cuuint64_t)a.tokens};
  cuuint64_t strides[2] = {(cuuint64_t)kHeadDim * 2, (cuuint64_t)a.q_stride * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)a.gqa, (cuuint32_t)tile_tokens};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<bf16*>(a.q), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool PAGED, bool TREE>
static cudaError_t launch_at(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& vm,
                             const AtParams& p, cudaStream_t s) {
  const cudaError_t e = ensure_dyn_smem((const void*)at_kernel<PAGED, TREE>, AtSmem::total);
  if (e != cudaSuccess) return e;
  // the warpgroups' shares count on the registers that the block is launched with
  static const bool regs_ok = [] {
    cudaFuncAttributes f;
    return cudaFuncGetAttributes(&f, (const void*)at_kernel<PAGED, TREE>) == cudaSuccess &&
           f.numRegs == kAtLaunchRegs;
  }();
  if (!regs_ok) return cudaErrorInvalidConfiguration;
  return launch_pdl_kernel(at_kernel<PAGED, TREE>, dim3(p.ctas), dim3(kAtThreads), AtSmem::total, s, qm,
                           km, vm, p);
}

cudaError_t launch_attention(const AttentionArgs& a, cudaStream_t s) {
  const int hq = a.n_kv * a.gqa, tile_tokens = kAtRows / a.gqa;
  const bool paged = a.pm.table != nullptr;
  const uint64_t rows = paged ? (uint64_t)a.pm.num_blocks * a.n_kv * a.pm.block : (uint64_t)a.n * a.n_kv * a.cap;
  const int box = paged && a.pm.block < kAtTile ? a.pm.block : kAtTile;
  CUtensorMap qm, km, vm;
  if (!make_queries_map(&qm, a, hq, tile_tokens) || !make_rows_map(&km, a.k, rows, box) ||
      !make_rows_map(&vm, a.v, rows, box))
    return cudaErrorInvalidValue;
  const AtSizes z = at_sizes(a.n, a.gqa, a.tokens);
  AtParams p{};
  p.n = a.n;
  p.n_kv = a.n_kv;
  p.gqa = a.gqa;
  p.hq = hq;
  p.tokens = a.tokens;
  p.cap = a.cap;
  p.words = a.words;
  p.room = z.room;
  p.ctas = device_sm_count();
  p.tile_tokens = tile_tokens;
  p.scale_log2 = a.scale_log2;
  p.q_start = a.q_start;
  p.len = a.len;
  p.mask = a.mask;
  p.pm = a.pm;
  p.out = a.out;
  unsigned char* w = static_cast<unsigned char*>(a.scratch);
  p.plan = reinterpret_cast<AtPlan*>(w);
  w += z.plan;
  p.first = reinterpret_cast<AtFirst*>(w);
  w += z.first;
  p.rec = reinterpret_cast<AtRec*>(w);
  w += z.rec;
  p.sorted = reinterpret_cast<AtRec*>(w);
  w += z.rec;
  p.unit_first = reinterpret_cast<int*>(w);
  w += z.unit;
  p.part_ml = reinterpret_cast<float2*>(w);
  w += z.ml;
  p.part_o = reinterpret_cast<float*>(w);
  p.status = a.status;
  p.wait_limit = a.wait_limit_ns ? WaitLimit{a.wait_limit_ns} : kWaitLimit;
  p.test_skip = a.test_skip;
  cudaError_t e = launch_pdl_kernel(at_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, p);
  if (e != cudaSuccess) return e;
  if (p.mask)
    e = paged ? launch_at<true, true>(qm, km, vm, p, s) : launch_at<false, true>(qm, km, vm, p, s);
  else
    e = paged ? launch_at<true, false>(qm, km, vm, p, s) : launch_at<false, false>(qm, km, vm, p, s);
  if (e != cudaSuccess || p.ctas < 2) return e;
  return launch_pdl_kernel(at_join_kernel, dim3(p.ctas - 1, 256 / kJoinRows), dim3(256), 0, s, p);
}

}  // namespace rkv
