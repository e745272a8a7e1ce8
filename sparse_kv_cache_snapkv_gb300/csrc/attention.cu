// Attention of packed new tokens over the cache that holds their own rows already (sm_103a): a whole
// prompt or a chunk of one (causal), or a tree of drafted tokens (a bit mask among the newest rows).
//
//   o_r = sum_j p_rj v_j / sum_j p_rj,   p_rj = 2^(scale log2(e) q_r . k_j - m_r),
// over the keys j that query row r sees. m_r is a reference, not the maximum: it is the maximum of an item's
// first 32 keys, and moves up where the p of a step come to more than kLargest; sums and outputs are then scaled
// once. So most steps look for no maximum, and bf16 and fp32 hold p, its sums and the outputs all the same.
//
// Rows are (token, query head of the KV group), heads fastest: a tile of 128 rows holds 128 / gqa tokens
// of one (unit, KV head), and an item is two tiles that read each key and value once. The cache streams
// by in steps of 128 rows: S = Q K^T and O += P V on tcgen05 (operands by TMA, S, P and O in TMEM), the two tiles
// in turns, so that one's softmax runs under the other's products. A softmax thread owns one row: no value
// crosses lanes. P goes back to TMEM, over the S it comes from, as the bf16 operand of P V: each p is rounded
// once, by at most 2^-8 of its value, where a second bf16 part would cost half as many tensor operations again;
// the outputs are bf16 numbers with a rounding of the same size.
//
// Sixteen warps: loads, the two tiles' products, pieces of work (one warp each of the first two and the last,
// as warps 0 to 3), four write outputs, four each are a tile's softmax. Between them only mbarriers, all waits
// bounded.
//
// Bound (times here and below are the GPU's, of calls replayed in a graph; a call from Python that is waited for
// by the next takes up to 40 us more): a prompt by the tensor cores (8192 tokens, 32 heads of 8 KV heads: 311 us,
// 1.77 PFLOP/s of the causal half, 92 % of a cuBLAS product's rate; the GPU is at its power limit); a tree by reading
// the cache (32 trees over up to 20480 rows: 264 us, 6.5 TB/s) or, with 256 rows an item, by both. A step of a pair
// takes some 2600 clocks, 2048 of them products; what is left is the chain from S through the softmax to P and the
// wakes between. Items of a prompt go to CTAs as they are, largest first in waves of alternating direction; where
// the longest item would outlast an equal share of all steps, every CTA takes an equal range of the steps
// instead, and a second kernel joins the parts of cut items in their order (131071 rows, 64 drafted tokens:
// 115 us, 80 of them the floor).
#include <cuda.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

#include "../../include/rkv_testing.h"
#include "common.cuh"
#include "rkv_internal.h"
#include "tensor_core.cuh"

namespace rkv {

constexpr int kAtThreads = 512;  // warp 0 loads, 1 and 2 multiply, 3 finds the pieces; 4..7: outputs;
                                // 8..11 and 12..15: a tile's softmax
constexpr int kAtRows = 128;     // rows of a tile
constexpr int kAtTile = 128;     // cache rows of a step
constexpr int kAtStages = 5;     // K and V tiles in flight
constexpr int kAtTileBytes = kAtTile * kHeadDim * 2;  // 32 KB
constexpr int kAtPieces = 4;     // pieces that the finding warp may be ahead
constexpr int kAtReaders = 15;   // warps that read them
constexpr uint32_t kAtCols = 512;                     // S or P of both tiles, O of both
constexpr int kPlanThreads = 1024;
constexpr int kFewPairs = 64;    // pairs of tiles whose plan a warp makes in its registers
constexpr int kPlanBuckets = 1024;
constexpr float kLargest = 1048576.f;  // 2^20: what the p of a row's step may come to before m is raised
constexpr float kNoMax = -1e30f;
constexpr int kSplitLeast = 2;   // steps of a CTA's range
// Steps that ranges must save over whole items, which is what parts and their join cost (8 steps each of 8
// items: whole 15.5 us, cut into 2 steps each 18.6; 12 steps of 16: 24.2 and 29.0; 16 of 32: 26.1 both ways).
constexpr int kSplitGain = 12;

struct AtSmem {
  static constexpr size_t q_off = 0;
  static constexpr size_t ring_off = 2 * (size_t)kAtTileBytes;
  static constexpr size_t bar_off = ring_off + (size_t)kAtStages * kAtTileBytes;
  static constexpr size_t piece_off = bar_off + 512;
  static constexpr size_t sum_off = piece_off + kAtPieces * 48;  // [2 turns][2 tiles][128]
  static constexpr size_t total = sum_off + 2 * 2 * kAtRows * 4;
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
  int few;          // 1: every CTA makes the plan of at most kFewPairs pairs itself
  int tile_tokens;  // 128 / gqa
  int part_rows;    // rows of an item that can be any: all 256, or those of the call's few tokens
  int whole;  // 1: outputs and parts begin on 32 bytes
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
  float2* part_ml;    // [2 ctas][part_rows]
  float* part_o;      // [2 ctas][part_rows][128]
  uint32_t* status;
  WaitLimit wait_limit;
  WaitLimit item_limit;  // of waits that may take as long as an item
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

// Whole items, unless the longest would outlast an equal share of all steps by what parts and their join cost. The
// items' waves are not looked at: a few more items of one length than CTAs stay whole too and take two waves, the
// second nearly empty (20 requests of one token over 16384 rows, 160 items: 343 us, as long as 32 requests'; the
// floor is 201), where the spread of a ragged batch evens its waves out.
__device__ __forceinline__ AtPlan at_decide(long long total, int longest, int count, int ctas) {
  const long long each = total < (1ll << 30) ? ((int)total + ctas - 1) / ctas : (total + ctas - 1) / ctas;
  const int split = total < (1ll << 30) && longest - each >= kSplitGain && longest * 4ll > each * 5ll;
  return AtPlan{split, count, (int)max((long long)kSplitLeast, min(each, 1ll << 30)), (int)min(total, 1ll << 30)};
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
    const AtPlan pl = at_decide(total, longest, count, p.ctas);
    sh_split = pl.split;
    sh_per = pl.per;
    *p.plan = pl;
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
// the pieces of a CTA: one warp finds them, the others read them in shared memory
// ------------------------------------------------------------------------------------------
struct __align__(16) Piece {
  int row0, t0, T, L;  // as in its AtRec
  int u, g, s0;        // unit, KV head, first step
  int steps;           // the larger of cnt; 0: there is no piece any more
  int cnt0, cnt1;      // steps of each tile, from s0
  int slot;            // where its part goes; -1: the item is whole
  int pad;
  __device__ __forceinline__ int cnt(int h) const { return h ? cnt1 : cnt0; }
};
static_assert(sizeof(Piece) == 48, "three 16-byte words");

// Field by field, so that a piece stays in registers (read through a pointer to it, it lay in local memory).
__device__ __forceinline__ void read_piece(Piece& x, const Piece* from) {
  const int4* src = reinterpret_cast<const int4*>(from);
  const int4 a = src[0], b = src[1], c = src[2];
  x.row0 = a.x;
  x.t0 = a.y;
  x.T = a.z;
  x.L = a.w;
  x.u = b.x;
  x.g = b.y;
  x.s0 = b.z;
  x.steps = b.w;
  x.cnt0 = c.x;
  x.cnt1 = c.y;
  x.slot = c.z;
}
__device__ __forceinline__ void write_piece(Piece* to, const Piece& x) {
  int4* dst = reinterpret_cast<int4*>(to);
  dst[0] = make_int4(x.row0, x.t0, x.T, x.L);
  dst[1] = make_int4(x.u, x.g, x.s0, x.steps);
  dst[2] = make_int4(x.cnt0, x.cnt1, x.slot, 0);
}

struct Pieces {
  int split, count, per, total;
  int entry, head, off, left;  // of the piece to come; left: steps (split) or items
  int wave;
  AtRec ahead;                 // its record, loaded under the piece before
  AtRec mine[2];               // few pairs: lane i holds those of pairs i and 32 + i,
  int rank[2];                 // and their places in the sorted order
  __device__ __forceinline__ void init(const AtParams& p) {
    AtFirst f{-1, 0, 0, 0};
    AtPlan pl;
    if (p.few) {
      pl = plan(p, f);
    } else {
      pl = *p.plan;
      if (pl.split) f = p.first[blockIdx.x];
    }
    split = pl.split;
    count = pl.count;
    per = pl.per;
    total = pl.total;
    wave = 0;
    off = head = entry = 0;
    if (split) {
      entry = f.rec;
      head = f.head;
      off = f.off;
      left = f.rec < 0 ? 0 : (int)min((long long)per, total - (long long)blockIdx.x * per);
      if (left > 0) ahead = record(p, entry);
    } else {
      item(p);
    }
  }
  __device__ __forceinline__ AtRec record(const AtParams& p, int e) const {
    if (!p.few) return split ? p.rec[e] : p.sorted[e];
    if (!split) {
      const uint32_t b0 = __ballot_sync(0xffffffffu, rank[0] == e), b1 = __ballot_sync(0xffffffffu, rank[1] == e);
      e = b0 ? __ffs(b0) - 1 : 31 + __ffs(b1);
    }
    AtRec r;
    const int src = e & 31;
    const bool hi = e >= 32;
    auto get = [&](int a, int b) {
      a = __shfl_sync(0xffffffffu, a, src);
      b = __shfl_sync(0xffffffffu, b, src);
      return hi ? b : a;
    };
    r.row0 = get(mine[0].row0, mine[1].row0);
    r.t0 = get(mine[0].t0, mine[1].t0);
    r.T = get(mine[0].T, mine[1].T);
    r.L = get(mine[0].L, mine[1].L);
    r.u = get(mine[0].u, mine[1].u);
    r.steps = get(mine[0].steps, mine[1].steps);
    r.before = get(mine[0].before, mine[1].before);
    r.pad = 0;
    return r;
  }
  // What at_plan_kernel does, for few pairs and by one warp. What the join reads is left where it looks.
  __device__ __forceinline__ AtPlan plan(const AtParams& p, AtFirst& f) {
    const int lane = threadIdx.x & 31, pair = 2 * p.tile_tokens;
    int row0[2], T[2], L[2], first[2], n = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int u = 32 * i + lane;
      row0[i] = T[i] = L[i] = 0;
      first[i] = 0x7fffffff;
      if (32 * i >= p.n) continue;
      if (u < p.n) at_unit(p, u, &row0[i], &T[i], &L[i]);
      const int tiles = (T[i] + pair - 1) / pair, incl = warp_incl_scan(tiles);
      first[i] = u < p.n ? n + incl - tiles : 0x7fffffff;  // the unit's first pair
      n += __shfl_sync(0xffffffffu, incl, 31);
    }
    // (units that overlap could come to more pairs than there is room for)
    if (n > p.room && lane == 0) set_status(p.status, RKV_DEV_BAD_WINDOW);
    n = min(n, p.room);
    int longest = 0, before = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = 32 * i + lane;
      mine[i] = AtRec{};
      if (32 * i >= n) continue;
      int u = 0;  // the last unit whose pairs begin at or before e
#pragma unroll 1
      for (int step = p.n > 32 ? 32 : 16; step && p.n > 1; step >>= 1) {
        const int at = u + step, a = __shfl_sync(0xffffffffu, first[0], at & 31), b = __shfl_sync(0xffffffffu, first[1], at & 31);
        if ((at >= 32 ? b : a) <= e) u = at;
      }
      auto get = [&](const int (&x)[2]) {
        const int a = __shfl_sync(0xffffffffu, x[0], u & 31), b = __shfl_sync(0xffffffffu, x[1], u & 31);
        return u >= 32 ? b : a;
      };
      AtRec& r = mine[i];
      r.u = u;
      r.T = get(T);
      r.L = get(L);
      r.t0 = (e - get(first)) * pair;
      r.row0 = get(row0) + r.t0;
      const int keys = p.mask ? r.L : r.L - r.T + min(r.t0 + pair, r.T);
      r.steps = e < n ? (keys + kAtTile - 1) / kAtTile : 0;
      const int incl = warp_incl_scan(r.steps);
      r.before = before + incl - r.steps;
      before += __shfl_sync(0xffffffffu, incl, 31);
      longest = max(longest, __reduce_max_sync(0xffffffffu, r.steps));
      r.pad = 0;
      if (blockIdx.x == 0 && e < n) p.rec[e] = r;
    }
    const AtPlan pl = at_decide((long long)before * p.n_kv, longest, n, p.ctas);
    if (blockIdx.x == 0 && lane == 0) *p.plan = pl;
    if (pl.split) {
      split = 1;
      const long long a = (long long)blockIdx.x * pl.per;
      if (a < pl.total) {  // the last pair that begins at or before a
        const uint32_t b0 = __ballot_sync(0xffffffffu, lane < n && (long long)mine[0].before * p.n_kv <= a);
        const uint32_t b1 = __ballot_sync(0xffffffffu, 32 + lane < n && (long long)mine[1].before * p.n_kv <= a);
        f.rec = b1 ? 63 - __clz(b1) : 31 - __clz(b0);
        const AtRec r = record(p, f.rec);
        const int x = (int)(a - (long long)r.before * p.n_kv);
        f.head = x / r.steps;
        f.off = x - f.head * r.steps;
      }
      if (lane == 0) p.first[blockIdx.x] = f;
    } else {
      const bool order = (long long)n * p.n_kv > gridDim.x;  // (else all are begun at once)
      int k[2] = {lane, 32 + lane};
      if (order) {
        k[0] = k[1] = 0;
        for (int e = 0; e < n; ++e) {
          const int a = __shfl_sync(0xffffffffu, mine[0].steps, e & 31), b = __shfl_sync(0xffffffffu, mine[1].steps, e & 31);
          const int y = e >= 32 ? b : a;
          k[0] += y > mine[0].steps || (y == mine[0].steps && e < lane);
          k[1] += y > mine[1].steps || (y == mine[1].steps && e < 32 + lane);
        }
      }
      rank[0] = lane < n ? k[0] : -1;
      rank[1] = 32 + lane < n ? k[1] : -1;
    }
    return pl;
  }
  // whole items come in waves of one per CTA, every second wave from the other end
  __device__ __forceinline__ void item(const AtParams& p) {
    const long long i = (long long)wave * gridDim.x + ((wave & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    ++wave;
    left = i < (long long)count * p.n_kv;
    if (left) {
      entry = (int)((uint32_t)i / (uint32_t)p.n_kv);
      head = (int)i - entry * p.n_kv;
      ahead = record(p, entry);
    }
  }
  __device__ __forceinline__ bool next(const AtParams& p, Piece& x) {
    x.steps = 0;
    if (left <= 0) return false;
    const AtRec r = ahead;
    x.row0 = r.row0;
    x.t0 = r.t0;
    x.T = r.T;
    x.L = r.L;
    x.u = r.u;
    x.g = head;
    x.s0 = off;
    int len = r.steps;
    x.slot = -1;
    if (split) {
      len = min(r.steps - off, left);
      x.slot = off > 0 ? 2 * (int)blockIdx.x : len < r.steps ? 2 * (int)blockIdx.x + 1 : -1;
      left -= len;
      off = 0;
      if (++head == p.n_kv) {
        head = 0;
        ++entry;
      }
      if (left > 0) ahead = record(p, entry);
    } else {
      item(p);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = x.t0 + h * p.tile_tokens;  // the tile's first token
      const int keys = p.mask ? x.L : x.L - x.T + min(t + p.tile_tokens, x.T);
      const int all = t < x.T ? (keys + kAtTile - 1) / kAtTile : 0;
      const int cnt = max(0, min(x.s0 + len, all) - x.s0);
      (h ? x.cnt1 : x.cnt0) = cnt;
      x.steps = max(x.steps, cnt);
    }
    return true;
  }
};

// A warpgroup's registers per thread: the first hands back what the others then take (setmaxnreg; the
// shares add up to what the block was launched with, so that no take can wait for ever).
constexpr int kAtLoadRegs = 64, kAtOutRegs = 80, kAtSoftmaxRegs = 184, kAtLaunchRegs = 128;
static_assert(kAtLoadRegs + kAtOutRegs + 2 * kAtSoftmaxRegs <= 4 * kAtLaunchRegs, "");
static_assert(kAtThreads * kAtLaunchRegs == 65536, "");
template <int N>
__device__ __forceinline__ void reg_release() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_take() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Upper halves of the operands' descriptors; the lower ones are the address in units of 16 bytes, and
// bits 16 on. K-major rows of 128 bytes (Q, K): eight rows are 1024 bytes apart. V is the B operand with its
// rows as the reduction and 64 dimensions in 128 bytes: the other 64 are 16 KB further, eight rows 1024 bytes.
constexpr uint32_t kDescHi = (1024u >> 4) | 1u << 14 | 2u << 29;
constexpr uint32_t kDescLoK = 1u << 16, kDescLoV = (16384u >> 4) << 16;
constexpr uint32_t kIdescS = idesc_bf16(kAtRows, kAtTile);
constexpr uint32_t kIdescO = idesc_bf16(kAtRows, kHeadDim) | (1u << 16);  // B is not K-major

// D (+)= A B, both in shared memory.
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t keep) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t}"
      ::"r"(d), "r"(a | kDescLoK), "r"(b | kDescLoK), "n"(kDescHi), "n"(kIdescS), "r"(keep));
}
// D (+)= A B with A (bf16, 128 x 16) in TMEM and B a tile of V.
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t keep) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 y, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n\t}"
      ::"r"(d), "r"(a), "r"(b | kDescLoV), "n"(kDescHi), "n"(kIdescO), "r"(keep));
}
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// A place of the ring, and the parity of its load.
struct Ring {
  int place;
  uint32_t phase;
  __device__ __forceinline__ void step() {
    if (++place == kAtStages) {
      place = 0;
      phase ^= 1u;
    }
  }
};

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
// A whole sector at once; dst begins on 32 bytes.
__device__ __forceinline__ void st_global32(void* dst, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               ::"l"(dst), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
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

// Which keys a row sees: all below `clear` and none from `end` on (the same for every row of a warp); of the
// others those up to `lim`, or in a tree those whose bit is set, T of them from `base` on (T = 0: not a row).
struct AtSees {
  int clear, end, lim, base, T;
  const uint32_t* bits;
};

// Sets the keys that the row does not see to -infinity, in 32 columns from key k on (k + 32 > clear).
template <bool TREE>
__device__ __forceinline__ void at_hide(uint32_t (&s)[32], int k, const AtSees& a) {
  if (TREE) {
    const int d = k - a.base;  // number of the first key among the new ones, above -32 (base is `clear`)
    // bits d .. d + 31 of the row, ones where d is below 0, zeros from T on
    uint32_t sees = 0u;
    if (a.T > 0) {
      const int w = d >> 5, o = d & 31;
      const uint32_t lo = w < 0 ? 0xffffffffu : w * 32 < a.T ? a.bits[w] : 0u;
      const uint32_t hi = (w + 1) * 32 < a.T ? a.bits[w + 1] : 0u;
      sees = o ? (lo >> o) | (hi << (32 - o)) : lo;
      const int end = a.T - d;
      if (end < 32) sees &= end <= 0 ? 0u : (1u << end) - 1u;
    }
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (!((sees >> i) & 1u)) s[i] = 0xff800000u;
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (k + i > a.lim) s[i] = 0xff800000u;
  }
}

// What most steps do not need, in functions of their own, so that the steps' code has neither its branches
// nor its registers (with branches for the masks between the chunks: 8K prompt 440 us).
//
// A step with keys that some row does not see: sets those to -infinity where S lies.
template <bool TREE>
__device__ __noinline__ void at_mask(uint32_t sp, int k0, AtSees sees) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    const int k = k0 + 32 * c;
    if (k + 32 <= sees.clear) continue;
    uint32_t s[32];
    if (k < sees.end) {
      tmem_ld32(sp + 32 * c, s);
      at_hide<TREE>(s, k, sees);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) s[i] = 0xff800000u;
    }
    tmem_st32(sp + 32 * c, s);
  }
  tmem_st_wait();
}

// The maximum of m and the first n scores (32 or 128).
__device__ __noinline__ float at_most(uint32_t sp, int n, float scale, float m) {
#pragma unroll 1
  for (int c = 0; c < n; c += 32) {
    uint32_t s[32];
    tmem_ld32(sp + c, s);
    float y[4] = {kNoMax, kNoMax, kNoMax, kNoMax};
#pragma unroll
    for (int i = 0; i < 32; i += 2)
      y[(i >> 1) & 3] = max3(y[(i >> 1) & 3], __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
    m = fmaxf(m, fmaxf(max3(y[0], y[1], y[2]), y[3]) * scale);
  }
  return m;
}

// Scales O by f. (The product before this step's S is done: S was issued behind it.)
__device__ __noinline__ void at_scale(uint32_t o, float f) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t s[32];
    tmem_ld32(o + 32 * c, s);
#pragma unroll
    for (int i = 0; i < 32; ++i) s[i] = __float_as_uint(__uint_as_float(s[i]) * f);
    tmem_st32(o + 32 * c, s);
  }
  tmem_st_wait();
}

// A row of O to where it goes, in stores of 16 bytes: for outputs or a workspace that begin on 16 bytes, which is all
// that the call asks for, and not on the 32 that a store of a sector does (packed prompts 213 us by sectors, 223 in
// halves; 64 drafted tokens over 131071 rows 118 and 121). Out of the way of the usual code: as a branch at each store
// it cost the packed prompts 4 us.
__device__ __noinline__ void at_write16(uint32_t od, bool valid, float* part, bf16* dst, bool none, float f) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t o[32];
    tmem_ld32(od + 32 * c, o);
    if (valid && part) {
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
}

struct AtBars {
  uint64_t full[kAtStages], empty[kAtStages];  // the ring of K and V tiles
  uint64_t qfull[2], qempty[2];
  uint64_t sfull[2];   // S of a step is there (and all products before it are done)
  uint64_t pfull[2];   // P of a step is written
  uint64_t ofull[2];   // the item's last product is done
  uint64_t ofree[2];   // O has been read
  uint64_t lfull[2][2];  // a tile's sums are there (by turns)
  uint64_t dirty, clean;      // a V tile with rows behind the last is next; they are zeros
  uint64_t pfilled[kAtPieces], pread[kAtPieces];  // pieces
  uint64_t turn[2];    // a tile's turn to issue
  uint64_t drain[2];   // everything a warp issued is done (after a wait gave up)
  uint32_t tmem;
};
static_assert(sizeof(AtBars) <= 512, "");

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
      mbar_init(&bar.empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.qfull[i], 1);
      mbar_init(&bar.qempty[i], 1);
      mbar_init(&bar.sfull[i], 1);
      mbar_init(&bar.pfull[i], 4);
      mbar_init(&bar.ofull[i], 1);
      mbar_init(&bar.ofree[i], 4);
      mbar_init(&bar.lfull[i][0], 4);
      mbar_init(&bar.lfull[i][1], 4);
      mbar_init(&bar.drain[i], 1);
      mbar_init(&bar.turn[i], 1);
    }
    for (int i = 0; i < kAtPieces; ++i) {
      mbar_init(&bar.pfilled[i], 1);
      mbar_init(&bar.pread[i], kAtReaders);
    }
    mbar_init(&bar.dirty, 2);
    mbar_init(&bar.clean, 1);
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
  const WaitLimit limit = p.wait_limit, item_limit = p.item_limit;
  bool aborted = false;
  Piece* pieces = reinterpret_cast<Piece*>(smem + AtSmem::piece_off);
  float* sums = reinterpret_cast<float*>(smem + AtSmem::sum_off);
  Piece x{};
  uint32_t npiece = 0;
  auto next = [&]() {  // the next piece, for a warp other than the one that finds them
    const uint32_t i = npiece % kAtPieces;
    if (!mbar_wait_warp(&bar.pfilled[i], (npiece / kAtPieces) & 1u, item_limit)) {
      aborted = true;
      return false;
    }
    read_piece(x, pieces + i);
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar.pread[i]);
    ++npiece;
    return x.steps > 0;
  };

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
          const int copies = min(kAtTile / rows, (x.L - k0 + rows - 1) / rows);
          if (lane == 0) mbar_arrive_expect_tx(&bar.full[s], (uint32_t)(copies * rows * 256));
          __syncwarp();
          for (int c = lane; c < copies; c += 32) {
            const int t = k0 + c * rows;
            const int b = c == lane ? blk : paged_block(p.pm, x.u, t, p.status);
            const int y = (b * p.n_kv + x.g) * p.pm.block + (t & (p.pm.block - 1));
            tma_load_2d(dst + c * rows * 128, map, 0, y, &bar.full[s]);
            tma_load_2d(dst + 16384 + c * rows * 128, map, 64, y, &bar.full[s]);
          }
        } else if (lane == 0) {
          const int y = (x.u * p.n_kv + x.g) * p.cap + k0;
          mbar_arrive_expect_tx(&bar.full[s], kAtTileBytes);
          tma_load_2d(dst, map, 0, y, &bar.full[s]);
          tma_load_2d(dst + 16384, map, 64, y, &bar.full[s]);
        }
        __syncwarp();
      };
      while (!aborted && next()) {
        for (int j = 0; j < x.steps && !aborted; ++j) {
          const int k0 = (x.s0 + j) * kAtTile;
          int blk = 0;
          if (PAGED && k0 + lane * rows < x.L && lane * rows < kAtTile)
            blk = paged_block(p.pm, x.u, k0 + lane * rows, p.status);
          int s = slot();
          if (s < 0) break;
          if (!(skip == RKV_TESTING_ATTENTION_KEYS && ld == 0)) tile(&kmap, s, k0, blk);
          ++ld;
          if (j == 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (aborted || x.cnt(h) == 0) continue;
              if (nq[h] > 0 && !mbar_wait_warp(&bar.qempty[h], (uint32_t)((nq[h] - 1) & 1), limit)) {
                aborted = true;
                continue;
              }
              if (lane == 0 && !(skip == RKV_TESTING_ATTENTION_QUERIES && nq[h] == 0)) {
                uint8_t* dst = qs + (size_t)h * kAtTileBytes;
                mbar_arrive_expect_tx(&bar.qfull[h], qbytes);
                for (int c = 0; c < 2; ++c)
                  tma_load_3d(dst + c * 16384, &qmap, 64 * c, x.g * p.gqa,
                              x.row0 + h * p.tile_tokens, &bar.qfull[h]);
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
    } else if (warp < 3) {
      // ------------------------------------------------------------------ products of a tile
      // A warp for each tile of the pair: one waits while the other issues (one warp for both left the tensor
      // cores idle between its waits: 8K prompt 425 us). The whole warp follows the steps and one lane issues, so
      // that descriptors are uniform values, a constant away from those of a place of the ring (with one lane
      // computing them for itself: 510 us).
      const int h = warp - 1;
      const uint32_t ring_lo = (smem_addr(ring) & 0x3FFFFu) >> 4;
      const uint32_t q_lo = ((smem_addr(qs) & 0x3FFFFu) >> 4) + h * (kAtTileBytes >> 4);
      const uint32_t st = tmem + h * 128, ot = st + 256;
      uint32_t nq = 0, np = 0, no = 0, nclean = 0;
      Ring kr{0, 0}, vr{0, 0}, at{0, 0};  // K tile of the step, V tile of the product to come, next load
      auto wait = [&](uint64_t* b, uint32_t parity) {
        if (!aborted && !mbar_wait_warp(b, parity & 1u, limit)) aborted = true;
      };
      // A step's scores are issued behind the product of the step before, which they follow in the tensor
      // cores. The tiles take turns with that: products of both at once would end together, and then both
      // softmaxes would run while the tensor cores wait (8K prompt 496 us). The turn passes on two products
      // before the last, which hides its way to the other warp.
      bool pend = false, first = false, last = false, tail = false;
      uint32_t nturn = 0;
      auto product = [&](bool pass) {  // O += P V
        const uint32_t b = ring_lo + vr.place * (kAtTileBytes >> 4), keep = first ? 0u : 1u;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          umma_ts(ot, st + 8 * kk, b + kk * (2048 >> 4), kk ? 1u : keep);
          if (kk == 5 && pass) mbar_arrive(&bar.turn[h ^ 1]);
        }
        if (last) umma_commit(&bar.ofull[h]);
      };
      auto scores = [&](bool end) {  // S = Q K^T
        const uint32_t b = ring_lo + kr.place * (kAtTileBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = (uint32_t)((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
          umma_ss(st, q_lo + off, b + off, kk > 0);
          if (kk == 5) mbar_arrive(&bar.turn[h ^ 1]);
        }
        umma_commit(&bar.sfull[h]);
        if (end) umma_commit(&bar.qempty[h]);
      };
      auto ready = [&]() {  // what the product to come needs
        wait(&bar.full[vr.place], vr.phase);
        if (tail) wait(&bar.clean, nclean++);
        if (first && no > 0) wait(&bar.ofree[h], no - 1);
        wait(&bar.pfull[h], np++);
        if (last) ++no;
      };
      while (!aborted && next()) {
        for (int j = 0; j < x.steps && !aborted; ++j) {
          const bool act = j < x.cnt(h), end = j == x.cnt(h) - 1;
          kr = at;
          at.step();
          if (act && j == 0) wait(&bar.qfull[h], nq++);
          wait(&bar.full[kr.place], kr.phase);
          if (h == 1 || nturn > 0) wait(&bar.turn[h], h == 1 ? nturn : nturn - 1);
          ++nturn;
          if (pend) ready();
          tc_fence_after();
          if (!aborted && elect_one()) {
            if (pend) product(!act);
            if (act) {
              scores(end);
            } else {  // a step that the tile has no part in
              if (!pend) mbar_arrive(&bar.turn[h ^ 1]);
              mbar_arrive(&bar.empty[kr.place]);
            }
          }
          __syncwarp();
          pend = act;
          first = j == 0;
          last = end;
          vr = at;
          at.step();
          tail = (x.s0 + j + 1) * kAtTile > x.L;
          if (tail && lane == 0) mbar_arrive(&bar.dirty);
          if (!act) {
            wait(&bar.full[vr.place], vr.phase);
            if (tail) wait(&bar.clean, nclean++);
            if (!aborted && lane == 0) mbar_arrive(&bar.empty[vr.place]);
            __syncwarp();
          }
        }
      }
      if (!aborted && pend) {
        ready();
        tc_fence_after();
        if (!aborted && elect_one()) product(false);
        __syncwarp();
      }
      if (aborted) {
        if (lane == 0) set_status(p.status, RKV_DEV_WAIT_TIMEOUT);
        // let issued products end (a commit is about those of its own lane)
        if (elect_one()) umma_commit(&bar.drain[h]);
        __syncwarp();
        mbar_wait_warp(&bar.drain[h], 0u, drain_limit(limit));
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------------ pieces, rows behind the last
      Pieces it;
      it.init(p);
      auto find = [&](uint32_t k) {  // piece k; false: there is none
        const uint32_t i = k % kAtPieces;
        if (k >= kAtPieces && !mbar_wait_warp(&bar.pread[i], (k / kAtPieces - 1) & 1u, item_limit)) {
          aborted = true;
          return false;
        }
        Piece y{};
        const bool any = it.next(p, y);
        if (lane == 0) {
          write_piece(pieces + i, y);
          mbar_arrive(&bar.pfilled[i]);
        }
        __syncwarp();
        return any;
      };
      // p is 0 for keys behind the last, but 0 times what the cache may hold there (infinity, NaN) is not. The
      // tile's place in the ring is its own from when its step's scores are issued (they are behind all products
      // that used the place) until its product, so the wait for its load cannot be taken for another one's.
      int steps = 0, ntail = 0;
      uint32_t found = 0;
      bool more = true;
      for (uint32_t k = 0; !aborted; ++k) {
        while (more && found <= k + 2 && !aborted) more = find(found++);
        if (aborted) break;
        // (its own reading of a piece: no other warp writes them)
        read_piece(x, pieces + k % kAtPieces);
        __syncwarp();
        if (x.steps == 0) break;
        const int at = x.L / kAtTile - x.s0, cut = x.L % kAtTile;  // the step that the sequence ends in
        if (cut && at >= 0 && at < x.steps) {
          const int load = 2 * (steps + at) + 1, s = load % kAtStages;
          if (!mbar_wait_warp(&bar.dirty, (uint32_t)(ntail++ & 1), item_limit) ||
              !mbar_wait_warp(&bar.full[s], (uint32_t)((load / kAtStages) & 1), limit)) {
            aborted = true;
            break;
          }
          uint4* v = reinterpret_cast<uint4*>(ring + (size_t)s * kAtTileBytes + cut * 128);
          for (int i = lane; i < (kAtTile - cut) * 8; i += 32)
            v[i] = v[i + 16384 / 16] = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.clean);
        }
        steps += x.steps;
      }
    }
  } else if (warp < 8) {
    reg_release<kAtOutRegs>();
    // ------------------------------------------------------------------ outputs
    // While the softmax warps are at the next item. A row's sum comes in one of two places, by turns.
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const int tok = row / p.gqa, head = row - tok * p.gqa;
    uint32_t no[2] = {0, 0};
    int steps = 0;
    while (!aborted && next()) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (aborted || x.cnt(h) == 0) continue;
        const int t = x.t0 + h * p.tile_tokens + tok;  // this row's token
        const bool valid = tok < p.tile_tokens && t < x.T;
        const uint32_t turn = no[h] & 1;
        if (!mbar_wait_warp(&bar.ofull[h], turn, item_limit) ||
            !mbar_wait_warp(&bar.lfull[h][turn], (no[h] >> 1) & 1u, limit)) {
          aborted = true;
          continue;
        }
        ++no[h];
        if (row == 0) mbar_arrive(&bar.empty[(2 * (steps + x.cnt(h) - 1) + 1) % kAtStages]);  // the last V tile
        __syncwarp();
        tc_fence_after();
        const float l = sums[turn * 256 + h * 128 + row];
        const bool none = l == 0.f;  // the row sees nothing: zeros, whatever v holds
        const float f = l > 0.f ? 1.f / l : l;
        const uint32_t od = tmem + ((uint32_t)(quarter * 32) << 16) + 256 + h * 128;
        bf16* dst = p.out + ((size_t)(x.row0 + h * p.tile_tokens + tok) * p.hq + x.g * p.gqa + head) * kHeadDim;
        float* part = p.part_o + ((size_t)max(x.slot, 0) * p.part_rows + h * 128 + row) * kHeadDim;
        if (!__any_sync(0xffffffffu, valid)) {
        } else if (!p.whole) {
          at_write16(od, valid, x.slot >= 0 ? part : nullptr, dst, none, f);
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            tmem_ld32(od + 32 * c, o);
            if (valid && x.slot >= 0) {
#pragma unroll
              for (int i = 0; i < 32; i += 8) st_global32(part + 32 * c + i, o + i);
            } else if (valid) {
#pragma unroll
              for (int i = 0; i < 32; i += 16) {
                uint32_t w[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  w[k] = none ? 0u : pack_bf16x2(__uint_as_float(o[i + 2 * k]) * f, __uint_as_float(o[i + 2 * k + 1]) * f);
                st_global32(dst + 32 * c + i, w);
              }
            }
            __syncwarp();
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.ofree[h]);
      }
      steps += x.steps;
    }
    if (aborted && lane == 0) set_status(p.status, RKV_DEV_WAIT_TIMEOUT);
  } else {
    reg_take<kAtSoftmaxRegs>();
    // ------------------------------------------------------------------ softmax of a tile
    const int h = (warp >> 2) - 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t sp = tmem + lanes + h * 128, od = tmem + lanes + 256 + h * 128;
    const uint64_t scale2 = pack2(p.scale_log2, p.scale_log2);
    const int tok = row / p.gqa;
    uint32_t ns = 0, no = 0;  // waits for S; items
    Ring at{0, 0};            // the step's K tile
    int vplace = 0;           // the V tile of the step before
    while (!aborted && next()) {
      const int t = x.t0 + h * p.tile_tokens + tok;  // this row's token
      const bool valid = tok < p.tile_tokens && t < x.T;
      const int base = x.L - x.T;
      const int lim = valid ? base + t : -1;  // last key of a causal row
      const bool idle = !__any_sync(0xffffffffu, valid);
      // keys below `clear` are seen by every row of the warp that is one
      const int clear = TREE ? base : __reduce_min_sync(0xffffffffu, valid ? lim : 0x7ffffffe) + 1;
      const uint32_t* bits = TREE ? p.mask + (size_t)(x.row0 + h * p.tile_tokens + tok) * p.words : nullptr;
      float m = kNoMax, l = 0.f;
      const int end = TREE ? x.L : __reduce_max_sync(0xffffffffu, lim) + 1;
      const AtSees sees{clear, end, lim, base, valid ? x.T : 0, bits};
      for (int j = 0; j < x.cnt(h); ++j) {
        // (an item that this tile has no part in is over for it at once, and it waits here while the other tile is at it)
        if (!mbar_wait_warp(&bar.sfull[h], ns++ & 1u, j ? limit : item_limit)) {
          aborted = true;
          break;
        }
        // This S is done, and the product before it: their tiles' places are free. (A commit for each cost the
        // issuing warp 50 clocks.)
        if (row == 0) {
          mbar_arrive(&bar.empty[at.place]);
          if (j > 0) mbar_arrive(&bar.empty[vplace]);
        }
        __syncwarp();
        at.step();
        vplace = at.place;
        at.step();
        if (idle) {
          if (lane == 0) mbar_arrive(&bar.pfull[h]);
          continue;
        }
        tc_fence_after();
        const int k0 = (x.s0 + j) * kAtTile;
        if (k0 + kAtTile > clear) at_mask<TREE>(sp, k0, sees);
        if (j == 0) m = at_most(sp, 32, p.scale_log2, m);  // (near enough: what passes it by far raises it)
        uint32_t out[2][32];
        float sum;
#pragma unroll 1
        for (bool again = false;; again = true) {
          // numerators relative to m, which most often holds: no maximum is looked for. A chunk's load runs
          // under the one before it.
          const uint64_t off = pack2(-m, -m);
          uint64_t acc[2] = {0ull, 0ull};
          uint32_t s[2][32];
          tmem_ld32_start(sp, s[0]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_ld_wait(s[c & 1]);
            if (c < 3) tmem_ld32_start(sp + 32 * (c + 1), s[(c + 1) & 1]);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 y = unpack2(fma2(pack2(__uint_as_float(s[c & 1][2 * i]), __uint_as_float(s[c & 1][2 * i + 1])),
                                            scale2, off));
              const float e0 = fast_exp2(y.x), e1 = fast_exp2(y.y);
              acc[i & 1] = add2(acc[i & 1], pack2(e0, e1));
              out[c >> 1][16 * (c & 1) + i] = pack_bf16x2(e0, e1);
            }
          }
          const float2 z = unpack2(add2(acc[0], acc[1]));
          sum = z.x + z.y;
          if (again || !__any_sync(0xffffffffu, valid && !(sum < kLargest))) break;
          const float to = at_most(sp, kAtTile, p.scale_log2, m), f = fast_exp2(m - to);
          if (j > 0) at_scale(od, f);
          l *= f;
          m = to;
        }
        tmem_st32(sp, out[0]);
        tmem_st32(sp + 32, out[1]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.pfull[h]);
        l += sum;
      }
      if (aborted) break;
      for (int j = x.cnt(h); j < x.steps; ++j) {  // steps of the other tile alone
        at.step();
        at.step();
      }
      if (x.slot >= 0 && valid)  // (l = 0: a part that the tile has no steps in, or that the row sees nothing of)
        p.part_ml[(size_t)x.slot * p.part_rows + h * 128 + row] = make_float2(m, l);
      if (x.cnt(h) > 0) {
        sums[(no & 1) * 256 + h * 128 + row] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.lfull[h][no & 1]);
        ++no;
      }
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

// Joins the parts of the items that ranges cut. Work: the borders of the ranges x groups of rows; of a cut item,
// the first border in it does all (a warp per row, four columns a lane). A lane holds a part's weight, so that
// the parts' loads do not wait for one another. What this waits for is a chain of three loads a row, so warps
// count: 64 an SM (chunks of 3 prompts 189 us; 32 with four rows each 203). Blocks go over the work themselves:
// with one for each group, a call that cuts nothing waited 9 us for them to end.
constexpr int kJoinWarps = 16, kJoinPerSm = 4, kJoinAhead = 2;

__global__ void __launch_bounds__(32 * kJoinWarps, kJoinPerSm) at_join_kernel(AtParams p) {
  pdl_wait();
  const AtPlan pl = *p.plan;
  if (!pl.split) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, borders = p.ctas - 1;
  const int groups = (p.part_rows + kJoinWarps - 1) / kJoinWarps;
  for (int work = blockIdx.x; work < borders * groups; work += gridDim.x) {
    const int y = work / borders, c = work - y * borders + 1;
    const AtFirst f = p.first[c];
    if (f.rec < 0 || f.off == 0) continue;
    const long long a = (long long)c * pl.per - f.off;
    const int c0 = (int)(a / pl.per);
    if (c0 != c - 1) continue;
    const AtRec r = p.rec[f.rec];
    const int parts = (int)((a + r.steps - 1) / pl.per) - c0 + 1;
    const int row = y * kJoinWarps + warp, t = (row & 127) / p.gqa, tok = (row >> 7) * p.tile_tokens + t;
    if (t >= p.tile_tokens || r.t0 + tok >= r.T) continue;
    auto at = [&](int i) { return (size_t)(i ? 2 * (c0 + i) : 2 * c0 + 1) * p.part_rows + row; };
    float m = kNoMax, l = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < parts; i0 += 32) {
      const int n = min(32, parts - i0);
      const float2 x = lane < n ? p.part_ml[at(i0 + lane)] : make_float2(kNoMax, 0.f);
      // (a part without a visible key has the sum 0, and its outputs are not looked at)
      float to = x.y == 0.f ? kNoMax : x.x;
#pragma unroll
      for (int b = 16; b; b >>= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, b));
      to = fmaxf(to, m);
      const float w = x.y == 0.f ? 0.f : fast_exp2(x.x - to), f0 = fast_exp2(m - to);
      float s = w * x.y;
#pragma unroll
      for (int b = 16; b; b >>= 1) s += __shfl_xor_sync(0xffffffffu, s, b);
      m = to;
      l = l * f0 + s;
      o.x *= f0;
      o.y *= f0;
      o.z *= f0;
      o.w *= f0;
      for (int i = 0; i < n; i += kJoinAhead) {
        float4 v[kJoinAhead];
        float wi[kJoinAhead];
#pragma unroll
        for (int q = 0; q < kJoinAhead; ++q) {
          wi[q] = __shfl_sync(0xffffffffu, w, min(i + q, 31));
          if (i + q >= n) wi[q] = 0.f;
          if (wi[q] != 0.f) v[q] = *reinterpret_cast<const float4*>(p.part_o + at(i0 + i + q) * kHeadDim + 4 * lane);
        }
#pragma unroll
        for (int q = 0; q < kJoinAhead; ++q) {
          if (wi[q] == 0.f) continue;
          o.x += v[q].x * wi[q];
          o.y += v[q].y * wi[q];
          o.z += v[q].z * wi[q];
          o.w += v[q].w * wi[q];
        }
      }
    }
    const float s = l > 0.f ? 1.f / l : l;
    bf16* dst = p.out + ((size_t)(r.row0 + tok) * p.hq + f.head * p.gqa + (row & 127) - t * p.gqa) * kHeadDim;
    *reinterpret_cast<uint2*>(dst + 4 * lane) =
        make_uint2(pack_bf16x2(o.x * s, o.y * s), pack_bf16x2(o.z * s, o.w * s));
  }
}

// ------------------------------------------------------------------------------------------
// host side
// ------------------------------------------------------------------------------------------
struct AtSizes {
  size_t plan, first, rec, unit, ml, o;
  int room, part_rows;
};

static AtSizes at_sizes(int n, int gqa, int tokens) {
  AtSizes z;
  const int pair = 2 * (kAtRows / gqa), ctas = device_sm_count();
  z.room = tokens / pair + n;
  z.plan = 256;
  z.first = align_up((size_t)ctas * sizeof(AtFirst), 256);
  z.rec = align_up((size_t)z.room * sizeof(AtRec), 256);
  z.unit = align_up((size_t)(n + 1) * 4, 256);
  z.part_rows = tokens <= kAtRows / gqa ? tokens * gqa : 2 * kAtRows;
  z.ml = align_up((size_t)2 * ctas * z.part_rows * sizeof(float2), 256);
  z.o = (size_t)2 * ctas * z.part_rows * kHeadDim * 4;
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
  static std::atomic<bool> regs_ok{false};  // (kept once it has been seen: an error of one call is not the next one's)
  if (!regs_ok.load(std::memory_order_relaxed)) {
    cudaFuncAttributes f;
    const cudaError_t seen = cudaFuncGetAttributes(&f, (const void*)at_kernel<PAGED, TREE>);
    if (seen != cudaSuccess) return seen;
    if (f.numRegs != kAtLaunchRegs) return cudaErrorInvalidConfiguration;
    regs_ok.store(true, std::memory_order_relaxed);
  }
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
  p.part_rows = z.part_rows;
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
  p.whole = (reinterpret_cast<uintptr_t>(p.out) | reinterpret_cast<uintptr_t>(p.part_o)) % 32 == 0;
  p.status = a.status;
  p.wait_limit = a.wait_limit_ns ? WaitLimit{a.wait_limit_ns} : kWaitLimit;
  // (a step takes some 2 us)
  p.item_limit = WaitLimit{p.wait_limit.ns + 20000ull * (uint64_t)((a.cap + kAtTile - 1) / kAtTile)};
  p.test_skip = a.test_skip;
  p.few = z.room <= kFewPairs;
  cudaError_t e = cudaSuccess;
  if (!p.few) e = launch_pdl_kernel(at_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, p);
  if (e != cudaSuccess) return e;
  if (p.mask)
    e = paged ? launch_at<true, true>(qm, km, vm, p, s) : launch_at<false, true>(qm, km, vm, p, s);
  else
    e = paged ? launch_at<true, false>(qm, km, vm, p, s) : launch_at<false, false>(qm, km, vm, p, s);
  // (items of so few steps are never cut)
  if (e != cudaSuccess || p.ctas < 2 || (a.cap + kAtTile - 1) / kAtTile < kSplitGain) return e;
  return launch_pdl_kernel(at_join_kernel, dim3(p.ctas * kJoinPerSm), dim3(32 * kJoinWarps), 0, s, p);
}

}  // namespace rkv
