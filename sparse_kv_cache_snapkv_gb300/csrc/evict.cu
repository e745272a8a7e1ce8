// Eviction by accumulated attention weight (sm_103a), in place.
//
// Per (unit, KV head) with L > keep rows: a row's key is the order-preserving integer of its
// weight, or the largest integer when its position is among the last `recent`. The keep-th largest
// key T and the number of keys equal to T that are still kept (the lowest rows) come from an
// MSB-first radix select; then the free rows below keep and the kept rows at or past keep, equally
// many, are listed in ascending order and paired. Sources lie at or past keep and destinations
// below it, so all moves are independent.
//
// What it has to move is little (8 bytes a row read, up to 8 written, 2 rows per move: 256 units of 4352
// rows 12 us, 32 of up to 32K in 4 bits 5 us at the copy rate); what bounds it is the chain of barriers of
// the select, so the select makes few passes, all of them over shared memory, by as many CTAs as there are
// SMs: 26 us and 32 us.
#include <cuda_runtime.h>
#include <cstdint>

#include "common.cuh"
#include "rkv_internal.h"
#include "tensor_core.cuh"

namespace rkv {

constexpr int kEvThreads = 1024;
constexpr int kEvMoveThreads = 256;
constexpr int kEvMoveWarps = kEvMoveThreads / 32;
// Up to this many rows' keys stay in a CTA's shared memory through the select; a unit that needs more
// than kEvMaxCluster CTAs for them has them made again from the weights for each pass.
constexpr int kEvSmemRows = 40960;
constexpr int kEvMaxCluster = 8;
constexpr int kEvClusterMost = 32736;  // rows of a cluster's CTA: two counts of them are one 32-bit sum
// A cluster grows while its CTAs have this many rows each (8 units of 8192 rows: 2048 16.9 us, 1024
// 19.0, 4096 17.5; 16 of 4352: 15.2, 15.6, 16.0, and 28.2 with 512).
constexpr int kEvClusterRows = 2048;
// up to this many rows, their weights and positions too (256 units of 4352 rows: 26 us, not held 32)
constexpr int kEvHeldRows = 8192;
constexpr int kEvBins = 2048;

// free rows and kept rows past keep of one (unit, KV head); at most `most` of each
static inline int most_moves(int cap, int keep) {
  const int past = cap > keep ? cap - keep : 0;
  return past < keep ? past : keep;
}

struct EvictLists {
  int32_t* count;  // [n*n_kv]
  int32_t* dst;    // [n*n_kv][most]
  int32_t* src;    // [n*n_kv][most]
  int most;
};

static EvictLists lists_of(const EvictArgs& a) {
  EvictLists l;
  const size_t units = (size_t)a.n * a.n_kv;
  l.most = most_moves(a.cap, a.keep);
  l.count = static_cast<int32_t*>(a.scratch);
  l.dst = l.count + align_up(units * 4, 256) / 4;
  l.src = l.dst + align_up(units * l.most * 4, 256) / 4;
  return l;
}

// Room for every call of no larger sizes, so that a workspace for the largest shape serves all: there
// are most moves where half of the rows are kept.
size_t evict_scratch_bytes(int n, int n_kv, int cap, int keep) {
  const size_t units = (size_t)n * n_kv, most = cap / 2 < keep ? cap / 2 : keep;
  return align_up(units * 4, 256) + 2 * align_up(units * most * 4, 256);
}

struct EvSmem {
  uint32_t hist[256];
  unsigned long long tmp[33];
  int digit, above, in_bin;
  int base[2];
};

// Order-preserving key of a weight. NaN is above every number and below a protected row.
__device__ __forceinline__ uint32_t weight_key(float w) {
  return w != w ? 0xfffffffeu : ordered_key(w);
}

// What a CTA needs of its (unit, KV head).
struct EvUnit {
  const float* w;
  const int32_t* pos;
  float* wo;
  int32_t* po;
  int32_t* from;
  int L, keep, seen;
  long long recent_from;
  __device__ __forceinline__ int position(int i) const {
    const int p = pos[i];
    return p >= 0 ? p : seen - (L - i);
  }
  // (64-bit: the positions and `seen` are the caller's, their difference may be anything)
  __device__ __forceinline__ uint32_t key(int i) const {
    return (long long)position(i) >= recent_from ? 0xffffffffu : weight_key(w[i]);
  }
};

// The unit's arrays; false when there is nothing to evict (then everything has been done, by the
// unit's `nt` threads, of which this is the tid-th).
__device__ __forceinline__ bool evict_unit(const EvictArgs& a, int ukv, EvUnit* x, int tid, int nt) {
  const int u = ukv / a.n_kv;
  const size_t row0 = (size_t)ukv * a.cap;
  x->L = a.len[u];
  x->keep = a.keep;
  x->w = a.weights + row0;
  x->pos = a.pos + row0;
  x->wo = a.weights_out + row0;
  x->po = a.pos_out + row0;
  x->from = a.src_rows ? a.src_rows + (size_t)ukv * a.keep : nullptr;
  if (x->L < 0 || x->L > a.cap) {
    if (tid == 0) set_status(a.status, RKV_DEV_LEN_OVER_CAP);
    return false;
  }
  if (x->L <= a.keep) {
    for (int i = tid; i < x->L; i += nt) {
      x->wo[i] = x->w[i];
      x->po[i] = x->pos[i];
    }
    if (x->from)
      for (int i = tid; i < a.keep; i += nt) x->from[i] = i < x->L ? i : -1;
    return false;
  }
  x->seen = a.seen[u];
  x->recent_from = (long long)x->seen - a.recent;
  return true;
}

// Moved rows' weights and positions, and the reset of the rows past keep (after a barrier, with the
// lists written). weight_of, position_of: of a row as it was.
template <typename W, typename P>
__device__ __forceinline__ void evict_finish(const EvUnit& x, const int32_t* dst, const int32_t* src,
                                             int moves, W weight_of, P position_of) {
  const int tid = threadIdx.x, nt = blockDim.x;
  for (int m = tid; m < moves; m += nt) {
    const int d = dst[m], s = src[m];
    const int p = position_of(s);
    const float w = weight_of(s);
    x.wo[d] = w;
    x.po[d] = p;
    if (x.from) x.from[d] = s;
  }
  __syncthreads();
  for (int i = x.keep + tid; i < x.L; i += nt) {
    x.wo[i] = 0.f;
    x.po[i] = -1;
  }
}

// Copies moved rows: one warp takes kB rows at a time, its lanes the 16-byte words of a row of every
// array (bf16: 16 + 16; 4 bits: 4 + 4, and the scales' 8 + 8 bytes as one word each).
template <int kB>
__device__ __forceinline__ void move_rows(const EvictArgs& a, int ukv, const int32_t* dst,
                                          const int32_t* src, int first, int step, int count) {
  const int lane = threadIdx.x & 31;
  const bool bf = a.row_bytes[2] == 0;
  // bf16: a lane's word is fixed; 4 bits: 10 lanes a row, three rows side by side
  const int sub = bf ? 0 : lane / 10, l = bf ? lane : lane % 10;
  const int side = bf ? 1 : 3;
  int arr, off;
  bool eight = false;
  if (bf) {
    arr = l >> 4;
    off = 16 * (l & 15);
  } else if (l < 8) {
    arr = l >> 2;
    off = 16 * (l & 3);
  } else {
    arr = l - 6;
    off = 0;
    eight = true;
  }
  if (sub >= side) return;  // (two lanes idle)
  uint8_t* base = a.rows[arr] + (size_t)ukv * a.cap * a.row_bytes[arr] + off;
  const int rb = a.row_bytes[arr];
  for (int m0 = first * kB * side; m0 < count; m0 += step * kB * side) {
    uint4 v[kB];
#pragma unroll
    for (int k = 0; k < kB; ++k) {
      const int m = m0 + k * side + sub;
      if (m < count) {
        const uint8_t* p = base + (size_t)src[m] * rb;
        if (eight) {
          const uint2 y = *reinterpret_cast<const uint2*>(p);
          v[k] = make_uint4(y.x, y.y, 0u, 0u);
        } else {
          v[k] = *reinterpret_cast<const uint4*>(p);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kB; ++k) {
      const int m = m0 + k * side + sub;
      if (m < count) {
        uint8_t* p = base + (size_t)dst[m] * rb;
        if (eight)
          *reinterpret_cast<uint2*>(p) = make_uint2(v[k].x, v[k].y);
        else
          *reinterpret_cast<uint4*>(p) = v[k];
      }
    }
  }
}

__device__ __forceinline__ void evict_length(const EvictArgs& a, int u) {
  const int L = a.len[u];
  a.len_out[u] = (L >= 0 && L <= a.cap) ? min(L, a.keep) : L;
}

// Whether no input is the lengths' output.
__host__ __device__ __forceinline__ bool lengths_apart(const EvictArgs& a) {
  return a.len_out != a.len && a.len_out != a.seen;
}

// Lengths that are inputs too move on after every reader.
__global__ void evict_length_kernel(EvictArgs a) {
  pdl_wait();
  pdl_trigger();
  const int u = blockIdx.x * blockDim.x + threadIdx.x;
  if (u < a.n) evict_length(a, u);
}

struct EvDigit {
  int wsum[32];
  int digit, above, in_bin;
};

// Finds the bin of the `remaining`-th largest key in a histogram of kEvBins counts.
__device__ __forceinline__ void find_digit(const uint32_t* hist, int remaining, EvDigit& d) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
  const int per = kEvBins / nt;  // 2 or 4 bins per thread, from the top
  int mine = 0;
  for (int j = 0; j < per; ++j) mine += (int)hist[kEvBins - 1 - tid * per - j];
  const int incl_w = warp_incl_scan(mine);
  if (lane == 31) d.wsum[warp] = incl_w;
  __syncthreads();
  int before = 0;
  const int ws = lane < nw ? d.wsum[lane] : 0;
  const int wi = warp_incl_scan(ws);
  before = __shfl_sync(0xffffffffu, wi - ws, warp);
  int acc = before + incl_w - mine;
  if (acc < remaining && acc + mine >= remaining) {
    for (int j = 0; j < per; ++j) {
      const int b = kEvBins - 1 - tid * per - j, c = (int)hist[b];
      if (acc + c >= remaining) {
        d.digit = b;
        d.above = acc;
        d.in_bin = c;
        break;
      }
      acc += c;
    }
  }
  __syncthreads();
}

// Exclusive prefix sums of cnt[0..n) in place (packed counters that do not overflow); returns the sum.
__device__ __forceinline__ uint32_t scan_counts(uint32_t* cnt, int n, uint32_t* tmp) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nt >> 5;
  const int per = (n + nt - 1) / nt;
  const int b = min(n, tid * per), e = min(n, b + per);
  uint32_t mine = 0;
  for (int i = b; i < e; ++i) mine += cnt[i];
  const uint32_t incl = (uint32_t)warp_incl_scan((int)mine);
  if (lane == 31) tmp[warp] = incl;
  __syncthreads();
  const uint32_t ws = lane < nw ? tmp[lane] : 0u;
  const uint32_t wi = (uint32_t)warp_incl_scan((int)ws);
  uint32_t at = __shfl_sync(0xffffffffu, wi - ws, warp) + incl - mine;
  const uint32_t total = __shfl_sync(0xffffffffu, wi, 31);
  for (int i = b; i < e; ++i) {
    const uint32_t c = cnt[i];
    cnt[i] = at;
    at += c;
  }
  __syncthreads();
  return total;
}

// One CTA per (unit, KV head), keys in shared memory: three histogram passes of 11, 11 and 10 bits
// (fewer when a bin is taken whole), then the kept rows as one bit each and the lists from prefix
// sums over groups of 32 rows. The lists take the keys' place; the CTA moves its rows itself.
// HELD: the weights and positions stay in shared memory too.
template <bool HELD>
__global__ void __launch_bounds__(kEvThreads) evict_kernel(EvictArgs a, int most) {
  extern __shared__ __align__(16) uint32_t ev_dyn[];
  __shared__ uint32_t hist[kEvBins];
  __shared__ EvDigit dg;
  __shared__ uint32_t tmp[32];
  const int groups_cap = (a.cap + 31) / 32;
  uint32_t* keys = ev_dyn;                      // [cap]
  uint32_t* cnt = keys + groups_cap * 32;       // [groups]
  uint32_t* kept = cnt + groups_cap;            // [groups]
  float* held_w = reinterpret_cast<float*>(kept + groups_cap);          // HELD: [cap]
  int32_t* held_p = reinterpret_cast<int32_t*>(held_w + groups_cap * 32);  // HELD: [cap], as they were
  const int ukv = blockIdx.x, tid = threadIdx.x, nt = blockDim.x, lane = tid & 31;
  EvUnit x;
  pdl_wait();
  pdl_trigger();
  int32_t* dst = reinterpret_cast<int32_t*>(keys);
  int32_t* src = dst + most;  // (2 most <= cap)
  if (evict_unit(a, ukv, &x, tid, nt)) {
    const int L = x.L, keep = x.keep, groups = (L + 31) / 32;
    auto weight_of = [&](int i) { return HELD ? held_w[i] : x.w[i]; };
    auto position_of = [&](int i) {
      const int q = HELD ? held_p[i] : x.pos[i];
      return q >= 0 ? q : x.seen - (L - i);
    };
    for (int b = tid; b < kEvBins; b += nt) hist[b] = 0;
    __syncthreads();
    // keys, and their top 11 bits counted
    constexpr int kU = 8;  // rows in flight per thread
    for (int i0 = 0; i0 < L; i0 += kU * nt) {
      float w[kU];
      int q[kU];
#pragma unroll
      for (int e = 0; e < kU; ++e) {
        const int i = i0 + e * nt + tid;
        if (i < L) {
          w[e] = x.w[i];
          q[e] = x.pos[i];
        }
      }
#pragma unroll
      for (int e = 0; e < kU; ++e) {
        const int i = i0 + e * nt + tid;
        if (i < L) {
          if (HELD) {
            held_w[i] = w[e];
            held_p[i] = q[e];
          }
          const int at = q[e] >= 0 ? q[e] : x.seen - (L - i);
          const uint32_t k = (long long)at >= x.recent_from ? 0xffffffffu : weight_key(w[e]);
          keys[i] = k;
          atomicAdd(&hist[k >> 21], 1u);
        }
      }
    }
    __syncthreads();
    find_digit(hist, keep, dg);
    uint32_t prefix = (uint32_t)dg.digit << 21;
    int remaining = keep - dg.above;
    bool all = dg.in_bin == remaining;  // every key of the bin is kept
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      if (all) break;
      const int shift = pass == 0 ? 10 : 0;
      const uint32_t high = pass == 0 ? 0xffe00000u : 0xfffffc00u;
      const uint32_t bins = pass == 0 ? 2047u : 1023u;
      for (int b = tid; b < kEvBins; b += nt) hist[b] = 0;
      __syncthreads();
      for (int i = tid; i < L; i += nt) {
        const uint32_t k = keys[i];
        if ((k & high) == prefix) atomicAdd(&hist[(k >> shift) & bins], 1u);
      }
      __syncthreads();
      find_digit(hist, remaining, dg);
      prefix |= (uint32_t)dg.digit << shift;
      remaining -= dg.above;
      all = dg.in_bin == remaining;
    }
    // kept: key above prefix, and of those equal the first `remaining` (all: every key from prefix on)
    const int span = (L + nt - 1) / nt * nt;
    if (!all) {
      for (int i = tid; i < span; i += nt) {
        const uint32_t m = __ballot_sync(0xffffffffu, i < L && keys[i] == prefix);
        if (lane == 0 && i < groups * 32) cnt[i >> 5] = __popc(m);
      }
      __syncthreads();
      scan_counts(cnt, groups, tmp);
    }
    for (int i = tid; i < span; i += nt) {
      const uint32_t k = i < L ? keys[i] : 0u;
      bool take = i < L && (all ? k >= prefix : k > prefix);
      if (!all) {
        const uint32_t m = __ballot_sync(0xffffffffu, i < L && k == prefix);
        if (i < L && k == prefix)
          take = (int)(cnt[i >> 5] + __popc(m & ((1u << lane) - 1u))) < remaining;
      }
      const uint32_t t = __ballot_sync(0xffffffffu, take);
      if (lane == 0 && i < groups * 32) kept[i >> 5] = t;
    }
    __syncthreads();
    for (int g = tid; g < groups; g += nt) {
      const int r0 = g * 32;
      const uint32_t low = r0 + 32 <= keep ? 0xffffffffu : (r0 >= keep ? 0u : (1u << (keep - r0)) - 1u);
      const uint32_t t = kept[g];
      cnt[g] = __popc(~t & low) | (__popc(t & ~low) << 16);  // (at most kEvSmemRows / 2 of each)
    }
    __syncthreads();
    const int moves = (int)(scan_counts(cnt, groups, tmp) & 0xffffu);
    // (the keys are done with: their memory takes the lists)
#pragma unroll 4
    for (int i = tid; i < L; i += nt) {
      const int g = i >> 5, r0 = g * 32, b = i & 31;
      const uint32_t low = r0 + 32 <= keep ? 0xffffffffu : (r0 >= keep ? 0u : (1u << (keep - r0)) - 1u);
      const uint32_t t = kept[g], under = (1u << b) - 1u;
      const bool k = (t >> b) & 1u;
      if (i < keep) {
        if (!k) {
          const int m = (int)(cnt[g] & 0xffffu) + __popc(~t & low & under);
          dst[m] = i;
        } else {
          if (x.from) x.from[i] = i;
          if (x.wo != x.w) x.wo[i] = weight_of(i);
          const int q = HELD ? held_p[i] : x.pos[i];
          if (x.po != x.pos || q < 0) x.po[i] = q >= 0 ? q : x.seen - (L - i);
        }
      } else if (k) {
        const int m = (int)(cnt[g] >> 16) + __popc(t & ~low & under);
        src[m] = i;
      }
    }
    __syncthreads();
    move_rows<8>(a, ukv, dst, src, tid >> 5, nt >> 5, moves);
    evict_finish(x, dst, src, moves, weight_of, position_of);
  }
  if (lengths_apart(a) && tid == 0 && ukv % a.n_kv == 0) evict_length(a, ukv / a.n_kv);
}

// The same by a cluster of C CTAs per (unit, KV head), each with its part of the rows: histograms and
// counts are read from one another's shared memory and every CTA finds the same digits. The lists go
// to global memory; a kept row past keep leaves its weight and position in the out arrays at its own
// place, for the kernel that moves it.
__global__ void __launch_bounds__(kEvThreads) evict_cluster_kernel(EvictArgs a, EvictLists ls, int C) {
  extern __shared__ __align__(16) uint32_t ev_dyn[];
  __shared__ uint32_t hist[2][kEvBins], sum[kEvBins];
  __shared__ EvDigit dg;
  __shared__ uint32_t tmp[32], equal, free_rows, past_rows;
  const int part_groups = ((a.cap + 31) / 32 + C - 1) / C;
  uint32_t* keys = ev_dyn;                       // [32 part_groups]
  uint32_t* cnt = keys + part_groups * 32;       // [part_groups]
  uint32_t* kept = cnt + part_groups;            // [part_groups]
  const int rank = (int)cluster_rank(), ukv = blockIdx.x / C;
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31;
  EvUnit x;
  pdl_wait();
  pdl_trigger();
  if (!evict_unit(a, ukv, &x, rank * nt + tid, C * nt)) {  // (the same for the whole cluster)
    if (rank == 0 && tid == 0) ls.count[ukv] = 0;
    return;
  }
  // this CTA's rows [r0, r0 + rows)
  const int keep = x.keep, per = ((x.L + 31) / 32 + C - 1) / C;
  const int r0 = min(x.L, rank * per * 32), rows = min(x.L, r0 + per * 32) - r0;
  const int groups = (rows + 31) / 32, span = (rows + nt - 1) / nt * nt;
  for (int b = tid; b < kEvBins; b += nt) hist[0][b] = hist[1][b] = 0;
  __syncthreads();
  constexpr int kU = 8;  // rows in flight per thread
  for (int j0 = 0; j0 < rows; j0 += kU * nt) {
    float w[kU];
    int q[kU];
#pragma unroll
    for (int e = 0; e < kU; ++e) {
      const int j = j0 + e * nt + tid;
      if (j < rows) {
        w[e] = x.w[r0 + j];
        q[e] = x.pos[r0 + j];
      }
    }
#pragma unroll
    for (int e = 0; e < kU; ++e) {
      const int j = j0 + e * nt + tid;
      if (j < rows) {
        const int at = q[e] >= 0 ? q[e] : x.seen - (x.L - (r0 + j));
        const uint32_t k = (long long)at >= x.recent_from ? 0xffffffffu : weight_key(w[e]);
        keys[j] = k;
        atomicAdd(&hist[0][k >> 21], 1u);
      }
    }
  }
  // the digit that the cluster's histograms together give (a barrier before and after its reads)
  auto digit = [&](const uint32_t* h, int remaining) {
    cluster_sync_all();
    for (int b = tid; b < kEvBins; b += nt) {
      uint32_t s = 0;
      for (int c = 0; c < C; ++c) s += ld_peer_u32(h + b, c);
      sum[b] = s;
    }
    __syncthreads();
    find_digit(sum, remaining, dg);
  };
  digit(hist[0], keep);
  uint32_t prefix = (uint32_t)dg.digit << 21;
  int remaining = keep - dg.above;
  bool all = dg.in_bin == remaining;  // every key of the bin is kept
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    if (all) break;
    const int shift = pass == 0 ? 10 : 0;
    const uint32_t high = pass == 0 ? 0xffe00000u : 0xfffffc00u;
    const uint32_t bins = pass == 0 ? 2047u : 1023u;
    uint32_t* h = hist[pass == 0 ? 1 : 0];
    if (pass == 1) {  // (every CTA has read the first one: each was at a cluster barrier since)
      for (int b = tid; b < kEvBins; b += nt) h[b] = 0;
      __syncthreads();
    }
    for (int j = tid; j < rows; j += nt) {
      const uint32_t k = keys[j];
      if ((k & high) == prefix) atomicAdd(&h[(k >> shift) & bins], 1u);
    }
    digit(h, remaining);
    prefix |= (uint32_t)dg.digit << shift;
    remaining -= dg.above;
    all = dg.in_bin == remaining;
  }
  // kept: key above prefix, and of those equal the first `remaining` (all: every key from prefix on)
  if (!all) {
    for (int j = tid; j < span; j += nt) {
      const uint32_t m = __ballot_sync(0xffffffffu, j < rows && keys[j] == prefix);
      if (lane == 0 && j < groups * 32) cnt[j >> 5] = __popc(m);
    }
    __syncthreads();
    const uint32_t mine = scan_counts(cnt, groups, tmp);
    if (tid == 0) equal = mine;
    cluster_sync_all();
    for (int c = 0; c < rank; ++c) remaining -= (int)ld_peer_u32(&equal, c);
  }
  for (int j = tid; j < span; j += nt) {
    const uint32_t k = j < rows ? keys[j] : 0u;
    bool take = j < rows && (all ? k >= prefix : k > prefix);
    if (!all) {
      const uint32_t m = __ballot_sync(0xffffffffu, j < rows && k == prefix);
      if (j < rows && k == prefix)
        take = (int)(cnt[j >> 5] + __popc(m & ((1u << lane) - 1u))) < remaining;
    }
    const uint32_t t = __ballot_sync(0xffffffffu, take);
    if (lane == 0 && j < groups * 32) kept[j >> 5] = t;
  }
  __syncthreads();
  // of group g: its rows below keep
  auto low_rows = [&](int g) {
    const int left = keep - (r0 + g * 32);
    return left >= 32 ? 0xffffffffu : (left <= 0 ? 0u : (1u << left) - 1u);
  };
  for (int g = tid; g < groups; g += nt) {
    const uint32_t low = low_rows(g), t = kept[g];
    cnt[g] = __popc(~t & low) | (__popc(t & ~low) << 16);  // (at most kEvClusterMost of both together)
  }
  __syncthreads();
  const uint32_t mine = scan_counts(cnt, groups, tmp);
  if (tid == 0) {
    free_rows = mine & 0xffffu;
    past_rows = mine >> 16;
  }
  cluster_sync_all();
  int free_at = 0, past_at = 0;
  for (int c = 0; c < rank; ++c) {
    free_at += (int)ld_peer_u32(&free_rows, c);
    past_at += (int)ld_peer_u32(&past_rows, c);
  }
  if (rank == C - 1 && tid == 0) ls.count[ukv] = free_at + (int)free_rows;
  int32_t* dst = ls.dst + (size_t)ukv * ls.most + free_at;
  int32_t* src = ls.src + (size_t)ukv * ls.most + past_at;
#pragma unroll 4
  for (int j = tid; j < rows; j += nt) {
    const int g = j >> 5, b = j & 31, i = r0 + j;
    const uint32_t low = low_rows(g), t = kept[g], under = (1u << b) - 1u;
    const bool k = (t >> b) & 1u;
    if (k) {
      if (i < keep && x.from) x.from[i] = i;
      if (i >= keep) src[(cnt[g] >> 16) + __popc(t & ~low & under)] = i;
      if (x.wo != x.w) x.wo[i] = x.w[i];
      const int q = x.pos[i];
      if (x.po != x.pos || q < 0) x.po[i] = q >= 0 ? q : x.seen - (x.L - i);
    } else if (i < keep) {
      dst[(cnt[g] & 0xffffu) + __popc(~t & low & under)] = i;
    } else {
      x.wo[i] = 0.f;
      x.po[i] = -1;
    }
  }
  cluster_sync_all();  // (no CTA ends before its shared memory has been read)
}

// The same for units of more rows than that holds: 8 bits at a time, the keys made again for
// each pass, the lists 1024 rows at a time.
__global__ void __launch_bounds__(kEvThreads) evict_select_kernel(EvictArgs a, EvictLists ls) {
  __shared__ EvSmem sm;
  const int ukv = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  EvUnit x;
  pdl_wait();
  pdl_trigger();
  if (!evict_unit(a, ukv, &x, tid, kEvThreads)) {
    if (tid == 0) ls.count[ukv] = 0;
    return;
  }
  const int L = x.L, keep = x.keep;
  auto key_of = [&](int i) { return x.key(i); };
  // the keep-th largest key, 8 bits at a time
  uint32_t prefix = 0, mask = 0;
  int remaining = keep;
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (tid < 256) sm.hist[tid] = 0;
    __syncthreads();
    for (int i = tid; i < L; i += kEvThreads) {
      const uint32_t k = key_of(i);
      if ((k & mask) == prefix) atomicAdd(&sm.hist[(k >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (warp == 0) {
      int cnt[8], s = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        cnt[j] = (int)sm.hist[255 - 8 * lane - j];
        s += cnt[j];
      }
      const int incl = warp_incl_scan(s);
      int acc = incl - s;
      if (acc < remaining && incl >= remaining) {
        for (int j = 0; j < 8; ++j) {
          if (acc + cnt[j] >= remaining) {
            sm.digit = 255 - 8 * lane - j;
            sm.above = acc;
            break;
          }
          acc += cnt[j];
        }
      }
    }
    __syncthreads();
    prefix |= (uint32_t)sm.digit << shift;
    mask |= 255u << shift;
    remaining -= sm.above;
  }
  // rows with key > prefix are kept, and the first `remaining` of those equal to it
  int eq_before = 0, free_before = 0, past_before = 0;
  int32_t* dst = ls.dst + (size_t)ukv * ls.most;
  int32_t* src = ls.src + (size_t)ukv * ls.most;
  for (int i0 = 0; i0 < L; i0 += kEvThreads) {
    const int i = i0 + tid;
    const uint32_t k = i < L ? key_of(i) : 0u;
    const bool eq = i < L && k == prefix;
    const unsigned long long e = block_excl_scan64(eq ? 1ull : 0ull, sm.tmp);
    const bool kept = i < L && (k > prefix || (eq && eq_before + (int)e < remaining));
    const bool hole = i < keep && !kept;
    const bool mover = i >= keep && kept;
    const unsigned long long y =
        block_excl_scan64((hole ? 1ull : 0ull) | (mover ? 1ull << 32 : 0ull), sm.tmp);
    if (hole) dst[free_before + (int)(y & 0xffffffffull)] = i;
    if (mover) src[past_before + (int)(y >> 32)] = i;
    if (tid == kEvThreads - 1) {
      sm.base[0] = (int)(y & 0xffffffffull) + (hole ? 1 : 0);
      sm.base[1] = (int)(y >> 32) + (mover ? 1 : 0);
      sm.in_bin = (int)e + (eq ? 1 : 0);
    }
    if (kept) {
      if (i < keep && x.from) x.from[i] = i;
      const int p = x.position(i);
      x.wo[i] = x.w[i];
      x.po[i] = p;
    } else if (i >= keep && i < L) {
      x.wo[i] = 0.f;
      x.po[i] = -1;
    }
    __syncthreads();
    free_before += sm.base[0];
    past_before += sm.base[1];
    eq_before += sm.in_bin;
    __syncthreads();
  }
  if (tid == 0) ls.count[ukv] = past_before;
}

// The moves of all (unit, KV head)s over the whole GPU.
__global__ void __launch_bounds__(kEvMoveThreads) evict_move_kernel(EvictArgs a, EvictLists ls) {
  pdl_wait();
  const int ukv = blockIdx.x, u = ukv / a.n_kv;
  if (blockIdx.y == 0 && ukv == u * a.n_kv && threadIdx.x == 0) evict_length(a, u);
  move_rows<4>(a, ukv, ls.dst + (size_t)ukv * ls.most, ls.src + (size_t)ukv * ls.most,
               blockIdx.y * kEvMoveWarps + (threadIdx.x >> 5), gridDim.y * kEvMoveWarps,
               ls.count[ukv]);
  // their weights and positions, which the select left in the out arrays
  const size_t row0 = (size_t)ukv * a.cap, list = (size_t)ukv * ls.most;
  for (int m = blockIdx.y * kEvMoveThreads + threadIdx.x; m < ls.count[ukv]; m += gridDim.y * kEvMoveThreads) {
    const int d = ls.dst[list + m], s = ls.src[list + m];
    const float w = a.weights_out[row0 + s];
    const int p = a.pos_out[row0 + s];
    a.weights_out[row0 + d] = w;
    a.pos_out[row0 + d] = p;
    a.weights_out[row0 + s] = 0.f;
    a.pos_out[row0 + s] = -1;
    if (a.src_rows) a.src_rows[(size_t)ukv * a.keep + d] = s;
  }
}

// CTAs of a cluster: more while the GPU has SMs for them and each has rows to work on (32 units of up
// to 32K rows: one CTA each 44.6 us, two 37.8, four 31.7, eight, more than there are SMs, 58.5), and as
// many as shared memory asks for (8 units of 131072 rows: clusters 41 us, evict_select_kernel 402);
// 0: more than kEvMaxCluster.
static int evict_cluster(int units, int cap) {
  int c = 1;
  while (c < kEvMaxCluster && (long long)units * 2 * c <= device_sm_count() && cap / (2 * c) >= kEvClusterRows)
    c *= 2;
  while (c <= kEvMaxCluster && (cap + c - 1) / c > kEvClusterMost) c *= 2;
  return c <= kEvMaxCluster ? c : 0;
}

static cudaError_t launch_cluster(const EvictArgs& a, const EvictLists& ls, int c, cudaStream_t s) {
  const size_t groups = ((a.cap + 31) / 32 + c - 1) / c, smem = groups * (32 + 2) * 4;
  const cudaError_t e = ensure_dyn_smem((const void*)evict_cluster_kernel, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.n * a.n_kv) * c);
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = c;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_cluster_kernel, a, ls, c);
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  const EvictLists ls = lists_of(a);
  const int units = a.n * a.n_kv;
  // With a unit for every SM, one CTA does all of it; fewer are spread over clusters, and their rows moved
  // by a second kernel. To 4096 rows in 4 bits, one CTA against clusters: 256 units of 4352 rows 20.9 and
  // 36.9 us, of 16384 105.6 and 120.5, of 32768 146.9 and 193.9, of 40960 170.0 and 219.3, 160 units of
  // 16384 91.2 and 90.7; in bf16 256 units of 4352 21.9 and 35.7, of 32768 214.1 and 259.4.
  if (a.cap <= kEvSmemRows && units >= device_sm_count()) {
    const size_t groups = (a.cap + 31) / 32;
    const bool held = a.cap <= kEvHeldRows;
    const size_t smem = groups * (32 + 2 + (held ? 64 : 0)) * 4;
    const auto kern = held ? evict_kernel<true> : evict_kernel<false>;
    cudaError_t e = ensure_dyn_smem((const void*)kern, smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl_kernel(kern, dim3(units), dim3(held ? 512 : kEvThreads), smem, s, a, ls.most);
    if (e != cudaSuccess || lengths_apart(a)) return e;
    return launch_pdl_kernel(evict_length_kernel, dim3((a.n + 255) / 256), dim3(256), 0, s, a);
  }
  const int c = evict_cluster(units, a.cap);
  const cudaError_t e =
      c ? launch_cluster(a, ls, c, s)
        : launch_pdl_kernel(evict_select_kernel, dim3(units), dim3(kEvThreads), 0, s, a, ls);
  if (e != cudaSuccess) return e;
  const int rows = 4 * kEvMoveWarps * (a.row_bytes[2] ? 3 : 1);  // of a CTA at a time
  int y = (ls.most + rows - 1) / rows;
  y = y < 1 ? 1 : (y > 1024 ? 1024 : y);
  return launch_pdl_kernel(evict_move_kernel, dim3(units, y), dim3(kEvMoveThreads), 0, s, a, ls);
}

}  // namespace rkv
