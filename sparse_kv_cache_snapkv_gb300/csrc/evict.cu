// Eviction by accumulated attention weight (sm_103a), in place.
//
// Per (unit, KV head) with L > keep rows: a row's key is the order-preserving integer of its
// weight, or the largest integer when its position is among the last `recent`. The keep-th largest
// key T and the number of keys equal to T that are still kept (the lowest rows) come from an
// MSB-first radix select; then the free rows below keep and the kept rows at or past keep, equally
// many, are listed in ascending order and paired. Sources lie at or past keep and destinations
// below it, so all moves are independent.
#include <cuda_runtime.h>
#include <cstdint>

#include "common.cuh"
#include "rkv_internal.h"

namespace rkv {

constexpr int kEvThreads = 1024;
constexpr int kEvMoveThreads = 256;
constexpr int kEvMoveWarps = kEvMoveThreads / 32;

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

size_t evict_scratch_bytes(int n, int n_kv, int cap, int keep) {
  const size_t units = (size_t)n * n_kv;
  return align_up(units * 4, 256) + 2 * align_up(units * most_moves(cap, keep) * 4, 256);
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

__global__ void __launch_bounds__(kEvThreads) evict_select_kernel(EvictArgs a, EvictLists ls) {
  __shared__ EvSmem sm;
  const int ukv = blockIdx.x, u = ukv / a.n_kv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int L = a.len[u], keep = a.keep;
  const bool bad = L < 0 || L > a.cap;
  if (tid == 0) {
    ls.count[ukv] = 0;
    if (bad) set_status(a.status, RKV_DEV_LEN_OVER_CAP);
  }
  if (bad) return;
  const size_t row0 = (size_t)ukv * a.cap;
  const float* w = a.weights + row0;
  const int32_t* pos = a.pos + row0;
  float* wo = a.weights_out + row0;
  int32_t* po = a.pos_out + row0;
  int32_t* from = a.src_rows ? a.src_rows + (size_t)ukv * keep : nullptr;
  if (L <= keep) {
    for (int i = tid; i < L; i += kEvThreads) {
      wo[i] = w[i];
      po[i] = pos[i];
    }
    if (from)
      for (int i = tid; i < keep; i += kEvThreads) from[i] = i < L ? i : -1;
    return;
  }
  const int seen = a.seen[u];
  auto position = [&](int i) {
    const int p = pos[i];
    return p >= 0 ? p : seen - (L - i);
  };
  // 64-bit sums: positions and seen are the caller's, and their difference may be anything
  auto key_of = [&](int i) {
    return (long long)position(i) >= (long long)seen - a.recent ? 0xffffffffu : weight_key(w[i]);
  };
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
    const unsigned long long x =
        block_excl_scan64((hole ? 1ull : 0ull) | (mover ? 1ull << 32 : 0ull), sm.tmp);
    if (hole) dst[free_before + (int)(x & 0xffffffffull)] = i;
    if (mover) src[past_before + (int)(x >> 32)] = i;
    if (tid == kEvThreads - 1) {
      sm.base[0] = (int)(x & 0xffffffffull) + (hole ? 1 : 0);
      sm.base[1] = (int)(x >> 32) + (mover ? 1 : 0);
      sm.in_bin = (int)e + (eq ? 1 : 0);
    }
    if (kept && i < keep) {
      if (from) from[i] = i;
      const int p = position(i);
      wo[i] = w[i];
      po[i] = p;
    }
    __syncthreads();
    free_before += sm.base[0];
    past_before += sm.base[1];
    eq_before += sm.in_bin;
    __syncthreads();
  }
  for (int m = tid; m < past_before; m += kEvThreads) {
    const int d = dst[m], s = src[m];
    const int p = position(s);
    const float x = w[s];
    wo[d] = x;
    po[d] = p;
    if (from) from[d] = s;
  }
  __syncthreads();
  for (int i = keep + tid; i < L; i += kEvThreads) {
    wo[i] = 0.f;
    po[i] = -1;
  }
  if (tid == 0) ls.count[ukv] = past_before;
}

// One warp per moved row; the lanes split its bytes in words of 8.
__global__ void __launch_bounds__(kEvMoveThreads) evict_move_kernel(EvictArgs a, EvictLists ls) {
  const int ukv = blockIdx.x, u = ukv / a.n_kv;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (blockIdx.y == 0 && ukv == u * a.n_kv && threadIdx.x == 0) {
    const int L = a.len[u];
    a.len_out[u] = (L >= 0 && L <= a.cap) ? min(L, a.keep) : L;
  }
  const int count = ls.count[ukv];
  const int32_t* dst = ls.dst + (size_t)ukv * ls.most;
  const int32_t* src = ls.src + (size_t)ukv * ls.most;
  for (int m = blockIdx.y * kEvMoveWarps + warp; m < count; m += gridDim.y * kEvMoveWarps) {
    const size_t d = (size_t)ukv * a.cap + dst[m], s = (size_t)ukv * a.cap + src[m];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (lane * 8 < a.row_bytes[k])
        *reinterpret_cast<uint2*>(a.rows[k] + d * a.row_bytes[k] + lane * 8) =
            *reinterpret_cast<const uint2*>(a.rows[k] + s * a.row_bytes[k] + lane * 8);
    }
  }
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  const EvictLists ls = lists_of(a);
  evict_select_kernel<<<a.n * a.n_kv, kEvThreads, 0, s>>>(a, ls);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  int y = (ls.most + 4 * kEvMoveWarps - 1) / (4 * kEvMoveWarps);
  y = y < 1 ? 1 : (y > 1024 ? 1024 : y);
  evict_move_kernel<<<dim3(a.n * a.n_kv, y), kEvMoveThreads, 0, s>>>(a, ls);
  return cudaGetLastError();
}

}  // namespace rkv
