// Block tables and slots of a batch of requests, kept on the GPU (sm_103a).
//
// Reserve: unit u needs ceil((len + new) / block) - held more blocks; they come off the top of the free
// stack in the order of the units, so a unit's are known from the sum of what the units before it need
// (also of those that could not be served: then a unit is served exactly if all needs up to its own are
// covered, which needs no second pass). A token's slot follows from its position alone: its block is an
// old entry of the table or, counted from the first new one, an entry of the stack.
// Release: a unit keeps ceil(len / block) blocks and the others go back, in the order of the units.
//
// Bound: a call's latency, and for prompts writing 8 bytes a token. One block forms the sums; a few
// thousand tokens are placed by that block too, more by a second kernel.
#include <cuda_runtime.h>
#include <climits>
#include <cstdint>

#include "common.cuh"
#include "rkv_internal.h"
#include "tensor_core.cuh"

namespace rkv {

constexpr int kSlotThreads = 1024;
constexpr int kSlotFew = 8192;  // places (or table entries) that the first block deals with itself

// What the sums say of a unit (workspace).
struct __align__(16) SlotUnit {
  int start;   // its first token's place in the packed order
  int len;     // tokens it has already
  int held;    // blocks it holds
  int before;  // blocks of the stack that go to units before it; -1: not served
};

__device__ __forceinline__ int ceil_blocks(long long tokens, int block) {
  return (int)((tokens + block - 1) / block);
}

// Places of Q tokens each, t = Q first, Q (first + step), ... Neighbours mostly share the unit and the block,
// which are looked up again only where they change. (One token each where there are few: 256 requests of one
// token 4.1 us, with four each 7.1; 1.08M tokens of 64 requests 11.3 us with one, 8.4 with four.)
template <int Q>
__device__ __forceinline__ void place_tokens(const SlotArgs& a, const SlotUnit* unit, int all, int count,
                                             long long first, long long step) {
  for (long long t0 = Q * first; t0 < a.room; t0 += Q * step) {
    int slot[Q], pos[Q];
    SlotUnit u{};
    int at = -1, end = -1;  // the unit, and the first token behind it
    int held = -1, b = -1;  // the block's number in the table, and the block
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      const long long t = t0 + i;
      slot[i] = -1;
      pos[i] = 0;
      if (t >= all || t >= a.room) continue;
      if (t >= end) {
        int lo = at < 0 ? 0 : at, hi = a.n;  // the last unit that begins at or before t
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (unit[mid].start <= t) lo = mid; else hi = mid;
        }
        at = lo;
        u = unit[lo];
        end = unit[lo + 1].start;
        held = -1;
      }
      if (u.before < 0) continue;
      const int p = u.len + (int)(t - u.start), j = p / a.block, off = p - j * a.block;
      if (j != held) {
        held = j;
        b = j < u.held ? a.table[(size_t)at * a.max_blocks + j] : a.free_blocks[count - 1 - u.before - (j - u.held)];
        if (b < 0 || b >= a.num_blocks) set_status(a.status, RKV_DEV_BAD_INDEX);
      }
      if (j >= u.held && off == 0) a.table[(size_t)at * a.max_blocks + j] = b;
      if (b >= 0 && b < a.num_blocks) {
        slot[i] = b * a.block + off;
        pos[i] = p;
      }
    }
    if (Q == 4 && t0 + Q <= a.room && a.wide) {
      *reinterpret_cast<int4*>(a.slots + t0) = make_int4(slot[0], slot[1 % Q], slot[2 % Q], slot[3 % Q]);
      *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1 % Q], pos[2 % Q], pos[3 % Q]);
    } else {
#pragma unroll
      for (int i = 0; i < Q; ++i)
        if (t0 + i < a.room) {
          a.slots[t0 + i] = slot[i];
          a.positions[t0 + i] = pos[i];
        }
    }
  }
}

// After the units: {tokens in all, entries of the stack before the call}.
__global__ void __launch_bounds__(kSlotThreads) reserve_kernel(SlotArgs a, SlotUnit* unit) {
  __shared__ unsigned long long tmp[33];
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  const int count = *a.free_count;
  const int there = count >= 0 && count <= a.num_blocks ? count : 0;
  if (there != count && tid == 0) set_status(a.status, RKV_DEV_BAD_INDEX);
  unsigned long long tokens = 0, blocks = 0;  // of the units before this round's
  unsigned long long taken = 0;
  for (int base = 0; base < a.n; base += kSlotThreads) {
    const int u = base + tid;
    int len = 0, add = 0, held = 0;
    bool fine = false;
    if (u < a.n) {
      len = a.len[u];
      add = a.new_len[u];
      held = a.held[u];
      const long long room = (long long)a.max_blocks * a.block;
      fine = len >= 0 && add >= 0 && held >= 0 && held <= a.max_blocks && (long long)len + add <= room;
      if (!fine) {
        set_status(a.status, RKV_DEV_LEN_OVER_CAP);
      } else if (held < ceil_blocks(len, a.block)) {
        set_status(a.status, RKV_DEV_BAD_INDEX);
        fine = false;
      }
      add = max(add, 0);
    }
    // tokens first: a unit that they have no room for takes no blocks
    const unsigned long long before_t = tokens + block_excl_scan64((unsigned long long)add, tmp);
    if (fine && before_t + add > (unsigned long long)a.room) {
      set_status(a.status, RKV_DEV_LEN_OVER_CAP);
      fine = false;
    }
    const int need = fine ? max(0, ceil_blocks((long long)len + add, a.block) - held) : 0;
    const unsigned long long before_b = blocks + block_excl_scan64((unsigned long long)need, tmp);
    const bool served = fine && (need == 0 || before_b + need <= (unsigned long long)there);
    if (fine && !served) set_status(a.status, RKV_DEV_NO_BLOCKS);
    if (u < a.n) {
      const int start = (int)min(before_t, (unsigned long long)INT_MAX);
      unit[u] = SlotUnit{start, len, held, served ? (int)min(before_b, (unsigned long long)INT_MAX) : -1};
      a.q_start[u] = start;
      a.len_out[u] = served ? len + add : len;
      a.held_out[u] = served ? held + need : held;
    }
    unsigned long long got = served ? (unsigned long long)need : 0ull, x;
    x = block_excl_scan64(got, tmp);
    if (tid == kSlotThreads - 1) {
      tmp[0] = before_t + add;
      tmp[1] = before_b + need;
      tmp[2] = x + got;
    }
    __syncthreads();
    tokens = tmp[0];
    blocks = tmp[1];
    taken += tmp[2];
    __syncthreads();
  }
  const int all = (int)min(tokens, (unsigned long long)INT_MAX);
  if (tid == 0) {
    a.q_start[a.n] = all;
    *a.free_count_out = count - (int)taken;
    unit[a.n] = SlotUnit{all, count, 0, 0};
  }
  if (a.room > kSlotFew) return;
  __syncthreads();
  place_tokens<1>(a, unit, all, count, tid, kSlotThreads);
}

__global__ void __launch_bounds__(256) place_kernel(SlotArgs a, const SlotUnit* unit) {
  pdl_wait();
  pdl_trigger();
  const SlotUnit end = unit[a.n];
  place_tokens<4>(a, unit, end.start, end.len, (long long)blockIdx.x * 256 + threadIdx.x,
               (long long)gridDim.x * 256);
}

// unit: {blocks it keeps, where its others go on the stack, how many they are, -}
__device__ __forceinline__ void give_back(const SlotArgs& a, const SlotUnit& x, int u, int first, int step) {
  for (int j = first; j < x.held; j += step) {
    const int b = a.table[(size_t)u * a.max_blocks + x.start + j];
    if (b < 0 || b >= a.num_blocks) set_status(a.status, RKV_DEV_BAD_INDEX);
    a.free_blocks[x.len + j] = b;
  }
}

__global__ void __launch_bounds__(kSlotThreads) release_kernel(SlotArgs a, SlotUnit* unit) {
  __shared__ unsigned long long tmp[33];
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  const int count = *a.free_count;
  unsigned long long total = 0;
  for (int base = 0; base < a.n; base += kSlotThreads) {
    const int u = base + tid;
    int keep = 0, give = 0;
    if (u < a.n) {
      const int len = a.len[u], held = a.held[u];
      keep = held;
      if (len < 0 || held < 0 || held > a.max_blocks) {
        set_status(a.status, RKV_DEV_LEN_OVER_CAP);
      } else {
        keep = min(held, ceil_blocks(len, a.block));
        give = held - keep;
      }
    }
    const unsigned long long before = total + block_excl_scan64((unsigned long long)give, tmp);
    if (u < a.n) unit[u] = SlotUnit{keep, count + (int)min(before, (unsigned long long)INT_MAX / 2), give, 0};
    if (tid == kSlotThreads - 1) tmp[0] = before + give;
    __syncthreads();
    total = tmp[0];
    __syncthreads();
  }
  // more blocks than the pool has: some were held twice, and nothing goes back
  const bool fine = count >= 0 && count <= a.num_blocks && total <= (unsigned long long)(a.num_blocks - count);
  if (!fine && tid == 0) set_status(a.status, RKV_DEV_BAD_INDEX);
  for (int u = tid; u < a.n; u += kSlotThreads) {
    SlotUnit x = unit[u];
    a.held_out[u] = fine ? x.start : x.start + x.held;
    if (!fine) unit[u].held = 0;
  }
  if (tid == 0) *a.free_count_out = fine ? count + (int)total : count;
  if ((long long)a.n * a.max_blocks > kSlotFew) return;
  __syncthreads();
  for (int u = tid >> 5; u < a.n; u += kSlotThreads / 32) give_back(a, unit[u], u, tid & 31, 32);
}

__global__ void __launch_bounds__(128) give_kernel(SlotArgs a, const SlotUnit* unit) {
  pdl_wait();
  pdl_trigger();
  for (int u = blockIdx.x; u < a.n; u += gridDim.x) give_back(a, unit[u], u, threadIdx.x, 128);
}

size_t slots_scratch_bytes(int n) { return align_up(((size_t)n + 1) * sizeof(SlotUnit), 256); }

cudaError_t launch_reserve_slots(const SlotArgs& a, cudaStream_t s) {
  SlotUnit* unit = static_cast<SlotUnit*>(a.scratch);
  const cudaError_t e = launch_pdl_kernel(reserve_kernel, dim3(1), dim3(kSlotThreads), 0, s, a, unit);
  if (e != cudaSuccess || a.room <= kSlotFew) return e;
  const int most = device_sm_count() * 8, ctas = (a.room - 1) / 1024 + 1;
  return launch_pdl_kernel(place_kernel, dim3(ctas < most ? ctas : most), dim3(256), 0, s, a,
                           (const SlotUnit*)unit);
}

cudaError_t launch_release_blocks(const SlotArgs& a, cudaStream_t s) {
  SlotUnit* unit = static_cast<SlotUnit*>(a.scratch);
  const cudaError_t e = launch_pdl_kernel(release_kernel, dim3(1), dim3(kSlotThreads), 0, s, a, unit);
  if (e != cudaSuccess || (long long)a.n * a.max_blocks <= kSlotFew) return e;
  const int most = device_sm_count() * 16;
  return launch_pdl_kernel(give_kernel, dim3(a.n < most ? a.n : most), dim3(128), 0, s, a,
                           (const SlotUnit*)unit);
}

}  // namespace rkv
