// Rotary positions of packed queries and keys, with the new rows stored in the cache (sm_103a).
//
// Pair i of a head's first `rot` dimensions, (x_2i, x_2i+1) or (x_i, x_i+rot/2), is turned by the angle
// pos * f_i and scaled by mscale. An angle of a far position has few bits behind the point in fp32
// (position 2^20: 2^-4), so it is kept as a fraction of a turn in 64-bit fixed point: f_i / (2 pi) once
// as a 64-bit fraction, times the position modulo 2^64, which drops whole turns exactly. Its upper 32
// bits, as a signed number in units of pi, go to sincospi; what is lost is below 2^-24 of a turn.
//
// Bound: reading and writing each row once. Eight threads share a head, with two 16-byte pieces each
// that hold eight whole pairs in either layout, so nothing crosses threads but the angles; a warp keeps
// its token's eight cosines and sines per lane for all of its heads.
#include <cuda_runtime.h>
#include <cstdint>

#include "common.cuh"
#include "rkv_internal.h"
#include "tensor_core.cuh"

namespace rkv {

constexpr int kRopeThreads = 256;
constexpr int kRopeAhead = 4;  // heads whose loads a thread has under way
// Blocks an SM, which its registers hold: each goes on to further tokens, so that a warp's fractions of a turn
// are worked out once (1666 tokens of 40 heads: 11.3 us with four times as many blocks, 8.5 so). With registers
// for three, loads of one head at a time and more warps: 142 us for the 34800 tokens below.
constexpr int kRopePerSm = 2;

__device__ __forceinline__ void rotate(uint4 a, uint4 b, const float* cs, const float* sn,
                                       bool interleaved, uint4* oa, uint4* ob) {
  float x[16], y[16];
  unpack8(a, x);
  unpack8(b, x + 8);
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[2 * i] = x[2 * i] * cs[i] - x[2 * i + 1] * sn[i];
      y[2 * i + 1] = x[2 * i + 1] * cs[i] + x[2 * i] * sn[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = x[i] * cs[i] - x[8 + i] * sn[i];
      y[8 + i] = x[8 + i] * cs[i] + x[i] * sn[i];
    }
  }
  *oa = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                   pack_bf16x2(y[6], y[7]));
  *ob = make_uint4(pack_bf16x2(y[8], y[9]), pack_bf16x2(y[10], y[11]), pack_bf16x2(y[12], y[13]),
                   pack_bf16x2(y[14], y[15]));
}

// A warp takes heads [part * per, ...) of one token after the other.
__global__ void __launch_bounds__(kRopeThreads, kRopePerSm) rope_append_kernel(RopeArgs a, int parts, int per) {
  const int lane = threadIdx.x & 31, c = lane & 7;
  const long long warps = (long long)gridDim.x * (kRopeThreads / 32);
  const long long warp = (long long)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int heads = a.hq + 2 * a.n_kv, half = a.rot / 2, turning = a.rot / 16;
  pdl_wait();
  pdl_trigger();
  // this lane's pairs, 2 lane and 2 lane + 1: fractions of a turn per position
  unsigned long long turn[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int pair = 2 * lane + i;
    const double t = pair < half ? (double)a.inv_freq[pair] * 0.15915494309189533577 : 0.0;  // 1 / (2 pi)
    turn[i] = (unsigned long long)__double2ull_rn((t - floor(t)) * 18446744073709551616.0);
  }
  // pieces of this thread: of a head's turned part, or of the rest
  const bool turned = c < turning;
  const int at0 = !turned ? a.rot + 16 * (c - turning) : a.interleaved ? 16 * c : 8 * c;
  const int at1 = !turned || a.interleaved ? at0 + 8 : half + at0;
  const long long rows = (long long)a.num_blocks * a.block;
  for (long long w = warp; w < (long long)a.tokens * parts; w += warps) {
    const int token = (int)(w / parts), part = (int)(w - (long long)token * parts);
    const int slot = a.slots[token];
    if (slot < 0) continue;
    if (slot >= rows) {
      if (lane == 0) set_status(a.status, RKV_DEV_BAD_INDEX);
      continue;
    }
    const unsigned long long pos = (unsigned long long)(long long)a.positions[token];
    float mine[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = (int)(uint32_t)((pos * turn[i]) >> 32);
      sincospif((float)t * 4.656612873077393e-10f, &mine[2 + i], &mine[i]);  // 2^-31
      mine[i] *= a.mscale;
      mine[2 + i] *= a.mscale;
    }
    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = __shfl_sync(0xffffffffu, mine[i & 1], 4 * c + (i >> 1));
      sn[i] = __shfl_sync(0xffffffffu, mine[2 + (i & 1)], 4 * c + (i >> 1));
    }
    const long long blk = slot / a.block, in_blk = slot - blk * a.block;
    const int end = min(heads, (part + 1) * per);
    // the loads of several heads first: a store might be to where a later load is from, for all the compiler
    // knows (34800 tokens of 48 heads: 153 us with one head at a time)
    for (int h0 = part * per + (lane >> 3); h0 < end; h0 += 4 * kRopeAhead) {
      uint4 x[kRopeAhead], y[kRopeAhead];
      bf16* dst[kRopeAhead];
#pragma unroll
      for (int i = 0; i < kRopeAhead; ++i) {
        const int h = h0 + 4 * i;
        const bf16* src;
        if (h < a.hq) {
          src = a.q + token * a.q_stride + h * kHeadDim;
          dst[i] = a.q_out + ((size_t)token * a.hq + h) * kHeadDim;
        } else {
          const bool key = h < a.hq + a.n_kv;
          const int g = key ? h - a.hq : h - a.hq - a.n_kv;
          src = (key ? a.k + token * a.k_stride : a.v + token * a.v_stride) + g * kHeadDim;
          dst[i] = (key ? a.k_cache : a.v_cache) + ((size_t)(blk * a.n_kv + g) * a.block + in_blk) * kHeadDim;
        }
        if (h < end) {
          x[i] = *reinterpret_cast<const uint4*>(src + at0);
          y[i] = *reinterpret_cast<const uint4*>(src + at1);
        }
      }
#pragma unroll
      for (int i = 0; i < kRopeAhead; ++i) {
        const int h = h0 + 4 * i;
        if (h >= end) break;
        if (turned && h < a.hq + a.n_kv) rotate(x[i], y[i], cs, sn, a.interleaved, &x[i], &y[i]);
        *reinterpret_cast<uint4*>(dst[i] + at0) = x[i];
        *reinterpret_cast<uint4*>(dst[i] + at1) = y[i];
      }
    }
  }
}

cudaError_t launch_rope_append(const RopeArgs& a, cudaStream_t s) {
  const int heads = a.hq + 2 * a.n_kv;
  // a warp for a token's heads where those fill the GPU twice, else for fewer heads, four at least (1666 tokens
  // of 40 heads: 8.6 us, filling it once 10.3, four times 13.1)
  const long long fill = (long long)device_sm_count() * kRopePerSm * (kRopeThreads / 16);
  int per = (heads + 3) / 4 * 4;
  while (per > 4 && (long long)a.tokens * ((heads + per - 1) / per) < fill) per = (per / 2 + 3) / 4 * 4;
  const int parts = (heads + per - 1) / per;
  const long long warps = (long long)a.tokens * parts;
  const long long most = (long long)device_sm_count() * kRopePerSm, ctas = (warps + 7) / 8;
  return launch_pdl_kernel(rope_append_kernel, dim3((unsigned)(ctas < most ? ctas : most)),
                           dim3(kRopeThreads), 0, s, a, parts, per);
}

}  // namespace rkv
