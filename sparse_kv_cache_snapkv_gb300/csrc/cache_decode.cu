// Append to and decode over a cache held in 4 bits, and the bf16 decode that also accumulates each
// token's attention weight (sm_103a).
//
// Decode, per (unit, KV head) with its G query heads and tokens j < L:
//   s_hj = scale q_h . K_j,  p_hj = exp(s_hj - m_h),  out_h = (sum_j p_hj V_j) / l_h,
//   weights_j += sum_h p_hj / l_h
// in one pass over K and V: each warp takes 16 tokens at a time with a running maximum and sum;
// the warps of a CTA, then the CTAs of a split sequence, are joined. The weights need the final
// sums, so the logits (4 G bytes per token against 144 or 512 of K and V) are kept in the
// workspace and turned into weights once those are known.
//
// Both products run on mma.sync m16n8k16 with the tokens (S^T = K Q^T) or the dimensions
// (O^T = V^T P^T) as the 16 rows and the query heads as the 8 columns: no row of the tile is
// padding at G = 8, and S^T leaves its maximum, its sum and P^T in the very lanes that hold the
// same heads' columns of O^T. A decode is bound by the cache's bytes; a tcgen05 tile of 128 rows
// would need the operands unpacked into shared memory first, which costs more than the product.
//
// The fragments come straight from global memory into registers. A fragment's columns may be
// any permutation of the dimensions as long as Q has the same one, and its rows any permutation of
// the tokens, so every lane takes 16 contiguous bytes of K codes (or of bf16 K) and 8 (16) of V,
// and no byte passes through shared memory. Each lane's next K is requested as soon as S^T is
// done, its next V after O^T: a warp always has loads in flight.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "cache4.cuh"
#include "common.cuh"
#include "rkv_internal.h"

namespace rkv {

// ==========================================================================================
// append
// ==========================================================================================
constexpr int kAppendThreads = 256;

__device__ __forceinline__ void load32(const void* p, uint32_t (&w)[8]) {
  const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
  w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
  w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}

__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// Tokens that unit u gets and has; 0 when the call may not touch it.
__device__ __forceinline__ int append_count(const Kv4AppendArgs& a, int u, int* have) {
  const int l = a.len[u], t = a.new_len ? a.new_len[u] : a.max_new;
  *have = l;
  if (l < 0 || t < 0 || t > a.max_new || l > a.cap - t) return -1;
  return t;
}

// One thread = one block of 16 values (32 bytes in, 8 + 1 out); blockIdx.y: K or V. Bound by the
// copy: 8 neighbouring threads make one row of codes and one of scales.
__global__ void __launch_bounds__(kAppendThreads) kv4_append_kernel(Kv4AppendArgs a) {
  const long long item = (long long)blockIdx.x * kAppendThreads + threadIdx.x;
  const long long row = item >> 3;
  const int blk = (int)(item & 7);
  const int ukv = (int)(row / a.max_new);
  const int i = (int)(row - (long long)ukv * a.max_new);
  if (ukv >= a.n * a.n_kv) return;
  const int u = ukv / a.n_kv, g = ukv - u * a.n_kv;
  int have;
  const int t = append_count(a, u, &have);
  const bool v = blockIdx.y != 0;
  if (g == 0 && i == 0 && blk == 0 && !v) {
    if (t < 0) set_status(a.status, RKV_DEV_LEN_OVER_CAP);
    // (len_out that is len itself is written by kv4_length_kernel, after every reader)
    if (a.len_out != a.len) a.len_out[u] = have + max(t, 0);
  }
  if (i >= t) return;
  const int at = have + i;
  size_t dst;
  if (a.pm.table)
    dst = paged_row(a.pm, paged_block(a.pm, u, at, a.status), a.n_kv, g, at);
  else
    dst = (size_t)ukv * a.cap + at;
  const size_t src = (size_t)row * kHeadDim + blk * kScaleGroup;
  uint32_t w[8], sb;
  load32((v ? a.new_v : a.new_k) + src, w);
  const uint2 c = quantise16(w, &sb);
  *reinterpret_cast<uint2*>((v ? a.v_codes : a.k_codes) + dst * kCodeBytes + blk * 8) = c;
  (v ? a.v_scales : a.k_scales)[dst * kRowScales + blk] = (uint8_t)sb;
  if (a.k_values) {
    values16(c, sb, w);
    store32((v ? a.v_values : a.k_values) + src, w);
  }
}

__global__ void kv4_length_kernel(Kv4AppendArgs a) {
  const int u = blockIdx.x * blockDim.x + threadIdx.x;
  if (u >= a.n) return;
  int have;
  const int t = append_count(a, u, &have);
  a.len_out[u] = have + max(t, 0);
}

cudaError_t launch_kv4_append(const Kv4AppendArgs& a, cudaStream_t s) {
  const long long items = (long long)a.n * a.n_kv * a.max_new * kRowScales;
  const long long ctas = (items + kAppendThreads - 1) / kAppendThreads;
  if (ctas > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  kv4_append_kernel<<<dim3((unsigned)ctas, 2), kAppendThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.len_out != a.len) return e;
  kv4_length_kernel<<<(a.n + 255) / 256, 256, 0, s>>>(a);
  return cudaGetLastError();
}

// ==========================================================================================
// decode
// ==========================================================================================
constexpr int kCdThreads = 256;
constexpr int kCdWarps = kCdThreads / 32;
constexpr int kCdTile = 16;                       // tokens a warp takes at a time
constexpr int kCdRound = kCdTile * kCdWarps;      // tokens a CTA takes at a time
constexpr int kCdWeightChunk = 1024;              // tokens a CTA of the join kernel turns into weights

void cache_decode_plan(int n, int n_kv, int cap, int* nsplit, int* tokens_per_split) {
  const long long units = (long long)n * n_kv;
  const long long target = 4LL * device_sm_count();  // two waves of two CTAs per SM
  const int rounds = (cap + kCdRound - 1) / kCdRound;
  long long ns = (target + units - 1) / units;
  ns = ns > rounds ? rounds : ns;
  const int per = (int)((rounds + ns - 1) / ns);
  *tokens_per_split = per * kCdRound;
  *nsplit = (rounds + per - 1) / per;
}

size_t cache_decode_scratch_bytes(int n, int n_kv, int gqa, int cap, bool with_weights) {
  int ns, tps;
  cache_decode_plan(n, n_kv, cap, &ns, &tps);
  const size_t units = (size_t)n * n_kv;
  return align_up(units * ns * gqa * 8, 256) + align_up(units * ns * gqa * kHeadDim * 4, 256) +
         (with_weights ? align_up(units * cap * gqa * 4, 256) : 0);
}

void cache_decode_carve(CacheDecodeArgs* a, void* scratch) {
  unsigned char* p = static_cast<unsigned char*>(scratch);
  const size_t rows = (size_t)a->n * a->n_kv * a->nsplit * a->gqa;
  a->part_ml = reinterpret_cast<float*>(p);
  p += align_up(rows * 8, 256);
  a->part_o = reinterpret_cast<float*>(p);
  p += align_up(rows * kHeadDim * 4, 256);
  a->logits = reinterpret_cast<float*>(p);
}

// Loads that do not stay in L1 (the cache is read once) and see what this CTA wrote before a barrier.
__device__ __forceinline__ uint4 ld_stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_stream8(const void* p) {
  uint2 v;
  asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "l"(p)
               : "memory");
  return v;
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Lane roles of the fragments: r = lane / 4, c = lane % 4. As rows of K, lane (r, c) holds parts of
// tokens tok(r) and 8 + tok(r) of the tile; as columns of V^T, tokens c, 4 + c, 8 + c, 12 + c.
// tok() makes the two agree: fragment row 2 c is token c, row 2 c + 1 token 4 + c.
__device__ __forceinline__ int frag_token(int r) { return (r >> 1) + 4 * (r & 1); }

// One lane's share of a 16-token tile of K or V. Dimensions by fragment position:
//   4 bits K: lane (., c) has dimensions 32 c .. 32 c + 31, four of them per 16-wide step;
//   4 bits V: lane (r, .) has 16 r .. 16 r + 15, two of them per 16-high step;
//   bf16 K: 32 i + 8 c .. + 7 (i = 0..3), bf16 V: 8 r .. + 7 and 64 + 8 r .. + 7.
template <bool KV4>
struct KTile;
template <bool KV4>
struct VTile;

template <>
struct KTile<true> {
  uint4 w[2];
  uint32_t sb[2];  // two scale bytes each
  __device__ __forceinline__ void load(const CacheDecodeArgs& a, size_t row0, int left, int r, int c) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = frag_token(r) + 8 * h;
      const size_t row = row0 + t;
      w[h] = make_uint4(0u, 0u, 0u, 0u);
      sb[h] = 0u;
      if (t < left) {
        w[h] = ld_stream16(static_cast<const uint8_t*>(a.k) + row * kCodeBytes + 16 * c);
        sb[h] = *reinterpret_cast<const uint16_t*>(a.k_scales + row * kRowScales + 2 * c);
      }
    }
  }
};

template <>
struct VTile<true> {
  uint2 w[4];
  uint32_t sb[4];
  __device__ __forceinline__ void load(const CacheDecodeArgs& a, size_t row0, int left, int r, int c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 4 * i + c;
      const size_t row = row0 + t;
      w[i] = make_uint2(0u, 0u);
      sb[i] = 0u;
      if (t < left) {
        w[i] = ld_stream8(static_cast<const uint8_t*>(a.v) + row * kCodeBytes + 8 * r);
        sb[i] = a.v_scales[row * kRowScales + r];
      }
    }
  }
};

template <>
struct KTile<false> {
  uint4 w[2][4];
  __device__ __forceinline__ void load(const CacheDecodeArgs& a, size_t row0, int left, int r, int c) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = frag_token(r) + 8 * h;
      const bf16* p = static_cast<const bf16*>(a.k) + (row0 + t) * kHeadDim + 8 * c;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[h][i] = t < left ? ld_stream16(p + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
};

template <>
struct VTile<false> {
  uint4 w[4][2];
  __device__ __forceinline__ void load(const CacheDecodeArgs& a, size_t row0, int left, int r, int c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 4 * i + c;
      const bf16* p = static_cast<const bf16*>(a.v) + (row0 + t) * kHeadDim + 8 * r;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        w[i][h] = t < left ? ld_stream16(p + 64 * h) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
};

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// S^T (16 tokens x 8 heads) of a K tile with the Q fragments.
__device__ __forceinline__ void scores_of(const KTile<true>& k, const uint2 (&q)[8], float (&s)[4]) {
  uint32_t sc[2][2];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const uint32_t x = ((k.sb[h] >> (8 * b)) & 0xffu) << 7;
      sc[h][b] = x | (x << 16);
    }
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // 8 dimensions: two 16-wide steps
    uint32_t lo[4], hi[4];
    codes_to_half2(word_of(k.w[0], i), lo);
    codes_to_half2(word_of(k.w[1], i), hi);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      lo[e] = hmul2(lo[e], sc[0][i >> 1]);
      hi[e] = hmul2(hi[e], sc[1][i >> 1]);
    }
    mma16816<true>(s, lo[0], hi[0], lo[1], hi[1], q[2 * i].x, q[2 * i].y);
    mma16816<true>(s, lo[2], hi[2], lo[3], hi[3], q[2 * i + 1].x, q[2 * i + 1].y);
  }
}

__device__ __forceinline__ void scores_of(const KTile<false>& k, const uint2 (&q)[8], float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    mma16816<false>(s, k.w[0][i].x, k.w[1][i].x, k.w[0][i].y, k.w[1][i].y, q[2 * i].x, q[2 * i].y);
    mma16816<false>(s, k.w[0][i].z, k.w[1][i].z, k.w[0][i].w, k.w[1][i].w, q[2 * i + 1].x,
                    q[2 * i + 1].y);
  }
}

// O^T += V^T P^T; p[row half][head of the pair] are the probabilities of this lane's S^T entries.
// 4 bits: P in fp16 (11 significant bits; p <= 2^15, see kCdShift), V exact in fp16.
__device__ __forceinline__ void accumulate(const VTile<true>& v, const float (&p)[4], float (&o)[8][4]) {
  const __half2 p0 = __floats2half2_rn(p[0], p[1]), p1 = __floats2half2_rn(p[2], p[3]);
  const uint32_t b0 = transpose8x8(*reinterpret_cast<const uint32_t*>(&p0));
  const uint32_t b1 = transpose8x8(*reinterpret_cast<const uint32_t*>(&p1));
  const uint32_t s01 = (v.sb[0] << 7) | (v.sb[1] << 23), s23 = (v.sb[2] << 7) | (v.sb[3] << 23);
  constexpr uint32_t m = 0x0f0f0f0fu;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const uint32_t w0 = w ? v.w[0].y : v.w[0].x, w1 = w ? v.w[1].y : v.w[1].x;
    const uint32_t w2 = w ? v.w[2].y : v.w[2].x, w3 = w ? v.w[3].y : v.w[3].x;
    uint32_t e01[4], d01[4], e23[4], d23[4];  // even and odd dimensions, tokens side by side
    codes_to_half2((w0 & m) | ((w1 << 4) & ~m), e01);
    codes_to_half2(((w0 >> 4) & m) | (w1 & ~m), d01);
    codes_to_half2((w2 & m) | ((w3 << 4) & ~m), e23);
    codes_to_half2(((w2 >> 4) & m) | (w3 & ~m), d23);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      mma16816<true>(o[4 * w + e], hmul2(e01[e], s01), hmul2(d01[e], s01), hmul2(e23[e], s23),
                     hmul2(d23[e], s23), b0, b1);
  }
}

// bf16: V is bf16, so P is too, as the sum of two bf16 numbers (17 significant bits): the second
// product is free under the cache's bytes and keeps P's rounding out of the result.
__device__ __forceinline__ void accumulate(const VTile<false>& v, const float (&p)[4], float (&o)[8][4]) {
  const __nv_bfloat162 h0 = __floats2bfloat162_rn(p[0], p[1]), h1 = __floats2bfloat162_rn(p[2], p[3]);
  const float2 f0 = __bfloat1622float2(h0), f1 = __bfloat1622float2(h1);
  const uint32_t b0 = transpose8x8(*reinterpret_cast<const uint32_t*>(&h0));
  const uint32_t b1 = transpose8x8(*reinterpret_cast<const uint32_t*>(&h1));
  const uint32_t c0 = transpose8x8(pack_bf16x2(p[0] - f0.x, p[1] - f0.y));
  const uint32_t c1 = transpose8x8(pack_bf16x2(p[2] - f1.x, p[3] - f1.y));
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t w0 = word_of(v.w[0][j >> 2], j & 3), w1 = word_of(v.w[1][j >> 2], j & 3);
    const uint32_t w2 = word_of(v.w[2][j >> 2], j & 3), w3 = word_of(v.w[3][j >> 2], j & 3);
    const uint32_t a0 = __byte_perm(w0, w1, 0x5410), a1 = __byte_perm(w0, w1, 0x7632);
    const uint32_t a2 = __byte_perm(w2, w3, 0x5410), a3 = __byte_perm(w2, w3, 0x7632);
    mma16816<false>(o[j], a0, a1, a2, a3, b0, b1);
    mma16816<false>(o[j], a0, a1, a2, a3, c0, c1);
  }
}

// Dimension of row r (hi: r + 8) of the j-th 16-high step of O^T.
template <bool KV4>
__device__ __forceinline__ int out_dim(int j, int r, int hi) {
  return KV4 ? 16 * r + 2 * j + hi : 64 * (j >> 2) + 8 * r + 2 * (j & 3) + hi;
}

// The running maximum follows the true one only when that has grown by more than 2^kCdLazy, so
// most tiles need no exchange between lanes and no rescaling: p may then reach 2^(kCdLazy +
// kCdShift). 4 bits: the shift by 2^7 uses fp16's whole range for P (at most 2^15), so that a
// weight down to 2^-31 of the largest one counts in the product.
constexpr float kCdLazy = 8.0f;
template <bool KV4>
constexpr float kCdShift = KV4 ? 7.0f : 0.0f;

template <int G>
struct CdSmem {
  float m[kCdWarps][8];
  float l[kCdWarps][8];
  float o[kCdWarps][G][kHeadDim];
  float lse[8];
};

// Length that the attention sees, and whether the step's token is appended.
__device__ __forceinline__ int decode_length(const CacheDecodeArgs& a, int u, bool* append) {
  const int l = a.len[u];
  *append = a.new_k != nullptr && l >= 0 && l < a.cap;
  return *append ? l + 1 : max(0, min(l, a.cap));
}

// -(m + log2 l), to be added to a logit (log2 domain) of the same head; no tokens: no weight
__device__ __forceinline__ float neg_lse(float m, float l) {
  return l > 0.f ? -(m + log2f(l)) : (l == 0.f ? -INFINITY : l);
}

// weights of tokens [t0, t1) from their logits
template <int G>
__device__ __forceinline__ void add_weights(const float* logits, float* weights, int t0, int t1,
                                            const float* nlse) {
  float nl[G];
#pragma unroll
  for (int h = 0; h < G; ++h) nl[h] = nlse[h];
  for (int t = t0 + threadIdx.x; t < t1; t += kCdThreads) {
    const float* x = logits + (size_t)t * G;
    float s = 0.f;
#pragma unroll
    for (int h = 0; h < G; ++h) s += fast_exp2(x[h] + nl[h]);
    weights[t] += s;
  }
}

template <int G, bool KV4>
__global__ void __launch_bounds__(kCdThreads, 2) cache_decode_kernel(CacheDecodeArgs a) {
  __shared__ CdSmem<G> sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, c = lane & 3;
  const int ukv = blockIdx.x, split = blockIdx.y;
  const int u = ukv / a.n_kv, g = ukv - u * a.n_kv;
  bool append;
  const int L = decode_length(a, u, &append);
  if (split == 0 && g == 0 && tid == 0) {
    const int l = a.len[u];
    if (l < 0 || l > a.cap || (a.new_k && !append)) set_status(a.status, RKV_DEV_LEN_OVER_CAP);
    // (len_out that is len itself is written by the join kernel, after every reader)
    if (a.new_k && a.len_out != a.len) a.len_out[u] = append ? l + 1 : l;
  }
  const int tb = split * a.tokens_per_split;
  const int te = min(L, tb + a.tokens_per_split);

  if (KV4 && append && L - 1 >= tb && L - 1 < te) {  // this CTA's tokens include the new one
    if (tid < 16) {
      const bool v = tid >= 8;
      const int blk = tid & 7, at = L - 1;
      const size_t dst = a.pm.table
                             ? paged_row(a.pm, paged_block(a.pm, u, at, a.status), a.n_kv, g, at)
                             : (size_t)ukv * a.cap + at;
      uint32_t w[8], sb;
      load32((v ? a.new_v : a.new_k) + (size_t)ukv * kHeadDim + blk * kScaleGroup, w);
      const uint2 cd = quantise16(w, &sb);
      uint8_t* codes = static_cast<uint8_t*>(const_cast<void*>(v ? a.v : a.k));
      *reinterpret_cast<uint2*>(codes + dst * kCodeBytes + blk * 8) = cd;
      const_cast<uint8_t*>(v ? a.v_scales : a.k_scales)[dst * kRowScales + blk] = (uint8_t)sb;
    }
    __syncthreads();
  }

  // Q fragments: lane (r, c) holds head r. 4 bits: fp16, each head scaled by a power of two that
  // puts its largest value in [2^8, 2^9): then every bf16 value down to 2^-25 of it is exact, and
  // what is lost below is far under the fp32 rounding of the sum.
  uint2 q[8];
  float cs[2];  // logit scale of heads 2 c, 2 c + 1
  {
    const bf16* qr = a.q + ((size_t)ukv * G + r) * kHeadDim;
    uint2 x[8];
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int d = KV4 ? 32 * c + 4 * j : 32 * (j >> 1) + 8 * c + 4 * (j & 1);
      x[j] = r < G ? *reinterpret_cast<const uint2*>(qr + d) : make_uint2(0u, 0u);
      if (KV4) {
        amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(x[j].x)), fabsf(bf16_hi(x[j].x))));
        amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(x[j].y)), fabsf(bf16_hi(x[j].y))));
      }
    }
    if (KV4) {
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // exponent of amax, kept where both 2^(8 - e) and 2^(e - 8) are normal numbers
      const int e = max(-110, min(126, (int)(__float_as_uint(amax) >> 23) - 127));
      const float up = __uint_as_float((uint32_t)(127 + 8 - e) << 23);
      const float down = a.scale_log2 * __uint_as_float((uint32_t)(127 - 8 + e) << 23);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const __half2 lo = __floats2half2_rn(bf16_lo(x[j].x) * up, bf16_hi(x[j].x) * up);
        const __half2 hi = __floats2half2_rn(bf16_lo(x[j].y) * up, bf16_hi(x[j].y) * up);
        q[j] = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                          *reinterpret_cast<const uint32_t*>(&hi));
      }
      cs[0] = __shfl_sync(0xffffffffu, down, 8 * c);
      cs[1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = x[j];
      cs[0] = cs[1] = a.scale_log2;
    }
  }

  float m[2] = {-1e30f, -1e30f}, l[2] = {0.f, 0.f}, o[8][4];
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  float* logits = a.weights ? a.logits + (size_t)ukv * a.cap * G : nullptr;

  auto row_of = [&](int t0) -> size_t {  // row of the first token of a tile (it lies in one block)
    return a.pm.table ? paged_row(a.pm, paged_block(a.pm, u, t0, a.status), a.n_kv, g, t0)
                      : (size_t)ukv * a.cap + t0;
  };
  KTile<KV4> kt;
  VTile<KV4> vt;
  int t0 = tb + warp * kCdTile;
  if (t0 < te) {
    const size_t row = row_of(t0);
    kt.load(a, row, te - t0, r, c);
    vt.load(a, row, te - t0, r, c);
  }
  while (t0 < te) {
    const int left = te - t0, tn = t0 + kCdRound;
    const size_t next = tn < te ? row_of(tn) : 0;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    scores_of(kt, q, s);
    if (tn < te) kt.load(a, next, te - tn, r, c);
    const int ra = frag_token(r), rb = ra + 8;
    s[0] = ra < left ? s[0] * cs[0] : -INFINITY;
    s[1] = ra < left ? s[1] * cs[1] : -INFINITY;
    s[2] = rb < left ? s[2] * cs[0] : -INFINITY;
    s[3] = rb < left ? s[3] * cs[1] : -INFINITY;
    if (logits) {
      if (2 * c < G) {
        float* x = logits + (size_t)(t0 + ra) * G + 2 * c;
        if (G == 1) {
          if (ra < left) x[0] = s[0];
          if (rb < left) x[8 * G] = s[2];
        } else {
          if (ra < left) *reinterpret_cast<float2*>(x) = make_float2(s[0], s[1]);
          if (rb < left) *reinterpret_cast<float2*>(x + 8 * G) = make_float2(s[2], s[3]);
        }
      }
    }
    float mt0 = fmaxf(s[0], s[2]), mt1 = fmaxf(s[1], s[3]);
    if (__any_sync(0xffffffffu, mt0 > m[0] + kCdLazy || mt1 > m[1] + kCdLazy)) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        mt0 = fmaxf(mt0, __shfl_xor_sync(0xffffffffu, mt0, d));
        mt1 = fmaxf(mt1, __shfl_xor_sync(0xffffffffu, mt1, d));
      }
      mt0 = fmaxf(mt0, m[0]);
      mt1 = fmaxf(mt1, m[1]);
      const float f0 = fast_exp2(m[0] - mt0), f1 = fast_exp2(m[1] - mt1);
      m[0] = mt0;
      m[1] = mt1;
      l[0] *= f0;
      l[1] *= f1;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        o[j][0] *= f0;
        o[j][1] *= f1;
        o[j][2] *= f0;
        o[j][3] *= f1;
      }
    }
    const float b0 = kCdShift<KV4> - m[0], b1 = kCdShift<KV4> - m[1];
    const float p[4] = {fast_exp2(s[0] + b0), fast_exp2(s[1] + b1), fast_exp2(s[2] + b0),
                        fast_exp2(s[3] + b1)};
    l[0] += p[0] + p[2];
    l[1] += p[1] + p[3];
    accumulate(vt, p, o);
    if (tn < te) vt.load(a, next, te - tn, r, c);
    t0 = tn;
  }

  // join the warps: lane (r, c) holds dimensions out_dim(., r, .) of heads 2 c, 2 c + 1
#pragma unroll
  for (int d = 4; d < 32; d <<= 1) {
    l[0] += __shfl_xor_sync(0xffffffffu, l[0], d);
    l[1] += __shfl_xor_sync(0xffffffffu, l[1], d);
  }
  if (r == 0) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      sm.m[warp][2 * c + e] = m[e];
      sm.l[warp][2 * c + e] = l[e];
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int h = 2 * c + (e & 1);
      if (h < G) sm.o[warp][h][out_dim<KV4>(j, r, e >> 1)] = o[j][e];
    }
  __syncthreads();
  for (int i = tid; i < G * kHeadDim; i += kCdThreads) {
    const int h = i / kHeadDim, d = i % kHeadDim;
    float M = -1e30f, S = 0.f, O = 0.f;
#pragma unroll
    for (int w = 0; w < kCdWarps; ++w) M = fmaxf(M, sm.m[w][h]);
#pragma unroll
    for (int w = 0; w < kCdWarps; ++w) {
      const float f = fast_exp2(sm.m[w][h] - M);
      S = fmaf(sm.l[w][h], f, S);
      O = fmaf(sm.o[w][h][d], f, O);
    }
    M -= kCdShift<KV4>;  // p was 2^(s - m + shift)
    if (a.nsplit == 1) {
      a.out[((size_t)ukv * G + h) * kHeadDim + d] = __float2bfloat16_rn(S == 0.f ? 0.f : O / S);
      if (d == 0) sm.lse[h] = neg_lse(M, S);
    } else {
      const size_t row = ((size_t)ukv * a.nsplit + split) * G + h;
      a.part_o[row * kHeadDim + d] = O;
      if (d == 0) reinterpret_cast<float2*>(a.part_ml)[row] = make_float2(M, S);
    }
  }
  if (a.nsplit == 1 && a.weights) {
    __syncthreads();
    add_weights<G>(logits, a.weights + (size_t)ukv * a.cap, tb, te, sm.lse);
  }
}

// Joins the splits: blockIdx.y = 0 writes the outputs (and a length that is its own input), the
// others turn kCdWeightChunk logits at a time into weights.
template <int G>
__global__ void __launch_bounds__(kCdThreads) cache_join_kernel(CacheDecodeArgs a) {
  __shared__ float nlse[8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ukv = blockIdx.x, u = ukv / a.n_kv;
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml) + (size_t)ukv * a.nsplit * G;
  bool append;
  int L;
  if (a.new_k && a.len_out != a.len) {
    L = max(0, min(a.len_out[u], a.cap));
  } else {
    L = decode_length(a, u, &append);
  }
  if (blockIdx.y == 0) {
    if (a.nsplit == 1) return;
    const float* po = a.part_o + (size_t)ukv * a.nsplit * G * kHeadDim;
    for (int i = tid; i < G * kHeadDim; i += kCdThreads) {
      const int h = i / kHeadDim;
      float M = -1e30f, S = 0.f, O = 0.f;
      for (int s = 0; s < a.nsplit; ++s) M = fmaxf(M, ml[s * G + h].x);
      for (int s = 0; s < a.nsplit; ++s) {
        const float2 x = ml[s * G + h];
        const float f = fast_exp2(x.x - M);
        S = fmaf(x.y, f, S);
        O = fmaf(po[(size_t)s * G * kHeadDim + i], f, O);
      }
      a.out[(size_t)ukv * G * kHeadDim + i] = __float2bfloat16_rn(S == 0.f ? 0.f : O / S);
    }
    return;
  }
  const int first = (blockIdx.y - 1) * kCdWeightChunk;
  if (first >= L) return;
  if (warp < G) {
    float M = -1e30f, S = 0.f;
    for (int s = lane; s < a.nsplit; s += 32) M = fmaxf(M, ml[s * G + warp].x);
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 8));
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 4));
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 2));
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 1));
    for (int s = lane; s < a.nsplit; s += 32) {
      const float2 x = ml[s * G + warp];
      S = fmaf(x.y, fast_exp2(x.x - M), S);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) S += __shfl_xor_sync(0xffffffffu, S, d);
    if (lane == 0) nlse[warp] = neg_lse(M, S);
  }
  __syncthreads();
  for (int t0 = first; t0 < L; t0 += (int)(gridDim.y - 1) * kCdWeightChunk)
    add_weights<G>(a.logits + (size_t)ukv * a.cap * G, a.weights + (size_t)ukv * a.cap, t0,
                   min(L, t0 + kCdWeightChunk), nlse);
}

// A length that is its own input moves on after every reader.
__global__ void cache_length_kernel(CacheDecodeArgs a) {
  const int u = blockIdx.x * blockDim.x + threadIdx.x;
  if (u >= a.n) return;
  bool append;
  const int L = decode_length(a, u, &append);
  if (append) a.len_out[u] = L;
}

template <int G>
static cudaError_t launch_group(const CacheDecodeArgs& a, cudaStream_t s) {
  const dim3 grid(a.n * a.n_kv, a.nsplit);
  if (a.kv4)
    cache_decode_kernel<G, true><<<grid, kCdThreads, 0, s>>>(a);
  else
    cache_decode_kernel<G, false><<<grid, kCdThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (a.nsplit > 1) {
    const int chunks = a.weights ? (a.cap + kCdWeightChunk - 1) / kCdWeightChunk : 0;
    cache_join_kernel<G><<<dim3(a.n * a.n_kv, 1 + (chunks < 4096 ? chunks : 4096)), kCdThreads, 0, s>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (a.new_k && a.len_out == a.len) {
    cache_length_kernel<<<(a.n + 255) / 256, 256, 0, s>>>(a);
    e = cudaGetLastError();
  }
  return e;
}

cudaError_t launch_cache_decode(const CacheDecodeArgs& a, cudaStream_t s) {
  switch (a.gqa) {
    case 1: return launch_group<1>(a, s);
    case 2: return launch_group<2>(a, s);
    case 4: return launch_group<4>(a, s);
    case 8: return launch_group<8>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace rkv
