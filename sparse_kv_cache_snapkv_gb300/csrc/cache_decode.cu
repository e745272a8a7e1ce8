// Append to and decode over a cache held in 4 bits, and the bf16 decode that also accumulates each
// token's attention weight (sm_103a).
//
// Decode, per (unit, KV head) with its G query heads and tokens j < L:
//   s_hj = scale q_h . K_j,  p_hj = exp(s_hj - m_h),  out_h = (sum_j p_hj V_j) / l_h,
//   weights_j += sum_h p_hj / l_h
// in one pass over K and V: each warp takes 16 tokens at a time with a running maximum and sum;
// the warps of a CTA, then the CTAs of a split sequence, are joined. The weights need the final
// sums, so the products (4 G bytes per token against 144 or 512 of K and V) are kept in the
// workspace and turned into weights once those are known.
//
// Measured against the bytes at the copy rate: 32 units of 32K in 4 bits, 8 heads, G = 4, with weights
// 233 us of 188; one unit of 131071 tokens 39.6 of 23.5; 16 ragged paged units of up to 20K, 4 heads,
// G = 8, 39 of 18; 16 ragged bf16 units of up to 32K with weights 229 of 208.
//
// Both products run on mma.sync m16n8k16 with the tokens (S^T = K Q^T) or the dimensions
// (O^T = V^T P^T) as the 16 rows and the query heads as the 8 columns: no row of the tile is
// padding at G = 8, and S^T leaves its maximum, its sum and P^T in the very lanes that hold the
// same heads' columns of O^T. A decode is bound by the cache's bytes; a tcgen05 tile of 128 rows
// would need the operands unpacked into shared memory first, which costs more than the product.
//
// A fragment's columns may be any permutation of the dimensions as long as Q has the same one, and
// its rows any permutation of the tokens, so every lane unpacks 16 contiguous bytes of K codes and 8
// of V straight into fragments. A 4-bit tile (2304 bytes) is copied to its warp's own ring in
// shared memory a step of two tiles ahead; bf16 fragments come from global memory directly.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "cache4.cuh"
#include "common.cuh"
#include "rkv_internal.h"
#include "tensor_core.cuh"

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

// The block that a new token goes to, -1 where the table's entry is none: block 0, read in its place
// elsewhere, may be another sequence's.
__device__ __forceinline__ int append_block(const PagedMap& m, int u, int t, uint32_t* status) {
  const int b = m.table[(size_t)u * m.max_blocks + t / m.block];
  if (b >= 0 && b < m.num_blocks) return b;
  set_status(status, RKV_DEV_BAD_INDEX);
  return -1;
}

// One thread = one block of 16 values (32 bytes in, 8 + 1 out); blockIdx.y: K or V. Bound by the
// copy: 8 neighbouring threads make one row of codes and one of scales.
__global__ void __launch_bounds__(kAppendThreads) kv4_append_kernel(Kv4AppendArgs a) {
  pdl_wait();
  pdl_trigger();
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
    // (len_out that is also an input is written by kv4_length_kernel, after every reader)
    if (a.len_out != a.len && a.len_out != a.new_len) a.len_out[u] = have + max(t, 0);
  }
  if (i >= t) return;
  const int at = have + i;
  size_t dst;
  bool there = true;
  if (a.pm.table) {
    const int b = append_block(a.pm, u, at, a.status);
    there = b >= 0;
    dst = paged_row(a.pm, b, a.n_kv, g, at);
  } else {
    dst = (size_t)ukv * a.cap + at;
  }
  const size_t src = (size_t)row * kHeadDim + blk * kScaleGroup;
  uint32_t w[8], sb;
  load32((v ? a.new_v : a.new_k) + src, w);
  const uint2 c = quantise16(w, &sb);
  if (there) {
    *reinterpret_cast<uint2*>((v ? a.v_codes : a.k_codes) + dst * kCodeBytes + blk * 8) = c;
    (v ? a.v_scales : a.k_scales)[dst * kRowScales + blk] = (uint8_t)sb;
  }
  if (a.k_values) {
    values16(c, sb, w);
    store32((v ? a.v_values : a.k_values) + src, w);
  }
}

__global__ void kv4_length_kernel(Kv4AppendArgs a) {
  pdl_wait();
  pdl_trigger();
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
  const cudaError_t e = launch_pdl_kernel(kv4_append_kernel, dim3((unsigned)ctas, 2),
                                          dim3(kAppendThreads), 0, s, a);
  if (e != cudaSuccess || (a.len_out != a.len && a.len_out != a.new_len)) return e;
  return launch_pdl_kernel(kv4_length_kernel, dim3((a.n + 255) / 256), dim3(256), 0, s, a);
}

// ==========================================================================================
// decode
// ==========================================================================================
// The work of a call is the sequence of all (unit, KV head)s' rounds of kCdRound tokens; CTA i of C
// takes the i-th of C equal parts of it, whatever the lengths are. A part is a run of segments, each
// within one (unit, KV head); only its first and its last can be shared with other CTAs, so two
// slots of partial results per CTA are enough. A second kernel joins the parts in their order, turns
// the kept products into weights and moves the lengths on, after every reader; nothing in the workspace has
// to hold anything before a call. (A CTA that came last at a counter could join in place: 32 units of
// 32K with weights took 242 us so, 231 as here, and the counters had to be zero before a call.)
constexpr int kCdThreads = 256;
constexpr int kCdWarps = kCdThreads / 32;
constexpr int kCdTile = 16;                   // tokens of a fragment tile
constexpr int kCdPerSm = 2;                   // CTAs that an SM holds
// Tokens that a warp takes at a time: two tiles of 4 bits (their products are independent, and the
// bookkeeping of a step is shared), one of bf16; and that a CTA takes at a time.
template <bool KV4>
constexpr int kCdStep = KV4 ? 2 * kCdTile : kCdTile;
template <bool KV4>
constexpr int kCdRound = kCdStep<KV4>* kCdWarps;
constexpr int kCdWeightChunk = 1024;          // tokens that a CTA turns into weights at a time
constexpr int kCdWeightCtasPerSm = 8;

// CTAs of a call: one per slot of the SMs; where that leaves a part fewer than kCdMinRounds rounds,
// the same number for each (unit, KV head), so that parts of equal lengths end with them.
constexpr int kCdMinRounds = 2;
constexpr int kCdMostCtas = 512;  // the joins have room for the factors of as many parts
static long long cache_decode_slots() {
  const int s = kCdPerSm * device_sm_count();
  return s < kCdMostCtas ? s : kCdMostCtas;
}
static int cache_decode_ctas(int n, int n_kv, int cap, bool kv4) {
  const int round = kv4 ? kCdRound<true> : kCdRound<false>;
  const long long units = (long long)n * n_kv, rounds = (cap + round - 1) / round;
  const long long slots = cache_decode_slots();
  if (units * rounds >= slots * kCdMinRounds || units >= slots) return (int)slots;
  const long long each = slots / units;
  return (int)(units * (each < rounds ? each : rounds));
}

// Room for the parts of every call of no larger sizes: a workspace for the largest shape serves all (the
// number of CTAs itself falls where more units, or more rows, make a part for each of them longer).
static size_t most_ctas(int n, int n_kv, int cap) {
  const long long units = (long long)n * n_kv, rounds = (cap + kCdRound<false> - 1) / kCdRound<false>;
  const long long slots = cache_decode_slots();
  return (size_t)(units * rounds < slots ? units * rounds : slots);
}

struct CacheScratch {
  size_t units, ml, cs, part_ml, part_o, logits, total;
};
static CacheScratch cache_scratch(int n, int n_kv, int gqa, int cap, bool with_weights) {
  const size_t units = (size_t)n * n_kv;
  const size_t slots = 2 * most_ctas(n, n_kv, cap);
  CacheScratch c;
  c.units = 0;
  c.ml = align_up(((size_t)n + 1) * sizeof(CdUnit), 256);
  c.cs = c.ml + align_up(units * gqa * 8, 256);
  c.part_ml = c.cs + align_up(units * gqa * 4, 256);
  c.part_o = c.part_ml + align_up(slots * gqa * 8, 256);
  c.logits = c.part_o + align_up(slots * gqa * kHeadDim * 4, 256);
  c.total = c.logits + (with_weights ? align_up(units * cap * gqa * 4, 256) : 0);
  return c;
}

size_t cache_decode_scratch_bytes(int n, int n_kv, int gqa, int cap, bool with_weights) {
  return cache_scratch(n, n_kv, gqa, cap, with_weights).total;
}

void cache_decode_carve(CacheDecodeArgs* a, void* scratch) {
  unsigned char* p = static_cast<unsigned char*>(scratch);
  const CacheScratch c = cache_scratch(a->n, a->n_kv, a->gqa, a->cap, a->weights != nullptr);
  a->unit = reinterpret_cast<CdUnit*>(p + c.units);
  a->ml = reinterpret_cast<float*>(p + c.ml);
  a->cs = reinterpret_cast<float*>(p + c.cs);
  a->part_ml = reinterpret_cast<float*>(p + c.part_ml);
  a->part_o = reinterpret_cast<float*>(p + c.part_o);
  a->logits = reinterpret_cast<float*>(p + c.logits);
}

// A load that does not stay in L1 (the cache is read once).
__device__ __forceinline__ uint4 ld_stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
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

// Lane roles of the fragments: r = lane / 4, c = lane % 4. Row s of a 16-token tile's fragment is
// token frag_token(s) (and s + 8 is frag_token(s) + 8): as rows of K, lane (r, c) holds parts of
// tokens frag_token(r) and + 8; as columns of V^T, tokens frag_token(2 c), frag_token(2 c + 1) and
// both + 8. The order makes the shared-memory reads below free of bank conflicts: rows are 64
// bytes, so two tokens of different parity make one 128-byte line.
__device__ __forceinline__ int frag_token(int s) { return s ^ ((s >> 1) & 1); }

// One warp's 16-token tile of a 4-bit cache in shared memory, as it lies in the cache but for V,
// whose rows' 16-byte quarters are swapped in pairs in every other four tokens (again for the
// banks). Dimensions by fragment position: K lane (., c): 32 c .. 32 c + 31, four per 16-wide step;
// V lane (r, .): 16 r .. 16 r + 15, two per 16-high step.
struct __align__(16) Kv4Tile {
  uint8_t k[kCdTile * kCodeBytes];
  uint8_t v[kCdTile * kCodeBytes];
  uint8_t ks[kCdTile * kRowScales];
  uint8_t vs[kCdTile * kRowScales];
};

// A lane's part of the copies of a tile: where it reads (from the tile's first row) and writes.
struct Kv4Lane {
  const uint8_t *k, *v, *s;  // this lane's 16 bytes of the codes, 8 of the scales, at row 0
  uint32_t dk, dv, ds;       // the same in a Kv4Tile
  int row, srow;             // rows they belong to (the second 16 bytes: row + 8)
  __device__ __forceinline__ void init(const CacheDecodeArgs& a, int lane) {
    row = lane >> 2;
    srow = lane & 15;
    k = static_cast<const uint8_t*>(a.k) + 16 * lane;
    v = static_cast<const uint8_t*>(a.v) + 16 * lane;
    s = (lane < 16 ? a.k_scales : a.v_scales) + 8 * srow;
    dk = 16 * lane;
    dv = 1024 + row * kCodeBytes + 16 * ((lane & 3) ^ ((row >> 1) & 2));
    ds = 2048 + 8 * lane;
  }
  // a whole tile; pk, pv, ps: k, v and s moved to its first row
  __device__ __forceinline__ void full(uint32_t tile, const uint8_t* pk, const uint8_t* pv,
                                       const uint8_t* ps) const {
    copy16(tile + dk, pk);
    copy16(tile + dk + 512, pk + 512);
    copy16(tile + dv, pv);
    copy16(tile + dv + 512, pv + 512);
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(tile + ds), "l"(ps) : "memory");
  }
  // the first `left` rows of it (0 or less: none), zeros for the others, which are not touched
  __device__ __forceinline__ void part(uint32_t tile, size_t at, int left) const {
    const bool lo = row < left, hi = row + 8 < left, sc = srow < left;
    const uint8_t *pk = k + at * kCodeBytes, *pv = v + at * kCodeBytes, *ps = s + at * kRowScales;
    zfill16(tile + dk, lo ? pk : k, lo);
    zfill16(tile + dk + 512, hi ? pk + 512 : k, hi);
    zfill16(tile + dv, lo ? pv : v, lo);
    zfill16(tile + dv + 512, hi ? pv + 512 : v, hi);
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(tile + ds), "l"(sc ? ps : s),
                 "r"(sc ? 8 : 0)
                 : "memory");
  }
  static __device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  }
  static __device__ __forceinline__ void zfill16(uint32_t dst, const void* src, bool read) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(read ? 16 : 0)
                 : "memory");
  }
};

// A scale byte as the same fp16 number twice; two bytes as a pair.
__device__ __forceinline__ uint32_t scale_twice(uint32_t b) { return b * 0x00800080u; }
__device__ __forceinline__ uint32_t scale_pair(uint32_t lo, uint32_t hi) {
  return (hi * 65536u + lo) * 128u;
}

// S^T (16 tokens x 8 heads) of a tile with the Q fragments.
__device__ __forceinline__ void scores_kv4(const Kv4Tile* t, const uint2 (&q)[8], int r, int c,
                                           float (&s)[4]) {
  const int ta = frag_token(r);
  const uint4 wa = *reinterpret_cast<const uint4*>(t->k + ta * kCodeBytes + 16 * c);
  const uint4 wb = *reinterpret_cast<const uint4*>(t->k + (ta + 8) * kCodeBytes + 16 * c);
  const uint32_t sa[2] = {scale_twice(t->ks[ta * kRowScales + 2 * c]),
                          scale_twice(t->ks[ta * kRowScales + 2 * c + 1])};
  const uint32_t sb[2] = {scale_twice(t->ks[(ta + 8) * kRowScales + 2 * c]),
                          scale_twice(t->ks[(ta + 8) * kRowScales + 2 * c + 1])};
  const uint32_t aw[4] = {wa.x, wa.y, wa.z, wa.w}, bw[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // 8 dimensions: two 16-wide steps
    uint32_t lo[4], hi[4];
    codes_to_half2(aw[i], lo);
    codes_to_half2(bw[i], hi);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      lo[e] = hmul2(lo[e], sa[i >> 1]);
      hi[e] = hmul2(hi[e], sb[i >> 1]);
    }
    mma16816<true>(s, lo[0], hi[0], lo[1], hi[1], q[2 * i].x, q[2 * i].y);
    mma16816<true>(s, lo[2], hi[2], lo[3], hi[3], q[2 * i + 1].x, q[2 * i + 1].y);
  }
}

// With at most four heads, columns 4 to 7 of the fragments hold the heads of columns 0 to 3 once more.
template <int G>
constexpr bool kCdTwice = G <= 4;

// O^T += V^T P^T; p are the probabilities of this lane's S^T entries (at most 2^15: see kCdShift).
// V is exact in fp16; P is the sum of two fp16 numbers (22 significant bits), as the bf16 form's is of
// two bf16: the first alone left the outputs off by up to 2^-11 of sum_j p_j |v_j|, which shows where
// they cancel. The second numbers are in columns 4 to 7 where those repeat the heads (32 units of 32K,
// G = 4: 233.1 us; P in one fp16 232.7, a second product 245.1), else in a product of their own (16 ragged
// paged units, G = 8: 39.1 us, P in one fp16 36.6).
template <int G>
__device__ __forceinline__ void accumulate_kv4(const Kv4Tile* t, const float (&p)[4], int r, int c,
                                               float (&o)[8][4]) {
  __half2 p0 = __floats2half2_rn(p[0], p[1]), p1 = __floats2half2_rn(p[2], p[3]);
  const float2 f0 = __half22float2(p0), f1 = __half22float2(p1);
  const __half2 l0 = __floats2half2_rn(p[0] - f0.x, p[1] - f0.y);
  const __half2 l1 = __floats2half2_rn(p[2] - f1.x, p[3] - f1.y);
  if (kCdTwice<G> && c >= 2) {
    p0 = l0;
    p1 = l1;
  }
  const uint32_t b0 = transpose8x8(*reinterpret_cast<const uint32_t*>(&p0));
  const uint32_t b1 = transpose8x8(*reinterpret_cast<const uint32_t*>(&p1));
  uint32_t c0 = 0u, c1 = 0u;
  if (!kCdTwice<G>) {
    c0 = transpose8x8(*reinterpret_cast<const uint32_t*>(&l0));
    c1 = transpose8x8(*reinterpret_cast<const uint32_t*>(&l1));
  }
  const int t0 = frag_token(2 * c), t1 = frag_token(2 * c + 1);
  const uint8_t* v0 = t->v + t0 * kCodeBytes + 16 * ((r >> 1) ^ ((t0 >> 1) & 2)) + 8 * (r & 1);
  const uint8_t* v1 = t->v + t1 * kCodeBytes + 16 * ((r >> 1) ^ ((t1 >> 1) & 2)) + 8 * (r & 1);
  const uint2 x0 = *reinterpret_cast<const uint2*>(v0), x1 = *reinterpret_cast<const uint2*>(v1);
  const uint2 x2 = *reinterpret_cast<const uint2*>(v0 + 512), x3 = *reinterpret_cast<const uint2*>(v1 + 512);
  const uint8_t* s = t->vs + r;
  const uint32_t s01 = scale_pair(s[t0 * kRowScales], s[t1 * kRowScales]);
  const uint32_t s23 = scale_pair(s[(t0 + 8) * kRowScales], s[(t1 + 8) * kRowScales]);
  constexpr uint32_t m = 0x0f0f0f0fu;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const uint32_t w0 = w ? x0.y : x0.x, w1 = w ? x1.y : x1.x;
    const uint32_t w2 = w ? x2.y : x2.x, w3 = w ? x3.y : x3.x;
    uint32_t e01[4], d01[4], e23[4], d23[4];  // even and odd dimensions, tokens side by side
    codes_to_half2((w0 & m) | ((w1 << 4) & ~m), e01);
    codes_to_half2(((w0 >> 4) & m) | (w1 & ~m), d01);
    codes_to_half2((w2 & m) | ((w3 << 4) & ~m), e23);
    codes_to_half2(((w2 >> 4) & m) | (w3 & ~m), d23);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t a0 = hmul2(e01[e], s01), a1 = hmul2(d01[e], s01);
      const uint32_t a2 = hmul2(e23[e], s23), a3 = hmul2(d23[e], s23);
      mma16816<true>(o[4 * w + e], a0, a1, a2, a3, b0, b1);
      if (!kCdTwice<G>) mma16816<true>(o[4 * w + e], a0, a1, a2, a3, c0, c1);
    }
  }
}

// The bf16 cache needs no unpacking: its fragments come straight from global memory, each lane's
// next K requested as soon as S^T is done and its next V after O^T. Dimensions by fragment
// position: K lane (., c): 32 i + 8 c .. + 7 (i = 0..3); V lane (r, .): 8 r .. + 7, 64 + 8 r .. + 7.
struct BfTile {
  uint4 k[2][4];
  uint4 v[4][2];
  __device__ __forceinline__ void load_k(const CacheDecodeArgs& a, size_t row, int left, int r, int c) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = frag_token(r) + 8 * h;
      const bf16* p = static_cast<const bf16*>(a.k) + (row + t) * kHeadDim + 8 * c;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        k[h][i] = t < left ? ld_stream16(p + 32 * i) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __device__ __forceinline__ void load_v(const CacheDecodeArgs& a, size_t row, int left, int r, int c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = frag_token(2 * c + (i & 1)) + 8 * (i >> 1);
      const bf16* p = static_cast<const bf16*>(a.v) + (row + t) * kHeadDim + 8 * r;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        v[i][h] = t < left ? ld_stream16(p + 64 * h) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
};

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

__device__ __forceinline__ void scores_bf(const BfTile& t, const uint2* q, float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint2 q0 = q[64 * i], q1 = q[64 * i + 32];
    mma16816<false>(s, t.k[0][i].x, t.k[1][i].x, t.k[0][i].y, t.k[1][i].y, q0.x, q0.y);
    mma16816<false>(s, t.k[0][i].z, t.k[1][i].z, t.k[0][i].w, t.k[1][i].w, q1.x, q1.y);
  }
}

// V is bf16, so P is too, as the sum of two bf16 numbers (16 significant bits): the second product
// is free under the cache's bytes and keeps P's rounding out of the result.
__device__ __forceinline__ void accumulate_bf(const BfTile& t, const float (&p)[4], float (&o)[8][4]) {
  const __nv_bfloat162 h0 = __floats2bfloat162_rn(p[0], p[1]), h1 = __floats2bfloat162_rn(p[2], p[3]);
  const float2 f0 = __bfloat1622float2(h0), f1 = __bfloat1622float2(h1);
  const uint32_t b0 = transpose8x8(*reinterpret_cast<const uint32_t*>(&h0));
  const uint32_t b1 = transpose8x8(*reinterpret_cast<const uint32_t*>(&h1));
  const uint32_t c0 = transpose8x8(pack_bf16x2(p[0] - f0.x, p[1] - f0.y));
  const uint32_t c1 = transpose8x8(pack_bf16x2(p[2] - f1.x, p[3] - f1.y));
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t w0 = word_of(t.v[0][j >> 2], j & 3), w1 = word_of(t.v[1][j >> 2], j & 3);
    const uint32_t w2 = word_of(t.v[2][j >> 2], j & 3), w3 = word_of(t.v[3][j >> 2], j & 3);
    const uint32_t a0 = __byte_perm(w0, w1, 0x5410), a1 = __byte_perm(w0, w1, 0x7632);
    const uint32_t a2 = __byte_perm(w2, w3, 0x5410), a3 = __byte_perm(w2, w3, 0x7632);
    mma16816<false>(o[j], a0, a1, a2, a3, b0, b1);
    mma16816<false>(o[j], a0, a1, a2, a3, c0, c1);
  }
}

// A (unit, KV head)'s outputs are joined in the order of the fragments: output i is head i % G and
// dimension out_dim(i / G). i / G = 8 (2 j + hi) + r for row r (hi: r + 8) of O^T's j-th step.
template <bool KV4>
__device__ __forceinline__ int out_dim(int x) {
  const int jh = x >> 3, r = x & 7;
  return KV4 ? 16 * r + jh : 64 * (jh >> 3) + 8 * r + (jh & 7);
}

// The running maximum follows the true one only when that has grown by more than 2^kCdLazy, so
// most tiles need no exchange between lanes and no rescaling: p may then reach 2^(kCdLazy +
// kCdShift). 4 bits: the shift by 2^7 uses fp16's whole range for P (at most 2^15), so that a
// weight down to 2^-31 of the largest one counts in the product.
constexpr float kCdLazy = 8.0f;
template <bool KV4>
constexpr float kCdShift = KV4 ? 7.0f : 0.0f;
template <bool KV4>
constexpr float kCdUnshift = KV4 ? 0x1p-7f : 1.0f;  // (a part's O and sum carry the shift)

// A warp's softmax state: maxima and sums of heads 2 c and 2 c + 1 (the sums per lane), O^T.
struct CdState {
  float m[2], l[2], o[8][4];
  __device__ __forceinline__ void clear() {
    m[0] = m[1] = -1e30f;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  }
};

// NT tiles' products -> their probabilities, after the maximum has followed. The products (their
// factors cs make logits in the log2 domain of them; rows past the end -inf) are kept for the weights
// at `logits`, which is the step's first row. cs meets them only in a multiply-add with the maximum:
// a product rounded by itself would be off by 2^-24 of a logit, not of a difference of two.
template <int G, bool KV4, int NT>
__device__ __forceinline__ void softmax_step(CdState& st, float (&s)[NT][4], const float (&cs)[2],
                                             int left, int r, int c, float* logits) {
  const int ta = frag_token(r);
  if (left < NT * kCdTile) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (ta + 16 * n >= left) s[n][0] = s[n][1] = -INFINITY;
      if (ta + 16 * n + 8 >= left) s[n][2] = s[n][3] = -INFINITY;
    }
  }
  if (logits && 2 * c < G) {
    float* x = logits + ta * G + 2 * c;
#pragma unroll
    for (int n = 0; n < 2 * NT; ++n) {  // eight rows each
      if (ta + 8 * n < left) {
        if (G == 1)
          x[8 * n] = s[n >> 1][2 * (n & 1)];
        else
          *reinterpret_cast<float2*>(x + 8 * n * G) =
              make_float2(s[n >> 1][2 * (n & 1)], s[n >> 1][2 * (n & 1) + 1]);
      }
    }
  }
  float m0 = fmaxf(s[0][0], s[0][2]), m1 = fmaxf(s[0][1], s[0][3]);
#pragma unroll
  for (int n = 1; n < NT; ++n) {
    m0 = fmaxf(m0, fmaxf(s[n][0], s[n][2]));
    m1 = fmaxf(m1, fmaxf(s[n][1], s[n][3]));
  }
  m0 *= cs[0];
  m1 *= cs[1];
  if (__any_sync(0xffffffffu, m0 > st.m[0] + kCdLazy || m1 > st.m[1] + kCdLazy)) {
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, d));
      m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, d));
    }
    m0 = fmaxf(m0, st.m[0]);
    m1 = fmaxf(m1, st.m[1]);
    const float f0 = fast_exp2(st.m[0] - m0), f1 = fast_exp2(st.m[1] - m1);
    st.m[0] = m0;
    st.m[1] = m1;
    st.l[0] *= f0;
    st.l[1] *= f1;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      st.o[j][0] *= f0;
      st.o[j][1] *= f1;
      st.o[j][2] *= f0;
      st.o[j][3] *= f1;
    }
  }
  const float b0 = kCdShift<KV4> - st.m[0], b1 = kCdShift<KV4> - st.m[1];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    s[n][0] = fast_exp2(fmaf(s[n][0], cs[0], b0));
    s[n][1] = fast_exp2(fmaf(s[n][1], cs[1], b1));
    s[n][2] = fast_exp2(fmaf(s[n][2], cs[0], b0));
    s[n][3] = fast_exp2(fmaf(s[n][3], cs[1], b1));
    st.l[0] += s[n][0] + s[n][2];
    st.l[1] += s[n][1] + s[n][3];
  }
}

// Length that the attention sees, and whether the step's token is appended.
__device__ __forceinline__ int decode_length(const CacheDecodeArgs& a, int u, bool* append) {
  const int l = a.len[u];
  *append = a.new_k != nullptr && l >= 0 && l < a.cap;
  return *append ? l + 1 : max(0, min(l, a.cap));
}

__device__ __forceinline__ CdUnit unit_of(const CacheDecodeArgs& a, int u, long long at) {
  bool append;
  const int l = a.len[u], L = decode_length(a, u, &append);
  return CdUnit{at, L, append ? l + 1 : l, l < 0 || l > a.cap || (a.new_k && !append), 0};
}

// What a head's probabilities are divided by: 1 / l, no weight where there are no tokens.
__device__ __forceinline__ float over(float l) { return l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l); }

// kCdWeightChunk tokens' weights 2^(cs x - m) / l from their products x and what is known of the heads;
// the loads can be on their way before that is.
struct CdHead {
  float cs, m, over;
};
template <int G>
struct CdWeights {
  static constexpr int kU = kCdWeightChunk / kCdThreads;  // tokens of a thread
  float x[kU][G], w[kU];
  __device__ __forceinline__ void load(const float* logits, const float* weights, int t0, int L) {
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int t = t0 + k * kCdThreads + (int)threadIdx.x;
      if (t < L) {
        const float* src = logits + (size_t)t * G;
        w[k] = weights[t];
        if (G % 4 == 0) {
#pragma unroll
          for (int h = 0; h < G; h += 4) {
            const float4 y = *reinterpret_cast<const float4*>(src + h);
            x[k][h] = y.x;
            x[k][h + 1] = y.y;
            x[k][h + 2] = y.z;
            x[k][h + 3] = y.w;
          }
        } else {
#pragma unroll
          for (int h = 0; h < G; ++h) x[k][h] = src[h];
        }
      }
    }
  }
  __device__ __forceinline__ void add(const CdHead* head, float* weights, int t0, int L) const {
    CdHead hd[G];
#pragma unroll
    for (int h = 0; h < G; ++h) hd[h] = head[h];
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int t = t0 + k * kCdThreads + (int)threadIdx.x;
      if (t < L) {
        float s = 0.f;
#pragma unroll
        for (int h = 0; h < G; ++h) s = fmaf(fast_exp2(fmaf(x[k][h], hd[h].cs, -hd[h].m)), hd[h].over, s);
        weights[t] = w[k] + s;
      }
    }
  }
};

// Joining the warps: their O^T fragments as they are (row (j, e), lane), padded so that neither the
// lanes' stores nor the reads meet in a bank more than twice.
constexpr int kCdORow = 34;
struct CdMerge {
  float m[kCdWarps][8];
  float l[kCdWarps][8];
  float o[kCdWarps][32 * kCdORow];
};
// two steps of two tiles per warp: one read, one on its way (a third step in flight: 32 units of 32K
// 243 us instead of 231)
constexpr int kCdRing = 2;
// the ring and the warps' join use the same memory one after the other
template <bool KV4>
constexpr size_t kCdSmemBytes = KV4 ? (size_t)kCdWarps * kCdRing * 2 * sizeof(Kv4Tile) : sizeof(CdMerge);
static_assert(kCdSmemBytes<true> >= sizeof(CdMerge), "the warps' join fits in the ring");

// Where a CTA begins: its first round's unit, KV head and round, and how much there is in all.
struct CdStart {
  long long total;  // rounds of the call
  long long begin, end;  // this CTA's part
  int ctas;         // CTAs with work
  int u, g, round;
};

template <bool KV4>
__device__ __forceinline__ int rounds_of(int L) {
  return (L + kCdRound<KV4> - 1) / kCdRound<KV4>;
}

// first round of CTA i of `ctas`, and the CTA that has round x
__device__ __forceinline__ long long part_begin(long long total, int ctas, int i) {
  return total * i / ctas;
}
__device__ __forceinline__ int part_of(long long total, int ctas, long long x) {
  return (int)(((x + 1) * ctas - 1) / total);
}

// Every CTA adds up the units' rounds (each thread a run of units) and finds its own part; the first
// writes down what it found of every unit, for the joins.
template <bool KV4>
__device__ __forceinline__ void find_start(const CacheDecodeArgs& a, CdStart* out,
                                           unsigned long long* tmp) {
  const int tid = threadIdx.x;
  if (a.n <= 32) {  // one warp, no barrier but the last
    if (tid < 32) {
      bool ap;
      const int R = tid < a.n ? rounds_of<KV4>(decode_length(a, tid, &ap)) : 0;
      const int incl = warp_incl_scan(R);  // (32 units of at most 2^23 rounds)
      const long long total = (long long)__shfl_sync(0xffffffffu, incl, 31) * a.n_kv;
      const int ctas = (int)min((long long)gridDim.x, total);
      const bool work = (int)blockIdx.x < ctas;
      const long long b = work ? total * blockIdx.x / ctas : 0;
      const long long at = (long long)(incl - R) * a.n_kv;
      if (tid == 0) {
        out->total = total;
        out->ctas = ctas;
        out->begin = b;
        out->end = work ? total * (blockIdx.x + 1) / ctas : 0;
      }
      if (blockIdx.x == 0) {
        if (tid < a.n) a.unit[tid] = unit_of(a, tid, at);
        if (tid == 0) a.unit[a.n] = CdUnit{total, 0, 0, 0, 0};
      }
      if (work && b >= at && b < at + (long long)R * a.n_kv) {
        out->u = tid;
        out->g = (int)((b - at) / R);
        out->round = (int)((b - at) - (long long)out->g * R);
      }
    }
    __syncthreads();
    return;
  }
  const int per = (a.n + kCdThreads - 1) / kCdThreads;
  const int u0 = min(a.n, tid * per), u1 = min(a.n, u0 + per);
  bool ap;
  unsigned long long mine = 0;
  for (int u = u0; u < u1; ++u) mine += rounds_of<KV4>(decode_length(a, u, &ap));
  const unsigned long long before = block_excl_scan64(mine, tmp);
  if (tid == kCdThreads - 1) out->total = (long long)(before + mine) * a.n_kv;
  __syncthreads();
  const long long total = out->total;
  if (blockIdx.x == 0) {
    long long at = (long long)before * a.n_kv;
    for (int u = u0; u < u1; ++u) {
      a.unit[u] = unit_of(a, u, at);
      at += (long long)rounds_of<KV4>(decode_length(a, u, &ap)) * a.n_kv;
    }
    if (tid == 0) a.unit[a.n] = CdUnit{total, 0, 0, 0, 0};
  }
  const int ctas = (int)min((long long)gridDim.x, total);
  if (ctas == 0 || (int)blockIdx.x >= ctas) {
    if (tid == 0) out->ctas = ctas;
    if (tid == 0) out->begin = out->end = 0;
  } else {
    const long long b = total * blockIdx.x / ctas;
    if (tid == 0) {
      out->ctas = ctas;
      out->begin = b;
      out->end = total * (blockIdx.x + 1) / ctas;
    }
    long long at = (long long)before * a.n_kv;
    if (b >= at && b < at + (long long)mine * a.n_kv) {
      for (int u = u0; u < u1; ++u) {
        const int R = rounds_of<KV4>(decode_length(a, u, &ap));
        const long long all = (long long)R * a.n_kv;
        if (b < at + all) {
          out->u = u;
          out->g = (int)((b - at) / R);
          out->round = (int)((b - at) - (long long)out->g * R);
          break;
        }
        at += all;
      }
    }
  }
  __syncthreads();
}

template <int G, bool KV4, bool PAGED>
__global__ void __launch_bounds__(kCdThreads, kCdPerSm) cache_decode_kernel(CacheDecodeArgs a) {
  // (the ring begins on a sector: where two lanes' 16 bytes of one sector of the cache do not make one
  // sector here, each is fetched by itself, and the 32 units of 32K took 280 us instead of 231)
  extern __shared__ __align__(128) unsigned char dyn[];
  __shared__ CdStart start;
  __shared__ unsigned long long scan[33];
  __shared__ uint2 qf[KV4 ? 1 : 8 * 32];
  CdMerge& mg = *reinterpret_cast<CdMerge*>(dyn);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = lane >> 2, c = lane & 3;
  bool append;
  pdl_wait();

  find_start<KV4>(a, &start, scan);
  constexpr int kStep = kCdStep<KV4>, kRound = kCdRound<KV4>;
  Kv4Tile* ring = reinterpret_cast<Kv4Tile*>(dyn) + warp * (2 * kCdRing);
  Kv4Lane my;
  if (KV4) my.init(a, lane);
  int u = start.u, g = start.g, round = start.round;
  bool first = true;
  for (long long at = start.begin; at < start.end; first = false) {
    const int L = decode_length(a, u, &append);
    const int R = rounds_of<KV4>(L);
    if (R == 0) {  // (a unit without tokens)
      ++u;
      continue;
    }
    const int rounds = (int)min((long long)(R - round), start.end - at);
    const int ukv = u * a.n_kv + g;
    const int tb = round * kCdRound<KV4>, te = min(L, (round + rounds) * kCdRound<KV4>);
    const bool whole = rounds == R;

    if (KV4 && append && round + rounds == R) {  // this segment's tokens include the new one
      if (tid < 16) {
        const bool v = tid >= 8;
        const int blk = tid & 7, row = L - 1;
        const int b = PAGED ? append_block(a.pm, u, row, a.status) : 0;
        const size_t dst = PAGED ? paged_row(a.pm, b, a.n_kv, g, row) : (size_t)ukv * a.cap + row;
        uint32_t w[8], sb;
        load32((v ? a.new_v : a.new_k) + (size_t)ukv * kHeadDim + blk * kScaleGroup, w);
        const uint2 cd = quantise16(w, &sb);
        uint8_t* codes = static_cast<uint8_t*>(const_cast<void*>(v ? a.v : a.k));
        if (b >= 0) {
          *reinterpret_cast<uint2*>(codes + dst * kCodeBytes + blk * 8) = cd;
          const_cast<uint8_t*>(v ? a.v_scales : a.k_scales)[dst * kRowScales + blk] = (uint8_t)sb;
        }
        __threadfence();
      }
      __syncthreads();
    }

    auto row_of = [&](int t) -> size_t {  // row of the first token of a tile (it lies in one block)
      return PAGED ? paged_row(a.pm, paged_block(a.pm, u, t, a.status), a.n_kv, g, t)
                   : (size_t)ukv * a.cap + t;
    };
    int t0 = tb + warp * kStep;
    // (contiguous: addresses of the next step's first row)
    const uint8_t* pk = my.k + ((size_t)ukv * a.cap + t0) * kCodeBytes;
    const uint8_t* pv = my.v + ((size_t)ukv * a.cap + t0) * kCodeBytes;
    const uint8_t* ps = my.s + ((size_t)ukv * a.cap + t0) * kRowScales;
    // the copies of the step from token t (one commit group, empty past the end)
    auto fetch = [&](int t, int place) {
      const uint32_t dst = smem_addr(ring + 2 * place);
      if (te - t >= kStep) {
        if (PAGED) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const size_t row = row_of(t + h * kCdTile);
            my.full(dst + h * sizeof(Kv4Tile), my.k + row * kCodeBytes, my.v + row * kCodeBytes,
                    my.s + row * kRowScales);
          }
        } else {
          my.full(dst, pk, pv, ps);
          my.full(dst + sizeof(Kv4Tile), pk + kCdTile * kCodeBytes, pv + kCdTile * kCodeBytes,
                  ps + kCdTile * kRowScales);
          pk += kRound * kCodeBytes;
          pv += kRound * kCodeBytes;
          ps += kRound * kRowScales;
        }
      } else if (t < te) {
        my.part(dst, row_of(t), te - t);
        my.part(dst + sizeof(Kv4Tile), te - t > kCdTile ? row_of(t + kCdTile) : 0, te - t - kCdTile);
      }
      cp_async_commit();
    };
    if (KV4) fetch(t0, 0);

    // Q fragments: lane (r, c) holds head r (kCdTwice: r % 4). 4 bits: fp16, each head scaled by a
    // power of two that puts its largest value in [2^8, 2^9): then every bf16 value down to 2^-25 of it
    // is exact, and what is lost below is far under the fp32 rounding of the sum.
    uint2 q[KV4 ? 8 : 1];
    float cs[2] = {a.scale_log2, a.scale_log2};  // logit scale of heads 2 c, 2 c + 1
    const int hr = KV4 && kCdTwice<G> ? r & 3 : r;
    const bf16* qr = a.q + ((size_t)ukv * G + hr) * kHeadDim;
    if (KV4) {
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        q[j] = hr < G ? *reinterpret_cast<const uint2*>(qr + 32 * c + 4 * j) : make_uint2(0u, 0u);
        amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(q[j].x)), fabsf(bf16_hi(q[j].x))));
        amax = fmaxf(amax, fmaxf(fabsf(bf16_lo(q[j].y)), fabsf(bf16_hi(q[j].y))));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // exponent of amax, kept where both 2^(8 - e) and 2^(e - 8) are normal numbers
      const int e = max(-110, min(126, (int)(__float_as_uint(amax) >> 23) - 127));
      const float up = __uint_as_float((uint32_t)(127 + 8 - e) << 23);
      const float down = a.scale_log2 * __uint_as_float((uint32_t)(127 - 8 + e) << 23);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const __half2 lo = __floats2half2_rn(bf16_lo(q[j].x) * up, bf16_hi(q[j].x) * up);
        const __half2 hi = __floats2half2_rn(bf16_lo(q[j].y) * up, bf16_hi(q[j].y) * up);
        q[j] = make_uint2(*reinterpret_cast<const uint32_t*>(&lo),
                          *reinterpret_cast<const uint32_t*>(&hi));
      }
      cs[0] = __shfl_sync(0xffffffffu, down, 8 * c);
      cs[1] = __shfl_sync(0xffffffffu, down, 8 * c + 4);
    } else {
      if (warp == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          qf[(j % (KV4 ? 1 : 8)) * 32 + lane] =
              r < G ? *reinterpret_cast<const uint2*>(qr + 32 * (j >> 1) + 8 * c + 4 * (j & 1))
                    : make_uint2(0u, 0u);
      }
      __syncthreads();
    }

    // (a factor of zero would make NaN of a masked product; below this every logit is zero)
    cs[0] = fmaxf(cs[0], 0x1p-126f);
    cs[1] = fmaxf(cs[1], 0x1p-126f);
    if (a.weights && round == 0 && warp == 0 && r == 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (2 * c + e < G) a.cs[(size_t)ukv * G + 2 * c + e] = cs[e];
    }

    CdState st;
    st.clear();
    float* logits = a.weights ? a.logits + ((size_t)ukv * a.cap + t0) * G : nullptr;
    if (KV4) {
      for (int place = 0; t0 < te; t0 += kRound) {
        cp_async_wait_all();
        __syncwarp();  // this step has landed for every lane, and every lane is done with the last
        fetch(t0 + kRound, place ^ 1);
        const Kv4Tile* t = ring + 2 * place;
        place ^= 1;
        float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        scores_kv4(t, reinterpret_cast<const uint2(&)[8]>(q), r, c, s[0]);
        scores_kv4(t + 1, reinterpret_cast<const uint2(&)[8]>(q), r, c, s[1]);
        softmax_step<G, true, 2>(st, s, cs, te - t0, r, c, logits);
        if (logits) logits += kRound * G;
        accumulate_kv4<G>(t, s[0], r, c, st.o);
        accumulate_kv4<G>(t + 1, s[1], r, c, st.o);
      }
    } else {
      BfTile t;
      if (t0 < te) {
        const size_t row = row_of(t0);
        t.load_k(a, row, te - t0, r, c);
        t.load_v(a, row, te - t0, r, c);
      }
      for (; t0 < te; t0 += kRound) {
        const int tn = t0 + kRound;
        const size_t next = tn < te ? row_of(tn) : 0;
        float s[1][4] = {{0.f, 0.f, 0.f, 0.f}};
        scores_bf(t, qf + lane, s[0]);
        if (tn < te) t.load_k(a, next, te - tn, r, c);
        softmax_step<G, false, 1>(st, s, cs, te - t0, r, c, logits);
        if (logits) logits += kRound * G;
        accumulate_bf(t, s[0], st.o);
        if (tn < te) t.load_v(a, next, te - tn, r, c);
      }
    }

    // join the warps: lane (r, c) holds dimensions out_dim(., r, .) of heads 2 c, 2 c + 1
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) {
      st.l[0] += __shfl_xor_sync(0xffffffffu, st.l[0], d);
      st.l[1] += __shfl_xor_sync(0xffffffffu, st.l[1], d);
    }
    __syncthreads();  // the join's memory is the ring's
    if (r == 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mg.m[warp][2 * c + e] = st.m[e];
        mg.l[warp][2 * c + e] = st.l[e];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) mg.o[warp][(4 * j + e) * kCdORow + lane] = st.o[j][e];
    __syncthreads();
    const size_t slot = 2 * (size_t)blockIdx.x + (first ? 0 : 1);
    {
      // a thread's outputs all belong to one head
      const int h = tid % G;
      float f[kCdWarps], M = -1e30f, S = 0.f;
#pragma unroll
      for (int w = 0; w < kCdWarps; ++w) M = fmaxf(M, mg.m[w][h]);
#pragma unroll
      for (int w = 0; w < kCdWarps; ++w) {
        f[w] = fast_exp2(mg.m[w][h] - M);
        S = fmaf(mg.l[w][h], f[w], S);
      }
      const float inv = S == 0.f ? 0.f : 1.f / S;
#pragma unroll
      for (int i0 = 0; i0 < G * kHeadDim; i0 += kCdThreads) {
        const int i = i0 + tid, x = i / G, jh = x >> 3, row = x & 7;
        if (G * kHeadDim % kCdThreads != 0 && i >= G * kHeadDim) break;
        const int at = (2 * jh + (h & 1)) * kCdORow + 4 * row + (h >> 1);  // 4 j + e, e = 2 hi + h % 2
        float O = 0.f;
#pragma unroll
        for (int w = 0; w < kCdWarps; ++w)
          O = fmaf(KV4 && kCdTwice<G> ? mg.o[w][at] + mg.o[w][at + 2] : mg.o[w][at], f[w], O);
        if (whole)
          a.out[((size_t)ukv * G + h) * kHeadDim + out_dim<KV4>(x)] = __float2bfloat16_rn(O * inv);
        else
          a.part_o[slot * G * kHeadDim + i] = O;
      }
      if (tid < G) {
        if (whole)
          reinterpret_cast<float2*>(a.ml)[(size_t)ukv * G + tid] = make_float2(M, S * kCdUnshift<KV4>);
        else
          reinterpret_cast<float2*>(a.part_ml)[slot * G + tid] = make_float2(M, S);
      }
    }

    __syncthreads();  // shared memory is used again
    at += rounds;
    round = 0;
    if (++g == a.n_kv) {
      g = 0;
      ++u;
    }
  }

  // (a launch that follows may take this CTA's place from here; from the start, 1021 tokens took 8.2 us
  // instead of 7.8)
  pdl_trigger();
}

// The joins: blockIdx.y = 0 the outputs and the length, the others kCdWeightChunk tokens' weights.
// `ctas`: CTAs of the decode's launch.
template <int G, bool KV4>
__global__ void __launch_bounds__(kCdThreads) cache_join_kernel(CacheDecodeArgs a, int ctas) {
  __shared__ float4 sums[kCdThreads];
  __shared__ float factor[kCdMostCtas * G];
  __shared__ float total_s[8];
  __shared__ CdHead head[8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ukv = blockIdx.x, u = ukv / a.n_kv, g = ukv - u * a.n_kv;
  // (no early trigger: the next launch's CTAs would wait in these CTAs' places, 1021 tokens 8.4 us
  // instead of 8.2)
  pdl_wait();
  const CdUnit un = a.unit[u];
  const long long total = a.unit[a.n].at;
  const int L = un.length, R = rounds_of<KV4>(L);
  if (blockIdx.y == 0) {
    if (g == 0 && tid == 0) {
      if (un.bad) set_status(a.status, RKV_DEV_LEN_OVER_CAP);
      if (a.len_out) a.len_out[u] = un.next;
    }
    if (L == 0)
      for (int i = tid; i < G * kHeadDim; i += kCdThreads)
        a.out[(size_t)ukv * G * kHeadDim + i] = __float2bfloat16_rn(0.f);
  }
  int t0 = ((int)blockIdx.y - 1) * kCdWeightChunk;
  if (t0 >= L || L == 0) return;
  const float* logits = a.logits + (size_t)ukv * a.cap * G;
  float* weights = a.weights + (size_t)ukv * a.cap;
  CdWeights<G> cw;
  if (blockIdx.y > 0) cw.load(logits, weights, t0, L);
  // the parts that share this (unit, KV head): those of its first and its last round
  ctas = (int)min((long long)ctas, total);
  const long long z0 = un.at + (long long)g * R;
  const int i0 = part_of(total, ctas, z0), parts = part_of(total, ctas, z0 + R - 1) - i0 + 1;
  if (parts == 1) {  // (its outputs are written)
    if (blockIdx.y == 0) return;
    if (tid < G) {
      const float2 x = reinterpret_cast<const float2*>(a.ml)[(size_t)ukv * G + tid];
      head[tid] = CdHead{a.cs[(size_t)ukv * G + tid], x.x, over(x.y)};
    }
  }
  const size_t s0 = 2 * (size_t)i0 + (part_begin(total, ctas, i0) == z0 ? 0 : 1);
  auto slot_of = [&](int k) { return k == 0 ? s0 : 2 * (size_t)(i0 + k); };
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
  if (parts > 1 && warp < G) {
    const float2 mine = lane < parts ? ml[slot_of(lane) * G + warp] : make_float2(-1e30f, 0.f);
    float M = mine.x, S = 0.f;
    for (int k = lane + 32; k < parts; k += 32) M = fmaxf(M, ml[slot_of(k) * G + warp].x);
#pragma unroll
    for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    for (int k = lane; k < parts; k += 32) {
      const float2 x = k == lane ? mine : ml[slot_of(k) * G + warp];
      const float f = fast_exp2(x.x - M);
      factor[k * G + warp] = f;
      S = fmaf(x.y, f, S);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) S += __shfl_xor_sync(0xffffffffu, S, d);
    if (lane == 0) {
      total_s[warp] = S;
      if (blockIdx.y > 0) head[warp] = CdHead{a.cs[(size_t)ukv * G + warp], M, over(S * kCdUnshift<KV4>)};
    }
  }
  __syncthreads();
  if (blockIdx.y > 0) {
    cw.add(head, weights, t0, L);
    const int step = ((int)gridDim.y - 1) * kCdWeightChunk;
    for (t0 += step; t0 < L; t0 += step) {
      cw.load(logits, weights, t0, L);
      cw.add(head, weights, t0, L);
    }
    return;
  }
  // four outputs per thread; with fewer than eight heads the threads also share the parts
  constexpr int kQuads = G * kHeadDim / 4, kShare = kCdThreads / kQuads;
  const int quad = tid % kQuads, share = tid / kQuads;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int k = share; k < parts; k += kShare) {
    const float4 x = reinterpret_cast<const float4*>(a.part_o + slot_of(k) * G * kHeadDim)[quad];
    float f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = factor[k * G + (4 * quad + e) % G];
    o.x = fmaf(x.x, f[0], o.x);
    o.y = fmaf(x.y, f[1], o.y);
    o.z = fmaf(x.z, f[2], o.z);
    o.w = fmaf(x.w, f[3], o.w);
  }
  if (kShare > 1) {
    sums[tid] = o;
    __syncthreads();
    if (share == 0)
      for (int e = 1; e < kShare; ++e) {
        const float4 x = sums[e * kQuads + quad];
        o.x += x.x;
        o.y += x.y;
        o.z += x.z;
        o.w += x.w;
      }
  }
  if (share == 0) {
    const float y[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 4 * quad + e, h = i % G;
      const float S = total_s[h];
      a.out[((size_t)ukv * G + h) * kHeadDim + out_dim<KV4>(i / G)] =
          __float2bfloat16_rn(S == 0.f ? 0.f : y[e] / S);
    }
  }
}

template <int G, bool KV4, bool PAGED>
static cudaError_t launch_group(const CacheDecodeArgs& a, cudaStream_t s) {
  const int ctas = cache_decode_ctas(a.n, a.n_kv, a.cap, KV4);
  constexpr size_t smem = kCdSmemBytes<KV4>;
  cudaError_t e = ensure_dyn_smem((const void*)cache_decode_kernel<G, KV4, PAGED>, smem);
  if (e != cudaSuccess) return e;
  e = launch_pdl_kernel(cache_decode_kernel<G, KV4, PAGED>, dim3(ctas), dim3(kCdThreads), smem, s, a);
  if (e != cudaSuccess) return e;
  // weights: CTAs for eight per SM, since each has the sums to find first (32 units of 32K: four per SM
  // 237 us, eight 231, sixteen 232, a CTA per chunk 237)
  const int units = a.n * a.n_kv, chunks = (a.cap + kCdWeightChunk - 1) / kCdWeightChunk;
  const int fill = (kCdWeightCtasPerSm * device_sm_count() + units - 1) / units;
  const int y = a.weights ? (chunks < fill ? chunks : fill) : 0;
  return launch_pdl_kernel(cache_join_kernel<G, KV4>, dim3(units, 1 + y), dim3(kCdThreads), 0, s, a, ctas);
}

template <int G>
static cudaError_t launch_kind(const CacheDecodeArgs& a, cudaStream_t s) {
  if (!a.kv4) return launch_group<G, false, false>(a, s);
  return a.pm.table ? launch_group<G, true, true>(a, s) : launch_group<G, true, false>(a, s);
}

cudaError_t launch_cache_decode(const CacheDecodeArgs& a, cudaStream_t s) {
  switch (a.gqa) {
    case 1: return launch_kind<1>(a, s);
    case 2: return launch_kind<2>(a, s);
    case 4: return launch_kind<4>(a, s);
    case 8: return launch_kind<8>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace rkv
