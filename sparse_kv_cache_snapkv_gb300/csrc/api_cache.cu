// C ABI of the 4-bit cache and of eviction by accumulated attention weight: argument validation,
// workspace carving, kernel launches. The contract of every entry point is in include/rkv.h.
#include <cuda_runtime.h>
#include <climits>
#include <cmath>
#include <cstdint>

#include "../../include/rkv.h"
#include "../../include/rkv_testing.h"
#include "api_util.h"
#include "rkv_internal.h"

using namespace rkv;

namespace {

// n * n_kv * gqa CTAs or rows have to be countable in 31 bits
bool counts_ok(int n, int n_kv, int gqa) {
  return n > 0 && n_kv > 0 && gqa > 0 && (long long)n * n_kv <= INT_MAX / gqa;
}

// rows of a cache: token arithmetic stays within 31 bits
bool cap_ok(int cap) { return cap > 0 && cap <= (1 << 30); }

// positive, finite, and still both after the factor log2(e)
bool scale_ok(float s) { return s > 0.f && std::isfinite(s * kLog2e) && s * kLog2e > 0.f; }

bool kv4_ok(const void* a, const void* b, const void* c, const void* d) {
  return a && b && c && d && aligned16(a) && aligned16(b) && aligned16(c) && aligned16(d);
}

// a row's index is a 32-bit coordinate of the tensor maps
bool prompt_rows_ok(int n, int n_kv, int gqa, int max_q, int max_len) {
  return (long long)n * n_kv * gqa * max_q <= INT_MAX - 512 &&
         (long long)n * n_kv * max_len <= INT_MAX - 512;
}

rkv_status ws_check(const void* ws, size_t ws_bytes, size_t need) {
  if (need == 0) return RKV_ERR_INVALID_ARG;
  return ws && aligned16(ws) && ws_bytes >= need ? RKV_OK : RKV_ERR_WORKSPACE;
}

void* after_status(void* ws) { return static_cast<unsigned char*>(ws) + kStatusBytes; }

rkv_status append_impl(const void* new_k, const void* new_v, const int32_t* new_len, int n,
                       int n_kv, int head_dim, int max_new, void* k_codes, void* k_scales,
                       void* v_codes, void* v_scales, const PagedMap& pm, int cap,
                       const int32_t* len, int32_t* len_out, void* k_values, void* v_values,
                       void* ws, size_t ws_bytes, void* stream) {
  if (head_dim != kHeadDim) return RKV_ERR_UNSUPPORTED;
  if (!new_k || !new_v || !aligned16(new_k) || !aligned16(new_v) || !len || !len_out ||
      !kv4_ok(k_codes, k_scales, v_codes, v_scales))
    return RKV_ERR_INVALID_ARG;
  if ((k_values == nullptr) != (v_values == nullptr) ||
      (k_values && (!aligned16(k_values) || !aligned16(v_values))))
    return RKV_ERR_INVALID_ARG;
  if (!counts_ok(n, n_kv, 1) || max_new <= 0 || !cap_ok(cap)) return RKV_ERR_INVALID_ARG;
  const rkv_status w = ws_check(ws, ws_bytes, rkv_kv4_append_workspace_bytes(n));
  if (w != RKV_OK) return w;
  Kv4AppendArgs a{};
  a.new_k = static_cast<const bf16*>(new_k);
  a.new_v = static_cast<const bf16*>(new_v);
  a.new_len = new_len;
  a.k_codes = static_cast<uint8_t*>(k_codes);
  a.k_scales = static_cast<uint8_t*>(k_scales);
  a.v_codes = static_cast<uint8_t*>(v_codes);
  a.v_scales = static_cast<uint8_t*>(v_scales);
  a.len = len;
  a.len_out = len_out;
  a.k_values = static_cast<bf16*>(k_values);
  a.v_values = static_cast<bf16*>(v_values);
  a.pm = pm;
  a.n = n;
  a.n_kv = n_kv;
  a.max_new = max_new;
  a.cap = cap;
  a.status = status_ptr(ws);
  return from_cuda(launch_kv4_append(a, as_stream(stream)));
}

rkv_status decode_impl(const CacheDecodeArgs& in, int head_dim, float scale, void* ws,
                       size_t ws_bytes, void* stream) {
  CacheDecodeArgs a = in;
  if (head_dim != kHeadDim || !gqa_ok(a.gqa)) return RKV_ERR_UNSUPPORTED;
  if (!a.q || !a.len || !a.out || !aligned16(a.q) || !aligned16(a.out)) return RKV_ERR_INVALID_ARG;
  if (a.kv4 ? !kv4_ok(a.k, a.k_scales, a.v, a.v_scales)
            : (!a.k || !a.v || !aligned16(a.k) || !aligned16(a.v) || !a.weights))
    return RKV_ERR_INVALID_ARG;
  if ((a.new_k == nullptr) != (a.new_v == nullptr) ||
      (a.new_k == nullptr) != (a.len_out == nullptr) ||
      (a.new_k && (!aligned16(a.new_k) || !aligned16(a.new_v))))
    return RKV_ERR_INVALID_ARG;
  if (a.weights && !aligned16(a.weights)) return RKV_ERR_INVALID_ARG;
  if (!counts_ok(a.n, a.n_kv, a.gqa) || !cap_ok(a.cap) || !scale_ok(scale))
    return RKV_ERR_INVALID_ARG;
  const rkv_status w =
      ws_check(ws, ws_bytes, rkv_kv4_decode_workspace_bytes(a.n, a.n_kv, a.gqa, a.cap,
                                                            a.weights != nullptr));
  if (w != RKV_OK) return w;
  a.scale_log2 = scale * kLog2e;
  a.status = status_ptr(ws);
  cache_decode_carve(&a, after_status(ws));
  return from_cuda(launch_cache_decode(a, as_stream(stream)));
}

rkv_status kv4_decode_impl(const void* q, const void* new_k, const void* new_v, void* k_codes,
                           void* k_scales, void* v_codes, void* v_scales, const PagedMap& pm,
                           const int32_t* len, int32_t* len_out, int n, int n_kv, int gqa,
                           int head_dim, int cap, float scale, void* out, float* weights,
                           void* ws, size_t ws_bytes, void* stream) {
  CacheDecodeArgs a{};
  a.q = static_cast<const bf16*>(q);
  a.k = k_codes;
  a.v = v_codes;
  a.k_scales = static_cast<const uint8_t*>(k_scales);
  a.v_scales = static_cast<const uint8_t*>(v_scales);
  a.len = len;
  a.len_out = len_out;
  a.new_k = static_cast<const bf16*>(new_k);
  a.new_v = static_cast<const bf16*>(new_v);
  a.pm = pm;
  a.n = n;
  a.n_kv = n_kv;
  a.gqa = gqa;
  a.cap = cap;
  a.out = static_cast<bf16*>(out);
  a.weights = weights;
  a.kv4 = true;
  return decode_impl(a, head_dim, scale, ws, ws_bytes, stream);
}

// a paged 4-bit cache: a 16-token tile must lie within one block
bool kv4_paged_ok(const void* table, int num_blocks, int block, int max_blocks) {
  return paged_ok(table, num_blocks, block, max_blocks) && block >= kMinKv4Block;
}

rkv_status evict_impl(EvictArgs a, int head_dim, void* ws, size_t ws_bytes, void* stream) {
  if (head_dim != kHeadDim) return RKV_ERR_UNSUPPORTED;
  for (int i = 0; i < 4; ++i)
    if (a.row_bytes[i] && (!a.rows[i] || !aligned16(a.rows[i]))) return RKV_ERR_INVALID_ARG;
  if (!a.len || !a.len_out || !a.weights || !a.weights_out || !a.pos || !a.pos_out || !a.seen)
    return RKV_ERR_INVALID_ARG;
  if (!counts_ok(a.n, a.n_kv, 1) || !cap_ok(a.cap) || a.keep <= 0 || a.recent < 0 ||
      a.recent > a.keep)
    return RKV_ERR_INVALID_ARG;
  const rkv_status w =
      ws_check(ws, ws_bytes, rkv_evict_workspace_bytes(a.n, a.n_kv, a.cap, a.keep));
  if (w != RKV_OK) return w;
  a.scratch = after_status(ws);
  a.status = status_ptr(ws);
  return from_cuda(launch_evict(a, as_stream(stream)));
}

rkv_status prompt_impl(const void* q, const int32_t* q_len, const void* k, const int32_t* len, int n,
                       int n_kv, int gqa, int head_dim, int max_q, int max_len, float scale,
                       float* weights, uint64_t wait_limit_ns, int test_skip, void* ws,
                       size_t ws_bytes, void* stream) {
  if (head_dim != kHeadDim || gqa > kMaxPromptGqa) return RKV_ERR_UNSUPPORTED;
  if (!q || !q_len || !k || !len || !weights || !aligned16(q) || !aligned16(k))
    return RKV_ERR_INVALID_ARG;
  if (!counts_ok(n, n_kv, gqa) || max_q <= 0 || max_len < max_q || !scale_ok(scale))
    return RKV_ERR_INVALID_ARG;
  if (!prompt_rows_ok(n, n_kv, gqa, max_q, max_len)) return RKV_ERR_TOO_LARGE;
  const rkv_status w =
      ws_check(ws, ws_bytes, rkv_prompt_weights_workspace_bytes(n, n_kv, gqa, max_q, max_len));
  if (w != RKV_OK) return w;
  PromptArgs a{};
  a.q = static_cast<const bf16*>(q);
  a.q_len = q_len;
  a.k = static_cast<const bf16*>(k);
  a.len = len;
  a.n = n;
  a.n_kv = n_kv;
  a.gqa = gqa;
  a.max_q = max_q;
  a.max_len = max_len;
  a.scale_log2 = scale * kLog2e;
  a.weights = weights;
  a.scratch = after_status(ws);
  a.status = status_ptr(ws);
  a.wait_limit_ns = wait_limit_ns;
  a.test_skip = test_skip;
  return from_cuda(launch_prompt_weights(a, as_stream(stream)));
}

EvictArgs evict_args(const int32_t* len, int32_t* len_out, const float* weights,
                     float* weights_out, const int32_t* pos, int32_t* pos_out,
                     const int32_t* seen, int n, int n_kv, int cap, int keep, int recent,
                     int32_t* src_rows) {
  EvictArgs a{};
  a.len = len;
  a.len_out = len_out;
  a.weights = weights;
  a.weights_out = weights_out;
  a.pos = pos;
  a.pos_out = pos_out;
  a.seen = seen;
  a.n = n;
  a.n_kv = n_kv;
  a.cap = cap;
  a.keep = keep;
  a.recent = recent;
  a.src_rows = src_rows;
  return a;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------------------- 4-bit cache
size_t rkv_kv4_append_workspace_bytes(int n) { return n > 0 ? kStatusBytes : 0; }

rkv_status rkv_kv4_append(const void* new_k, const void* new_v, const int32_t* new_len, int n,
                          int n_kv, int head_dim, int max_new, void* k_codes, void* k_scales,
                          void* v_codes, void* v_scales, int cap, const int32_t* len,
                          int32_t* len_out, void* k_values, void* v_values, void* ws,
                          size_t ws_bytes, void* stream) {
  RKV_TRACE();
  return append_impl(new_k, new_v, new_len, n, n_kv, head_dim, max_new, k_codes, k_scales,
                     v_codes, v_scales, PagedMap{}, cap, len, len_out, k_values, v_values, ws,
                     ws_bytes, stream);
}

rkv_status rkv_kv4_append_paged(const void* new_k, const void* new_v, const int32_t* new_len,
                                int n, int n_kv, int head_dim, int max_new, void* k_codes,
                                void* k_scales, void* v_codes, void* v_scales, int num_blocks,
                                int block, const int32_t* block_table, int max_blocks,
                                const int32_t* len, int32_t* len_out, void* k_values,
                                void* v_values, void* ws, size_t ws_bytes, void* stream) {
  RKV_TRACE();
  if (!kv4_paged_ok(block_table, num_blocks, block, max_blocks)) return RKV_ERR_INVALID_ARG;
  const PagedMap pm{block_table, max_blocks, block, num_blocks};
  return append_impl(new_k, new_v, new_len, n, n_kv, head_dim, max_new, k_codes, k_scales,
                     v_codes, v_scales, pm, max_blocks * block, len, len_out, k_values, v_values,
                     ws, ws_bytes, stream);
}

size_t rkv_kv4_decode_workspace_bytes(int n, int n_kv, int gqa, int cap, int with_weights) {
  if (!counts_ok(n, n_kv, gqa) || !gqa_ok(gqa) || !cap_ok(cap)) return 0;
  return kStatusBytes + cache_decode_scratch_bytes(n, n_kv, gqa, cap, with_weights != 0);
}

rkv_status rkv_kv4_decode(const void* q, const void* new_k, const void* new_v, void* k_codes,
                          void* k_scales, void* v_codes, void* v_scales, const int32_t* len,
                          int32_t* len_out, int n, int n_kv, int gqa, int head_dim, int cap,
                          float scale, void* out, float* weights, void* ws, size_t ws_bytes,
                          void* stream) {
  RKV_TRACE();
  return kv4_decode_impl(q, new_k, new_v, k_codes, k_scales, v_codes, v_scales, PagedMap{}, len,
                         len_out, n, n_kv, gqa, head_dim, cap, scale, out, weights, ws, ws_bytes,
                         stream);
}

rkv_status rkv_kv4_decode_paged(const void* q, const void* new_k, const void* new_v,
                                void* k_codes, void* k_scales, void* v_codes, void* v_scales,
                                const int32_t* block_table, const int32_t* len, int32_t* len_out,
                                int n, int n_kv, int gqa, int head_dim, int num_blocks, int block,
                                int max_blocks, float scale, void* out, float* weights, void* ws,
                                size_t ws_bytes, void* stream) {
  RKV_TRACE();
  if (!kv4_paged_ok(block_table, num_blocks, block, max_blocks)) return RKV_ERR_INVALID_ARG;
  const PagedMap pm{block_table, max_blocks, block, num_blocks};
  return kv4_decode_impl(q, new_k, new_v, k_codes, k_scales, v_codes, v_scales, pm, len, len_out,
                         n, n_kv, gqa, head_dim, max_blocks * block, scale, out, weights, ws,
                         ws_bytes, stream);
}

// ------------------------------------------------------------------------------- weights
size_t rkv_dense_decode_weights_workspace_bytes(int n, int n_kv, int gqa, int max_len) {
  return rkv_kv4_decode_workspace_bytes(n, n_kv, gqa, max_len, 1);
}

rkv_status rkv_dense_decode_weights(const void* q, const void* k, const void* v,
                                    const int32_t* len, int n, int n_kv, int gqa, int head_dim,
                                    int max_len, float scale, void* out, float* weights, void* ws,
                                    size_t ws_bytes, void* stream) {
  RKV_TRACE();
  CacheDecodeArgs a{};
  a.q = static_cast<const bf16*>(q);
  a.k = k;
  a.v = v;
  a.len = len;
  a.n = n;
  a.n_kv = n_kv;
  a.gqa = gqa;
  a.cap = max_len;
  a.out = static_cast<bf16*>(out);
  a.weights = weights;
  return decode_impl(a, head_dim, scale, ws, ws_bytes, stream);
}

size_t rkv_prompt_weights_workspace_bytes(int n, int n_kv, int gqa, int max_q, int max_len) {
  if (!counts_ok(n, n_kv, gqa) || gqa > kMaxPromptGqa || max_q <= 0 || max_len < max_q ||
      !prompt_rows_ok(n, n_kv, gqa, max_q, max_len))
    return 0;
  return kStatusBytes + prompt_scratch_bytes(n, n_kv, gqa, max_q, max_len);
}

rkv_status rkv_prompt_weights(const void* q, const int32_t* q_len, const void* k,
                              const int32_t* len, int n, int n_kv, int gqa, int head_dim,
                              int max_q, int max_len, float scale, float* weights, void* ws,
                              size_t ws_bytes, void* stream) {
  RKV_TRACE();
  return prompt_impl(q, q_len, k, len, n, n_kv, gqa, head_dim, max_q, max_len, scale, weights, 0, 0,
                     ws, ws_bytes, stream);
}

rkv_status rkv_testing_prompt_wait_timeout(const void* q, const int32_t* q_len, const void* k,
                                           const int32_t* len, int n, int n_kv, int gqa,
                                           int head_dim, int max_q, int max_len, float scale,
                                           float* weights, int what, uint64_t wait_limit_ns,
                                           void* ws, size_t ws_bytes, void* stream) {
  RKV_TRACE();
  if (what < RKV_TESTING_PROMPT_KEYS || what > RKV_TESTING_PROMPT_SUMS ||
      wait_limit_ns < 1000ull || wait_limit_ns > 1000000000ull)
    return RKV_ERR_INVALID_ARG;
  return prompt_impl(q, q_len, k, len, n, n_kv, gqa, head_dim, max_q, max_len, scale, weights,
                     wait_limit_ns, what, ws, ws_bytes, stream);
}

// ------------------------------------------------------------------------------- eviction
size_t rkv_evict_workspace_bytes(int n, int n_kv, int cap, int keep) {
  if (!counts_ok(n, n_kv, 1) || !cap_ok(cap) || keep <= 0) return 0;
  return kStatusBytes + evict_scratch_bytes(n, n_kv, cap, keep);
}

rkv_status rkv_evict(void* k, void* v, const int32_t* len, int32_t* len_out, const float* weights,
                     float* weights_out, const int32_t* pos, int32_t* pos_out,
                     const int32_t* seen, int n, int n_kv, int head_dim, int cap, int keep,
                     int recent, int32_t* src_rows, void* ws, size_t ws_bytes, void* stream) {
  RKV_TRACE();
  EvictArgs a = evict_args(len, len_out, weights, weights_out, pos, pos_out, seen, n, n_kv, cap,
                           keep, recent, src_rows);
  a.rows[0] = static_cast<uint8_t*>(k);
  a.rows[1] = static_cast<uint8_t*>(v);
  a.row_bytes[0] = a.row_bytes[1] = kHeadDim * 2;
  return evict_impl(a, head_dim, ws, ws_bytes, stream);
}

rkv_status rkv_evict_kv4(void* k_codes, void* k_scales, void* v_codes, void* v_scales,
                         const int32_t* len, int32_t* len_out, const float* weights,
                         float* weights_out, const int32_t* pos, int32_t* pos_out,
                         const int32_t* seen, int n, int n_kv, int head_dim, int cap, int keep,
                         int recent, int32_t* src_rows, void* ws, size_t ws_bytes, void* stream) {
  RKV_TRACE();
  EvictArgs a = evict_args(len, len_out, weights, weights_out, pos, pos_out, seen, n, n_kv, cap,
                           keep, recent, src_rows);
  a.rows[0] = static_cast<uint8_t*>(k_codes);
  a.rows[1] = static_cast<uint8_t*>(v_codes);
  a.rows[2] = static_cast<uint8_t*>(k_scales);
  a.rows[3] = static_cast<uint8_t*>(v_scales);
  a.row_bytes[0] = a.row_bytes[1] = kCodeBytes;
  a.row_bytes[2] = a.row_bytes[3] = kRowScales;
  return evict_impl(a, head_dim, ws, ws_bytes, stream);
}

}  // extern "C"
