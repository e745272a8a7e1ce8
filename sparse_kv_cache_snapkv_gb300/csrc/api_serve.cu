// C ABI of a serving step around the cache (places, rotary positions, attention of packed tokens):
// argument validation, workspace carving, kernel launches. The contract is in include/rkv.h.
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

constexpr int kMostRows = 1 << 30;  // rows of a pool or table: slots and positions stay within 31 bits
constexpr int kMostUnits = 1 << 30;  // of a call: steps over the units, and pairs of tiles, stay within 31 bits

rkv_status ws_check(const void* ws, size_t ws_bytes, size_t need) {
  if (need == 0) return RKV_ERR_INVALID_ARG;
  return ws && aligned16(ws) && ws_bytes >= need ? RKV_OK : RKV_ERR_WORKSPACE;
}

void* after_status(void* ws) { return static_cast<unsigned char*>(ws) + kStatusBytes; }

// a slice's tokens keep every head's rows on 16 bytes and do not overlap
bool stride_ok(int64_t stride, int heads) {
  return stride % 8 == 0 && stride >= (int64_t)heads * kHeadDim && stride <= (1ll << 38);
}

bool slot_sizes_ok(int n, int num_blocks, int block, int max_blocks) {
  return n > 0 && n <= kMostUnits && num_blocks > 0 && block > 0 && max_blocks > 0 &&
         (long long)num_blocks * block <= kMostRows && (long long)max_blocks * block <= kMostRows;
}

rkv_status attention_impl(const void* q, int64_t q_stride, const int32_t* q_start, const int32_t* mask,
                          int words, bool tree, const void* k, const void* v, const PagedMap& pm,
                          const int32_t* len, int n, int n_kv, int gqa, int head_dim, int tokens, int cap,
                          float scale, void* out, uint64_t wait_limit_ns, int test_skip, void* ws,
                          size_t ws_bytes, void* stream) {
  if (head_dim != kHeadDim || gqa > kMaxAttentionGqa) return RKV_ERR_UNSUPPORTED;
  if (!q || !q_start || !k || !v || !len || !out || !aligned16(q) || !aligned16(k) || !aligned16(v) ||
      !aligned16(out) || q == out)
    return RKV_ERR_INVALID_ARG;
  if (tree && (!mask || words <= 0 || words > kMaxTreeWords)) return RKV_ERR_INVALID_ARG;
  if (n <= 0 || n_kv <= 0 || gqa <= 0 || tokens <= 0 || cap <= 0 || cap > kMostRows ||
      (long long)n_kv * gqa > INT_MAX / kHeadDim || !stride_ok(q_stride, n_kv * gqa) ||
      !(scale > 0.f && std::isfinite(scale * kLog2e) && scale * kLog2e > 0.f))
    return RKV_ERR_INVALID_ARG;
  // a row's index is a 32-bit coordinate of the tensor maps
  const double rows = pm.table ? (double)pm.num_blocks * n_kv * pm.block : (double)n * n_kv * cap;
  if (rows > INT_MAX - 512 || (double)tokens * n_kv * gqa > INT_MAX - 512) return RKV_ERR_TOO_LARGE;
  const rkv_status w = ws_check(ws, ws_bytes, rkv_prompt_attention_workspace_bytes(n, n_kv, gqa, tokens));
  if (w != RKV_OK) return w;
  AttentionArgs a{};
  a.q = static_cast<const bf16*>(q);
  a.q_stride = q_stride;
  a.q_start = q_start;
  a.mask = tree ? reinterpret_cast<const uint32_t*>(mask) : nullptr;
  a.k = static_cast<const bf16*>(k);
  a.v = static_cast<const bf16*>(v);
  a.pm = pm;
  a.len = len;
  a.n = n;
  a.n_kv = n_kv;
  a.gqa = gqa;
  a.tokens = tokens;
  a.cap = cap;
  a.words = words;
  a.scale_log2 = scale * kLog2e;
  a.out = static_cast<bf16*>(out);
  a.scratch = after_status(ws);
  a.status = status_ptr(ws);
  a.wait_limit_ns = wait_limit_ns;
  a.test_skip = test_skip;
  return from_cuda(launch_attention(a, as_stream(stream)));
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------------------- places
size_t rkv_reserve_slots_workspace_bytes(int n) {
  return n > 0 && n <= kMostUnits ? kStatusBytes + slots_scratch_bytes(n) : 0;
}
size_t rkv_release_blocks_workspace_bytes(int n) { return rkv_reserve_slots_workspace_bytes(n); }

rkv_status rkv_reserve_slots(const int32_t* new_len, const int32_t* len, const int32_t* held,
                             int32_t* block_table, const int32_t* free_blocks,
                             const int32_t* free_count, int n, int num_blocks, int block,
                             int max_blocks, int max_tokens, int32_t* q_start, int32_t* slots,
                             int32_t* positions, int32_t* len_out, int32_t* held_out,
                             int32_t* free_count_out, void* ws, size_t ws_bytes, void* stream) {
  RKV_TRACE();
  if (!new_len || !len || !held || !block_table || !free_blocks || !free_count || !q_start || !slots ||
      !positions || !len_out || !held_out || !free_count_out)
    return RKV_ERR_INVALID_ARG;
  if (!slot_sizes_ok(n, num_blocks, block, max_blocks) || max_tokens <= 0 || max_tokens > kMostRows)
    return RKV_ERR_INVALID_ARG;
  const rkv_status w = ws_check(ws, ws_bytes, rkv_reserve_slots_workspace_bytes(n));
  if (w != RKV_OK) return w;
  SlotArgs a{};
  a.new_len = new_len;
  a.len = len;
  a.held = held;
  a.table = block_table;
  a.free_blocks = const_cast<int32_t*>(free_blocks);
  a.free_count = free_count;
  a.q_start = q_start;
  a.slots = slots;
  a.positions = positions;
  a.len_out = len_out;
  a.held_out = held_out;
  a.free_count_out = free_count_out;
  a.n = n;
  a.max_blocks = max_blocks;
  a.num_blocks = num_blocks;
  a.block = block;
  a.room = max_tokens;
  a.wide = aligned16(slots) && aligned16(positions);
  a.scratch = after_status(ws);
  a.status = status_ptr(ws);
  return from_cuda(launch_reserve_slots(a, as_stream(stream)));
}

rkv_status rkv_release_blocks(const int32_t* len, const int32_t* held, const int32_t* block_table,
                              int32_t* free_blocks, const int32_t* free_count, int n,
                              int num_blocks, int block, int max_blocks, int32_t* held_out,
                              int32_t* free_count_out, void* ws, size_t ws_bytes, void* stream) {
  RKV_TRACE();
  if (!len || !held || !block_table || !free_blocks || !free_count || !held_out || !free_count_out)
    return RKV_ERR_INVALID_ARG;
  if (!slot_sizes_ok(n, num_blocks, block, max_blocks)) return RKV_ERR_INVALID_ARG;
  const rkv_status w = ws_check(ws, ws_bytes, rkv_release_blocks_workspace_bytes(n));
  if (w != RKV_OK) return w;
  SlotArgs a{};
  a.len = len;
  a.held = held;
  a.table = const_cast<int32_t*>(block_table);
  a.free_blocks = free_blocks;
  a.free_count = free_count;
  a.held_out = held_out;
  a.free_count_out = free_count_out;
  a.n = n;
  a.max_blocks = max_blocks;
  a.num_blocks = num_blocks;
  a.block = block;
  a.scratch = after_status(ws);
  a.status = status_ptr(ws);
  return from_cuda(launch_release_blocks(a, as_stream(stream)));
}

// ------------------------------------------------------------------------------- rotary positions
rkv_status rkv_rope_frequencies(int kind, int rot_dim, double base, double factor, int ctx,
                                double fast, double slow, float* inv_freq, float* mscale) {
  const bool by_pairs = kind == RKV_ROPE_BY_PARTS || kind == RKV_ROPE_BY_WHOLE_PARTS;
  const bool parts = by_pairs || kind == RKV_ROPE_SMOOTH;
  if (kind < RKV_ROPE_PLAIN || kind > RKV_ROPE_BY_WHOLE_PARTS || rot_dim < 2 || rot_dim > kHeadDim || rot_dim % 2 ||
      !(base > 1.0) || !std::isfinite(base) || !inv_freq || !mscale)
    return RKV_ERR_INVALID_ARG;
  if (kind != RKV_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return RKV_ERR_INVALID_ARG;
  if (kind == RKV_ROPE_BASE && rot_dim < 4) return RKV_ERR_INVALID_ARG;
  if (parts && (ctx <= 0 || !(slow > 0.0) || !(fast > slow) || !std::isfinite(fast)))
    return RKV_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586;
  if (kind == RKV_ROPE_BASE) base *= std::pow(factor, rot_dim / (rot_dim - 2.0));
  // the (real) number of the pair that turns t times within ctx
  auto pair_of = [&](double t) { return rot_dim * std::log(ctx / (t * two_pi)) / (2.0 * std::log(base)); };
  double first = 0.0, last = 1.0;  // the ramp's ends
  if (by_pairs) {
    first = pair_of(fast);
    last = pair_of(slow);
  }
  if (kind == RKV_ROPE_BY_WHOLE_PARTS) {
    auto within = [&](double x) { return x < 0.0 ? 0.0 : x > rot_dim - 1.0 ? rot_dim - 1.0 : x; };
    first = within(std::floor(first));
    last = within(std::ceil(last));
    if (last == first) last += 0.001;
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rot_dim);
    double keep = 1.0;  // share of the unscaled frequency
    if (kind == RKV_ROPE_LINEAR) keep = 0.0;
    if (by_pairs) keep = (last - i) / (last - first);
    if (kind == RKV_ROPE_SMOOTH) keep = (ctx * f / two_pi - slow) / (fast - slow);
    keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
    inv_freq[i] = (float)(kind == RKV_ROPE_PLAIN || kind == RKV_ROPE_BASE
                              ? f
                              : f * keep + f / factor * (1.0 - keep));
  }
  *mscale = by_pairs ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  return RKV_OK;
}

size_t rkv_rope_append_workspace_bytes(void) { return kStatusBytes; }

rkv_status rkv_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                           const void* v, int64_t v_stride, const int32_t* positions,
                           const float* inv_freq, const int32_t* slots, int tokens, int hq,
                           int n_kv, int head_dim, int rot_dim, int interleaved, float mscale,
                           void* q_out, void* k_pool, void* v_pool, int num_blocks, int block,
                           void* ws, size_t ws_bytes, void* stream) {
  RKV_TRACE();
  if (head_dim != kHeadDim || rot_dim < 16 || rot_dim > kHeadDim || rot_dim % 16) return RKV_ERR_UNSUPPORTED;
  if (!q || !k || !v || !positions || !inv_freq || !slots || !q_out || !k_pool || !v_pool || !aligned16(q) ||
      !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_pool) || !aligned16(v_pool))
    return RKV_ERR_INVALID_ARG;
  if (tokens <= 0 || hq <= 0 || n_kv <= 0 || (long long)hq + 2ll * n_kv > INT_MAX / kHeadDim ||
      num_blocks <= 0 || block <= 0 || !stride_ok(q_stride, hq) || !stride_ok(k_stride, n_kv) ||
      !stride_ok(v_stride, n_kv) || !std::isfinite(mscale) || (interleaved != 0 && interleaved != 1))
    return RKV_ERR_INVALID_ARG;
  if (q == q_out && q_stride != (int64_t)hq * kHeadDim) return RKV_ERR_INVALID_ARG;
  const rkv_status w = ws_check(ws, ws_bytes, rkv_rope_append_workspace_bytes());
  if (w != RKV_OK) return w;
  RopeArgs a{};
  a.q = static_cast<const bf16*>(q);
  a.k = static_cast<const bf16*>(k);
  a.v = static_cast<const bf16*>(v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.slots = slots;
  a.q_out = static_cast<bf16*>(q_out);
  a.k_cache = static_cast<bf16*>(k_pool);
  a.v_cache = static_cast<bf16*>(v_pool);
  a.tokens = tokens;
  a.hq = hq;
  a.n_kv = n_kv;
  a.rot = rot_dim;
  a.interleaved = interleaved;
  a.num_blocks = num_blocks;
  a.block = block;
  a.mscale = mscale;
  a.status = status_ptr(ws);
  return from_cuda(launch_rope_append(a, as_stream(stream)));
}

// ------------------------------------------------------------------------------- attention
size_t rkv_prompt_attention_workspace_bytes(int n, int n_kv, int gqa, int tokens) {
  if (n <= 0 || n > kMostUnits || n_kv <= 0 || gqa <= 0 || gqa > kMaxAttentionGqa || tokens <= 0 ||
      (double)tokens * n_kv * gqa > INT_MAX - 512)
    return 0;
  return kStatusBytes + attention_scratch_bytes(n, gqa, tokens);
}

rkv_status rkv_prompt_attention(const void* q, int64_t q_stride, const int32_t* q_start,
                                const void* k, const void* v, const int32_t* len, int n, int n_kv,
                                int gqa, int head_dim, int tokens, int max_len, float scale,
                                void* out, void* ws, size_t ws_bytes, void* stream) {
  RKV_TRACE();
  return attention_impl(q, q_stride, q_start, nullptr, 0, false, k, v, PagedMap{}, len, n, n_kv, gqa,
                        head_dim, tokens, max_len, scale, out, 0, 0, ws, ws_bytes, stream);
}

rkv_status rkv_prompt_attention_paged(const void* q, int64_t q_stride, const int32_t* q_start,
                                      const void* k_pool, const void* v_pool,
                                      const int32_t* block_table, const int32_t* len, int n,
                                      int n_kv, int gqa, int head_dim, int tokens, int num_blocks,
                                      int block, int max_blocks, float scale, void* out, void* ws,
                                      size_t ws_bytes, void* stream) {
  RKV_TRACE();
  if (!paged_ok(block_table, num_blocks, block, max_blocks)) return RKV_ERR_INVALID_ARG;
  const PagedMap pm{block_table, max_blocks, block, num_blocks};
  return attention_impl(q, q_stride, q_start, nullptr, 0, false, k_pool, v_pool, pm, len, n, n_kv, gqa,
                        head_dim, tokens, max_blocks * block, scale, out, 0, 0, ws, ws_bytes, stream);
}

rkv_status rkv_tree_attention(const void* q, int64_t q_stride, const int32_t* q_start,
                              const int32_t* mask, int mask_words, const void* k, const void* v,
                              const int32_t* len, int n, int n_kv, int gqa, int head_dim,
                              int tokens, int max_len, float scale, void* out, void* ws,
                              size_t ws_bytes, void* stream) {
  RKV_TRACE();
  return attention_impl(q, q_stride, q_start, mask, mask_words, true, k, v, PagedMap{}, len, n, n_kv, gqa,
                        head_dim, tokens, max_len, scale, out, 0, 0, ws, ws_bytes, stream);
}

rkv_status rkv_tree_attention_paged(const void* q, int64_t q_stride, const int32_t* q_start,
                                    const int32_t* mask, int mask_words, const void* k_pool,
                                    const void* v_pool, const int32_t* block_table,
                                    const int32_t* len, int n, int n_kv, int gqa, int head_dim,
                                    int tokens, int num_blocks, int block, int max_blocks,
                                    float scale, void* out, void* ws, size_t ws_bytes,
                                    void* stream) {
  RKV_TRACE();
  if (!paged_ok(block_table, num_blocks, block, max_blocks)) return RKV_ERR_INVALID_ARG;
  const PagedMap pm{block_table, max_blocks, block, num_blocks};
  return attention_impl(q, q_stride, q_start, mask, mask_words, true, k_pool, v_pool, pm, len, n, n_kv, gqa,
                        head_dim, tokens, max_blocks * block, scale, out, 0, 0, ws, ws_bytes, stream);
}

rkv_status rkv_testing_attention_wait_timeout(const void* q, int64_t q_stride,
                                              const int32_t* q_start, const void* k,
                                              const void* v, const int32_t* len, int n, int n_kv,
                                              int gqa, int head_dim, int tokens, int max_len,
                                              float scale, void* out, int what,
                                              uint64_t wait_limit_ns, void* ws, size_t ws_bytes,
                                              void* stream) {
  RKV_TRACE();
  if (what < RKV_TESTING_ATTENTION_QUERIES || what > RKV_TESTING_ATTENTION_VALUES ||
      wait_limit_ns < 1000ull || wait_limit_ns > 1000000000ull)
    return RKV_ERR_INVALID_ARG;
  return attention_impl(q, q_stride, q_start, nullptr, 0, false, k, v, PagedMap{}, len, n, n_kv, gqa,
                        head_dim, tokens, max_len, scale, out, wait_limit_ns, what, ws, ws_bytes, stream);
}

}  // extern "C"
