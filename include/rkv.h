/*
 * rkv.h -- C ABI of the RocketKV hot path on GB300 (sm_103a): SnapKV++ prefill eviction and
 * hybrid sparse decode attention, plus a dense decode used as the full-KV timing reference.
 *
 * The method is described in "RocketKV: Accelerating Long-Context LLM Inference via Two-Stage KV
 * Cache Compression" (Behnam et al., arXiv 2502.14051). Sections cited below are those of the
 * authors' OpenReview responses on paperhub.cn (same title), which hold the method's details:
 *   [LAT]   "Lack of Direct Latency Comparison"           -- token budget split half / half
 *   [APPROX]"Explanation of Calculating Approximate Attention Scores" -- pages, Kmin/Kmax,
 *                                                             top-|q| channels, GQA group sums
 *   [PAGE]  "Is Page Always Divided Into 4?"              -- ratio decomposition, page size
 *   [EVICT] "Is Needle Among Evicted Tokens"              -- eviction per head and per layer
 *   [KSIZE] "Potential Sensitivity to Kernel Size in SnapKV++" -- adaptive pooling size
 *   [STEP]  "Are Different KV Tokens Retrieved at Each Decoding Step?" -- selection per step
 *   [SNAP++]"Novelty of SnapKV++"                          -- GQA-aware SnapKV scoring
 *   [MT]    "SCBench Results"                              -- RocketKV-MT: nothing evicted, the
 *                                                             decode selects among kept tokens
 * and [KEYPTS] = "Key points" of the summarizepaper.com summary (full-KV baseline, SnapKV++).
 *
 * Conventions shared by every call
 * --------------------------------
 *  - Every tensor pointer is DEVICE memory owned by the caller. The library allocates nothing
 *    and keeps no state between calls. bf16 tensors are passed as void* and must be 16-byte
 *    aligned. All integer tensors are int32.
 *  - n counts independent problems (batch x layers flattened; "unit" below = one of the n).
 *    Query heads of unit u: Hq = n_kv * gqa, query head h belongs to KV head h / gqa.
 *  - head_dim must be 128 (RKV_ERR_UNSUPPORTED otherwise).
 *  - Every call is asynchronous on `stream` (a cudaStream_t passed as void*; NULL = legacy
 *    default stream). Arguments are validated on the host before any launch; an invalid
 *    argument returns RKV_ERR_INVALID_ARG / RKV_ERR_UNSUPPORTED / RKV_ERR_WORKSPACE and launches
 *    nothing. A failed launch returns RKV_ERR_CUDA.
 *  - ws / ws_bytes: scratch owned by the caller, at least the size the matching
 *    *_workspace_bytes() returns. Its first 256 bytes hold a device status word that kernels set
 *    when they detect an inconsistency in device-resident data (e.g. a length beyond capacity,
 *    a bounded wait that ran out). It must be zero before first use (allocate it zeroed).
 *    rkv_check_status() synchronises the stream, reads and clears it. Kernels never trap.
 *  - Two calls that share one workspace must not overlap on the GPU (same stream is fine).
 */
#ifndef RKV_H_
#define RKV_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  RKV_OK = 0,
  RKV_ERR_INVALID_ARG = 1,
  RKV_ERR_UNSUPPORTED = 2,
  RKV_ERR_WORKSPACE = 3,
  RKV_ERR_CUDA = 4,
  RKV_ERR_DEVICE_STATUS = 5,
  RKV_ERR_TOO_LARGE = 6
} rkv_status;

/* Device status bits (reported by rkv_check_status through *bits). */
#define RKV_DEV_LEN_OVER_CAP   0x1u  /* a length exceeds cap / page_cap (work for it skipped) */
#define RKV_DEV_BAD_WINDOW     0x2u  /* a sequence shorter than the window (unit skipped)     */
#define RKV_DEV_WAIT_TIMEOUT   0x4u  /* a bounded mbarrier wait ran out (unit abandoned)      */
#define RKV_DEV_SELECT_FAILED  0x8u  /* a top-k selection produced the wrong count (or: a CTA's
                                        shared memory began off its alignment; it did nothing) */
#define RKV_DEV_BAD_INDEX      0x10u /* a kept index outside the valid rows (row 0 read)      */
#define RKV_DEV_NO_BLOCKS      0x20u /* fewer free blocks than a unit needs (unit not served) */

/* Human-readable name of a status code (static string). */
const char* rkv_status_string(rkv_status s);

/* Synchronise `stream`, read the device status word in `ws`, clear it, and return RKV_OK if it
 * was zero or RKV_ERR_DEVICE_STATUS otherwise (bits in *bits when bits != NULL). */
rkv_status rkv_check_status(void* ws, void* stream, uint32_t* bits);

/* Pure host planner ([PAGE], [LAT], [KSIZE]). The overall ratio ctx / budget is split between
 * the two stages, and stage 2's share between the sequence dimension (page) and the head
 * dimension (head_dim / channels). page = 0 picks 4 and channels = 0 picks head_dim / 4; the
 * stage-1 keep is then min(ctx, budget * page * head_dim / channels), which makes the
 * approximation read exactly as many bytes as budget / 2 tokens of K and V. kernel_size: 7 for
 * ctx <= 8192, 15 for ctx <= 32768, else 31 (larger pooling for longer prompts). Any output
 * pointer may be NULL. Errors: RKV_ERR_INVALID_ARG for non-positive sizes, channels > head_dim,
 * budget odd or budget / 2 < page. */
rkv_status rkv_plan(int ctx, int budget, int head_dim, int page, int channels,
                    int* keep, int* page_out, int* channels_out, int* kernel_size);

/* The even split of [PAGE] for any ratio: with R = ctx / budget, each stage gets sqrt(R), and
 * stage 2's share is split evenly between the page size and the channel reduction, so that
 * page ~ R^(1/4) and head_dim / channels ~ R^(1/4) (128K tokens at budget 512: R = 256, page 4,
 * channels head_dim / 4, keep 8192). Where R^(1/4) is not a power of two the page is the power
 * of two nearest to it on a log2 scale (halves round up), within [1, min(64, budget / 2)];
 * channels = round(head_dim * page / sqrt(R)) within [1, head_dim]; keep and kernel_size as for
 * rkv_plan. Errors: RKV_ERR_INVALID_ARG for ctx <= 0, budget < 2 or odd, head_dim <= 0. */
rkv_status rkv_plan_even_split(int ctx, int budget, int head_dim, int* keep, int* page,
                               int* channels, int* kernel_size);

/* ------------------------------------------------------------------------------------------ */
/* Stage 1: SnapKV++ eviction ([SNAP++], [EVICT], [KSIZE], [KEYPTS])                            */
/* ------------------------------------------------------------------------------------------ */
size_t rkv_snapkv_workspace_bytes(int n, int n_kv, int gqa, int max_len, int window);

/* For each unit u and KV head g: score every prefix position i < L_u - window with the window
 * queries -- softmax(q . k / sqrt-scale) over all keys visible to each window query (the prefix
 * plus the causal part of the window), summed over the window and over the gqa query heads of
 * the group -- max-pool the scores with an odd kernel (stride 1, same length, clipped ends), keep
 * the keep - window highest (ties -> lower position) and append the window, then gather those
 * rows of K and V into the compact cache.
 *   k, v      [n][n_kv][max_len][128] bf16, rows >= L_u ignored
 *   seq_lens  [n] int32 on device, window <= L_u <= max_len
 *   q_win     [n][n_kv*gqa][window][128] bf16 -- the last `window` queries of every head
 *   window    1 <= window, gqa * window <= 256
 *   kernel_size odd >= 1, or 0 to pick it per sequence from L_u (7 / 15 / 31 as rkv_plan)
 *   keep      tokens kept per (unit, KV head) including the window; window < keep <= cap.
 *             A sequence with L_u <= keep keeps all L_u tokens.
 *   scale     logit scale (1/sqrt(128) for the usual attention)
 *   k_out, v_out [n][n_kv][cap][128] bf16: rows 0 .. out_len[u]-1 written (kept positions in
 *             ascending order, the window last)
 *   kept_idx  [n][n_kv][keep] int32: original positions of the kept rows; -1 past out_len[u]
 *   out_len   [n] int32: min(L_u, keep)
 *   scores_out NULL or [n][n_kv][max_len - window] fp32: the un-pooled prefix scores
 */
rkv_status rkv_snapkv_compress(const void* k, const void* v, const int32_t* seq_lens,
                               const void* q_win, int n, int n_kv, int gqa, int head_dim,
                               int max_len, int window, int kernel_size, int keep, float scale,
                               void* k_out, void* v_out, int cap, int32_t* kept_idx,
                               int32_t* out_len, float* scores_out, void* ws, size_t ws_bytes,
                               void* stream);

/* [SNAP++] The scoring half of rkv_snapkv_compress alone: for each unit u and KV head g, the
 * score of every prefix position i < L_u - window (softmax probabilities of the window queries
 * over the keys each may see, summed over the window and over the gqa query heads of the group),
 * with no pooling, selection or gather. For a caller that pools or selects by its own rule, and
 * for timing the two tensor-core score passes on their own.
 *   k, seq_lens, q_win, window, scale as rkv_snapkv_compress (no V needed)
 *   scores_out [n][n_kv][max_len - window] fp32 (required): entries i >= L_u - window of a
 *             unit are left untouched
 * Workspace rkv_snapkv_workspace_bytes; errors as rkv_snapkv_compress. */
rkv_status rkv_snapkv_scores(const void* k, const int32_t* seq_lens, const void* q_win, int n,
                             int n_kv, int gqa, int head_dim, int max_len, int window,
                             float scale, float* scores_out, void* ws, size_t ws_bytes,
                             void* stream);

/* [MT] The selection half of rkv_snapkv_compress (scores, pooling, top-k) without the gather:
 * RocketKV-MT evicts nothing, so each turn filters the full, unfiltered history again
 * ("SCBench Results": the next turn's prefill takes all earlier tokens as its prefix and SnapKV++
 * filters once more) and the decode reads the kept rows through the index list.
 *   k         [n][n_kv][max_len][128] bf16: the full cache, rows >= L_u ignored (no V needed)
 *   seq_lens  [n] int32: history length L_u this turn (earlier turns, generated tokens, the new
 *             input), window <= L_u <= max_len
 *   q_win     [n][n_kv*gqa][window][128] bf16: the last `window` queries of this turn's input
 *   kept_idx  [n][n_kv][kept_stride] int32, kept_stride >= keep: entries 0 .. keep-1 of each
 *             (unit, KV head) written as in rkv_snapkv_compress (-1 past out_len[u]); entries
 *             keep .. kept_stride-1 untouched, so the list can be handed to
 *             rkv_build_page_summaries_mt / rkv_hybrid_decode_mt with kcap = kept_stride
 *   out_len   [n] int32: min(L_u, keep), the kept_len of the MT calls
 * Other arguments, workspace (rkv_snapkv_workspace_bytes) and errors as rkv_snapkv_compress. */
rkv_status rkv_snapkv_select(const void* k, const int32_t* seq_lens, const void* q_win, int n,
                             int n_kv, int gqa, int head_dim, int max_len, int window,
                             int kernel_size, int keep, float scale, int32_t* kept_idx,
                             int kept_stride, int32_t* out_len, float* scores_out, void* ws,
                             size_t ws_bytes, void* stream);

/* rkv_snapkv_compress with average pooling in place of max pooling (a SnapKV pooling variant;
 * the pages describe max pooling only): each prefix score is replaced by the mean of the scores
 * over the in-range positions of its clipped window [max(0, i - r), min(n - 1, i + r)],
 * r = kernel_size / 2, before the top-k. The window sums are exact (fixed point), so the result
 * depends only on the fp32 scores. kernel_size odd in [1, 1048575], or 0 as above. Other
 * arguments, outputs, workspace and errors as rkv_snapkv_compress. */
rkv_status rkv_snapkv_compress_avg_pool(const void* k, const void* v, const int32_t* seq_lens,
                                        const void* q_win, int n, int n_kv, int gqa,
                                        int head_dim, int max_len, int window, int kernel_size,
                                        int keep, float scale, void* k_out, void* v_out, int cap,
                                        int32_t* kept_idx, int32_t* out_len, float* scores_out,
                                        void* ws, size_t ws_bytes, void* stream);

/* rkv_snapkv_compress followed by rkv_build_page_summaries(k_out, out_len, page, page_cap,
 * first_token = 0, kmin, kmax) in one pass: the gather builds the page summaries of the rows it
 * writes ([APPROX]), so the compact cache is not read back. Same outputs, bit for bit. page a
 * power of two <= 64; page_cap a multiple of 8 with page_cap * page >= keep; kmin, kmax
 * [n][n_kv][128][page_cap] bf16 (pages past ceil(out_len[u] / page) untouched). Workspace:
 * rkv_snapkv_workspace_bytes. */
rkv_status rkv_snapkv_compress_summarized(const void* k, const void* v,
                                          const int32_t* seq_lens, const void* q_win, int n,
                                          int n_kv, int gqa, int head_dim, int max_len,
                                          int window, int kernel_size, int keep, float scale,
                                          void* k_out, void* v_out, int cap, int32_t* kept_idx,
                                          int32_t* out_len, float* scores_out, int page,
                                          int page_cap, void* kmin, void* kmax, void* ws,
                                          size_t ws_bytes, void* stream);

/* The ablation without the GQA enhancement ([SNAP++], [KEYPTS]: plain SnapKV): every query
 * head is scored and filtered on its own -- its W window rows only, no sum over the group -- and
 * keeps its own copy of the selected rows of its K/V head h / gqa. Same arguments as
 * rkv_snapkv_compress, with the per-unit outputs per query head:
 *   k_out, v_out [n][n_kv*gqa][cap][128] bf16; kept_idx [n][n_kv*gqa][keep] int32;
 *   scores_out NULL or [n][n_kv*gqa][max_len - window] fp32; out_len [n] int32.
 * window <= 256. Workspace: rkv_snapkv_per_head_workspace_bytes. The result is a cache that the
 * decode calls use with n_kv*gqa K/V heads and gqa = 1. */
size_t rkv_snapkv_per_head_workspace_bytes(int n, int n_kv, int gqa, int max_len, int window);
rkv_status rkv_snapkv_compress_per_head(const void* k, const void* v, const int32_t* seq_lens,
                                        const void* q_win, int n, int n_kv, int gqa,
                                        int head_dim, int max_len, int window, int kernel_size,
                                        int keep, float scale, void* k_out, void* v_out, int cap,
                                        int32_t* kept_idx, int32_t* out_len, float* scores_out,
                                        void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------------------ */
/* Stage 2: page summaries ([APPROX])                                                          */
/* ------------------------------------------------------------------------------------------ */
size_t rkv_summaries_workspace_bytes(void);

/* Element-wise min and max of K over pages of `page` consecutive cache rows, stored
 * channel-major so that one channel of all pages is one contiguous row:
 *   k_cache [n][n_kv][cap][128] bf16, len [n] int32 (device)
 *   kmin, kmax [n][n_kv][128][page_cap] bf16; page p of unit u covers rows p*page ..
 *   min(len_u, (p+1)*page) - 1 (a partial last page uses its valid rows only).
 *   Pages from first_token / page up to the last page are (re)computed; first_token = 0
 *   rebuilds everything. page is a power of two <= 64; page_cap is a multiple of 8 and
 *   page_cap * page >= the largest len (checked on device: RKV_DEV_LEN_OVER_CAP).
 */
rkv_status rkv_build_page_summaries(const void* k_cache, const int32_t* len, int n, int n_kv,
                                    int head_dim, int cap, int page, int page_cap,
                                    int first_token, void* kmin, void* kmax, void* ws,
                                    size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------------------ */
/* Stage 2: hybrid sparse decode ([APPROX], [LAT], [STEP], [PAGE])                              */
/* ------------------------------------------------------------------------------------------ */
/* The decode's workspace: the status word and one append counter per unit (both zero at first
 * use; the counters are back at zero after every call). */
size_t rkv_hybrid_decode_workspace_bytes(int n, int n_kv, int gqa, int page_cap, int budget,
                                         int page);

/* One decode step. If new_k / new_v are given, token len_u is first appended to every KV head
 * of unit u (cache rows and the page summary it lands in) and len[u] is incremented, inside the
 * same launch; the new token can be selected in this step. Then, per (unit, KV head g):
 *   len_u <= budget: exact attention over every cached token;
 *   otherwise: the `channels` channels with the largest sum over the group of |q_h| (ties ->
 *   lower channel) are kept; with q_g = sum_h q_h, each page scores
 *   sum_{kept i} q_g[i] * (q_g[i] >= 0 ? Kmax[i][page] : Kmin[i][page]) (unscaled); the
 *   (budget/2)/page best pages (ties -> lower page) are selected and all gqa query heads attend
 *   exactly over their valid tokens.
 *   q        [n][n_kv*gqa][128] bf16
 *   new_k, new_v NULL (no append) or [n][n_kv][128] bf16
 *   k_cache, v_cache [n][n_kv][cap][128] bf16; len [n] int32 (device)
 *   kmin, kmax [n][n_kv][128][page_cap] bf16, as built by rkv_build_page_summaries
 *   budget    even, budget/2 >= page; page a power of two <= 64; 1 <= channels <= 128
 *   gqa       1, 2, 4 or 8
 *   out       [n][n_kv*gqa][128] bf16
 *   sel_channels NULL or [n][n_kv][channels] int32 (ascending; -1 on the dense path)
 *   sel_pages NULL or [n][n_kv][(budget/2)/page] int32 (ascending; -1 where unused)
 *   approx_scores NULL or [n][n_kv][page_cap] fp32 (pages >= ceil(len_u/page) untouched)
 * A decode CTA keeps one fp32 score per page of page_cap in shared memory: page_cap may be up to
 * 31,168 (fewer when budget/page is large: 27,136 at budget/page = 4096); beyond that the call
 * returns RKV_ERR_UNSUPPORTED. The same limit holds for the RocketKV-MT and paged variants.
 */
rkv_status rkv_hybrid_decode(const void* q, const void* new_k, const void* new_v,
                             void* k_cache, void* v_cache, int32_t* len, void* kmin, void* kmax,
                             int n, int n_kv, int gqa, int head_dim, int cap, int page_cap,
                             int budget, int page, int channels, float scale, void* out,
                             int32_t* sel_channels, int32_t* sel_pages, float* approx_scores,
                             void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------------------ */
/* RocketKV-MT: the full cache stays, the decode is restricted to the kept tokens ([MT])        */
/* ------------------------------------------------------------------------------------------ */
/* The multi-turn variant evicts nothing: every prompt token stays in the cache (the next turn
 * re-filters the whole history), and the decode selects only among the tokens SnapKV++ kept.
 * Here the kept tokens are named by an index list instead of being copied. For unit u and KV head
 * g the kept sequence is kept_idx[u][g][j], j = 0 .. kept_len[u]-1: rows of the full cache, in
 * the order the decode treats as token order (rkv_snapkv_compress writes such a list). Both calls
 * compute exactly what rkv_build_page_summaries / rkv_hybrid_decode compute on the compact cache
 * whose row j is k_full[u][g][kept_idx[u][g][j]] (same values, same order, same results); page
 * numbers (sel_pages, approx_scores, kmin / kmax columns) count pages of the kept sequence.
 *
 * Page summaries of the kept sequence:
 *   k_full [n][n_kv][full_cap][128] bf16; kept_idx [n][n_kv][kcap] int32; kept_len [n] int32
 *   kmin, kmax [n][n_kv][128][page_cap] bf16; page, page_cap, first_token as for
 *   rkv_build_page_summaries, with kept_len[u] <= kcap and <= page_cap * page (else
 *   RKV_DEV_LEN_OVER_CAP, unit skipped). A kept index outside [0, full_cap) sets
 *   RKV_DEV_BAD_INDEX and row 0 is read in its place. Workspace: rkv_summaries_workspace_bytes.
 */
rkv_status rkv_build_page_summaries_mt(const void* k_full, const int32_t* kept_idx,
                                       const int32_t* kept_len, int n, int n_kv, int head_dim,
                                       int full_cap, int kcap, int page, int page_cap,
                                       int first_token, void* kmin, void* kmax, void* ws,
                                       size_t ws_bytes, void* stream);

/* One decode step over the kept sequence. If new_k / new_v are given, each unit's new token is
 * first written to row full_len[u] of every KV head of the full cache, appended to the kept list
 * (kept_idx[u][g][kept_len[u]] = full_len[u]) and folded into the page summary it lands in; then
 * full_len[u] and kept_len[u] are incremented (RKV_DEV_LEN_OVER_CAP if full_len[u] = full_cap or
 * kept_len[u] = kcap: nothing appended). The rest is rkv_hybrid_decode on the kept sequence:
 * the dense path when kept_len[u] <= budget, else channel pick, page scores, page top-k and exact
 * attention over the selected pages' kept tokens. A kept index outside [0, full_len[u]) sets
 * RKV_DEV_BAD_INDEX and row 0 is read in its place.
 *   q, out [n][n_kv*gqa][128] bf16; new_k, new_v NULL or [n][n_kv][128] bf16
 *   k_full, v_full [n][n_kv][full_cap][128] bf16; full_len [n] int32
 *   kept_idx [n][n_kv][kcap] int32; kept_len [n] int32
 *   kmin, kmax, budget, page, page_cap, channels, gqa, sel_channels, sel_pages, approx_scores:
 *   as for rkv_hybrid_decode (pages of the kept sequence). Workspace:
 *   rkv_hybrid_decode_workspace_bytes.
 */
rkv_status rkv_hybrid_decode_mt(const void* q, const void* new_k, const void* new_v,
                                void* k_full, void* v_full, int32_t* full_len, int32_t* kept_idx,
                                int32_t* kept_len, void* kmin, void* kmax, int n, int n_kv,
                                int gqa, int head_dim, int full_cap, int kcap, int page_cap,
                                int budget, int page, int channels, float scale, void* out,
                                int32_t* sel_channels, int32_t* sel_pages, float* approx_scores,
                                void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------------------ */
/* Paged (block-table) compact cache, for serving engines that page their KV cache             */
/* ------------------------------------------------------------------------------------------ */
/* The same three steps -- stage 1 with its gather, page summaries, decode -- on a compact cache
 * held in fixed-size blocks of a shared pool instead of one contiguous region per unit (a
 * storage layout of the serving engine; the computation is that of the non-paged calls, with
 * identical results):
 *   k_pool, v_pool [num_blocks][n_kv][block][128] bf16; block a power of two <= 65536;
 *   block_table [n][max_blocks] int32: token t of unit u (every K/V head g) is row t % block of
 *   block block_table[u][t / block]; capacity = max_blocks * block tokens per unit.
 * Blocks are the caller's: every block a call may write (stage 1: tokens < keep; an append:
 * token len[u]) must be listed in the table beforehand. A table entry outside [0, num_blocks)
 * that a kernel meets sets RKV_DEV_BAD_INDEX and block 0 is used in its place.
 *
 * rkv_snapkv_compress_paged: rkv_snapkv_compress (workspace rkv_snapkv_workspace_bytes) whose
 *   kept rows go to the pools; keep <= capacity.
 * rkv_build_page_summaries_paged: rkv_build_page_summaries over the paged cache (len[u] <=
 *   capacity, else RKV_DEV_LEN_OVER_CAP); workspace rkv_summaries_workspace_bytes.
 * rkv_hybrid_decode_paged: rkv_hybrid_decode over the paged cache, appends included (len[u] <
 *   capacity to append); workspace rkv_hybrid_decode_workspace_bytes. */
rkv_status rkv_snapkv_compress_paged(const void* k, const void* v, const int32_t* seq_lens,
                                     const void* q_win, int n, int n_kv, int gqa, int head_dim,
                                     int max_len, int window, int kernel_size, int keep,
                                     float scale, void* k_pool, void* v_pool, int num_blocks,
                                     int block, const int32_t* block_table, int max_blocks,
                                     int32_t* kept_idx, int32_t* out_len, float* scores_out,
                                     void* ws, size_t ws_bytes, void* stream);
rkv_status rkv_build_page_summaries_paged(const void* k_pool, const int32_t* block_table,
                                          const int32_t* len, int n, int n_kv, int head_dim,
                                          int num_blocks, int block, int max_blocks, int page,
                                          int page_cap, int first_token, void* kmin, void* kmax,
                                          void* ws, size_t ws_bytes, void* stream);
rkv_status rkv_hybrid_decode_paged(const void* q, const void* new_k, const void* new_v,
                                   void* k_pool, void* v_pool, const int32_t* block_table,
                                   int32_t* len, void* kmin, void* kmax, int n, int n_kv, int gqa,
                                   int head_dim, int num_blocks, int block, int max_blocks,
                                   int page_cap, int budget, int page, int channels, float scale,
                                   void* out, int32_t* sel_channels, int32_t* sel_pages,
                                   float* approx_scores, void* ws, size_t ws_bytes,
                                   void* stream);

/* ------------------------------------------------------------------------------------------ */
/* Full-KV decode attention, the baseline the method is compared against ([KEYPTS])            */
/* ------------------------------------------------------------------------------------------ */
size_t rkv_dense_decode_workspace_bytes(int n, int n_kv, int gqa, int max_len);

/* out[u][h] = softmax(scale * q[u][h] . K[u][g]^T) V[u][g] over the len_u cached tokens
 * (g = h / gqa), split over the sequence across thread blocks and merged.
 *   q [n][n_kv*gqa][128] bf16; k, v [n][n_kv][max_len][128] bf16; len [n] int32 (device,
 *   1 <= len_u <= max_len); out [n][n_kv*gqa][128] bf16; gqa 1, 2, 4 or 8.
 */
rkv_status rkv_dense_decode(const void* q, const void* k, const void* v, const int32_t* len,
                            int n, int n_kv, int gqa, int head_dim, int max_len, float scale,
                            void* out, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------------------ */
/* Allocation-free dense decode (a library convenience; the paper has no counterpart)          */
/* ------------------------------------------------------------------------------------------ */
/* Same computation, arguments and layouts as rkv_dense_decode, but without ws / ws_bytes: the
 * split-K partials go to an 8 MiB array of device memory that the library reserves statically
 * (every GPU that loads the library holds it until the process exits).
 *
 * It exists for callers that cannot call cudaMalloc to build a workspace: code that is only
 * handed its input and output tensors (a plugin boundary, say), or a host whose device memory
 * belongs entirely to its own pool. The caller still passes inputs and outputs; nothing is
 * allocated or freed by this call.
 *
 *  - Limit: 256 B + the partials of rkv_dense_decode_workspace_bytes(n, n_kv, gqa, max_len) must
 *    fit in 8 MiB; otherwise RKV_ERR_TOO_LARGE is returned and nothing is launched (the sizes
 *    are checked before the pointers).
 *  - Set-up: the first call on each device looks up the device address of the array (with that
 *    device current). Make that first call before any stream capture.
 *  - All calls share the one array, which keeps the last call's contents. Each call clears the
 *    status word at its start; calls that overlap on the GPU (different streams, or different
 *    host threads) race on the array and must be serialised by the caller.
 *  - Device-detected inconsistencies (len > max_len is clamped) are not reported by this entry
 *    point. */
rkv_status rkv_dense_decode_noalloc(const void* q, const void* k, const void* v,
                                    const int32_t* len, int n, int n_kv, int gqa, int head_dim,
                                    int max_len, float scale, void* out, void* stream);

/* ------------------------------------------------------------------------------------------ */
/* A cache held in 4 bits                                                                      */
/* ------------------------------------------------------------------------------------------ */
/* The other way to a smaller cache: every token stays, in 144 bytes per KV head instead of 512.
 * A row of 128 values (K or V of one token) is stored as
 *   codes  64 bytes: e2m1 numbers (sign, magnitudes 0 .5 1 1.5 2 3 4 6), dimension 2 j in the low
 *          half of byte j, 2 j + 1 in the high half;
 *   scales 8 bytes, one per 16 consecutive dimensions: an unsigned number of 5 exponent and 3
 *          mantissa bits (byte b stands for the fp16 number whose bits are b << 7), b <= 226.
 * A row's value is code * scale: at most 6 significant bits, exact in bf16 and in fp16.
 * Quantisation of 16 values x: scale = max|x| / 6 rounded to the nearest such number (ties to
 * even, at most 10240), code = the e2m1 number nearest to x / scale (ties to even, at most 6 in
 * magnitude), with x's sign bit. NaN becomes +0; values beyond +-61440 are clipped to it first;
 * a block whose largest magnitude is at most 3 * 2^-17 becomes zeros.
 *
 * Layouts: k_codes, v_codes [n][n_kv][cap][64], k_scales, v_scales [n][n_kv][cap][8] bytes; paged:
 * pools [num_blocks][n_kv][block][64] and [..][8] with a block table as for the paged calls above,
 * block at least 16. All 16-byte aligned. Rows at and past a unit's length are never read.
 *
 * Workspaces of this part's calls and of the next one's: no *_workspace_bytes falls when one of its
 * arguments grows, so a workspace made for the largest shape serves every smaller one. */

/* Quantise the new_len[u] new rows of every KV head of unit u behind its len[u] cached ones.
 *   new_k, new_v [n][n_kv][max_new][128] bf16: rows 0 .. new_len[u]-1 are taken
 *   new_len  [n] int32 (device) or NULL (max_new rows of every unit)
 *   len      [n] int32: rows in the cache before the call
 *   len_out  [n] int32: len[u] + new_len[u]; may be the same array as len or new_len. A unit with new_len[u]
 *            outside [0, max_new], len[u] < 0 or len[u] + new_len[u] > cap sets
 *            RKV_DEV_LEN_OVER_CAP and is left as it was (len_out[u] = len[u]).
 *   k_values, v_values NULL or [n][n_kv][max_new][128] bf16: the values the rows now stand for
 *            (for a prompt whose own attention is to see what the decode will see); rows past
 *            new_len[u] are left as they were. Both or neither.
 * Paged: a row whose table entry is outside [0, num_blocks) sets RKV_DEV_BAD_INDEX and is not
 * stored (as the decode's new row; block 0 is only read in a block's place).
 * Workspace rkv_kv4_append_workspace_bytes. */
size_t rkv_kv4_append_workspace_bytes(int n);
rkv_status rkv_kv4_append(const void* new_k, const void* new_v, const int32_t* new_len, int n,
                          int n_kv, int head_dim, int max_new, void* k_codes, void* k_scales,
                          void* v_codes, void* v_scales, int cap, const int32_t* len,
                          int32_t* len_out, void* k_values, void* v_values, void* ws,
                          size_t ws_bytes, void* stream);
rkv_status rkv_kv4_append_paged(const void* new_k, const void* new_v, const int32_t* new_len,
                                int n, int n_kv, int head_dim, int max_new, void* k_codes,
                                void* k_scales, void* v_codes, void* v_scales, int num_blocks,
                                int block, const int32_t* block_table, int max_blocks,
                                const int32_t* len, int32_t* len_out, void* k_values,
                                void* v_values, void* ws, size_t ws_bytes, void* stream);

/* One decode step over the 4-bit cache: out[u][h] = softmax(scale * q[u][h] . K[u][g]^T) V[u][g]
 * over the unit's tokens (g = h / gqa), in one pass over the cache. If new_k / new_v are given, the
 * step's token is first quantised into row len[u] (as rkv_kv4_append; the attention sees its
 * quantised row) and len_out[u] = len[u] + 1; a unit that is full sets RKV_DEV_LEN_OVER_CAP,
 * appends nothing and attends to its cap tokens. A unit without tokens gets zeros.
 *   q, out [n][n_kv*gqa][128] bf16; gqa 1, 2, 4 or 8
 *   new_k, new_v NULL or [n][n_kv][128] bf16; len_out [n] int32 (may be len), NULL without them
 *   weights NULL or [n][n_kv][cap] fp32, 16-byte aligned (paged: cap = max_blocks * block): the
 *           softmax weight of every token, summed over the group's query heads, is added to its
 *           entry (rows at and past the length are left as they are, so entries of rows to come
 *           should hold zero)
 * Workspace rkv_kv4_decode_workspace_bytes (cap as above; with_weights: whether weights are asked
 * for, which takes 4 * gqa bytes per cached row). Results do not depend on what the workspace
 * holds, status word apart. */
size_t rkv_kv4_decode_workspace_bytes(int n, int n_kv, int gqa, int cap, int with_weights);
rkv_status rkv_kv4_decode(const void* q, const void* new_k, const void* new_v, void* k_codes,
                          void* k_scales, void* v_codes, void* v_scales, const int32_t* len,
                          int32_t* len_out, int n, int n_kv, int gqa, int head_dim, int cap,
                          float scale, void* out, float* weights, void* ws, size_t ws_bytes,
                          void* stream);
rkv_status rkv_kv4_decode_paged(const void* q, const void* new_k, const void* new_v,
                                void* k_codes, void* k_scales, void* v_codes, void* v_scales,
                                const int32_t* block_table, const int32_t* len, int32_t* len_out,
                                int n, int n_kv, int gqa, int head_dim, int num_blocks, int block,
                                int max_blocks, float scale, void* out, float* weights, void* ws,
                                size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------------------ */
/* Eviction by accumulated attention weight                                                    */
/* ------------------------------------------------------------------------------------------ */
/* SnapKV++ evicts once, by what the last window of the prompt attends to. These calls evict again
 * and again while a sequence grows, by what everything so far has attended to: the prompt call and
 * the decode calls add each token's softmax weight (summed over the query heads of its KV group)
 * to an array, and the eviction keeps the tokens with the largest sums besides the newest ones.
 * A unit's entries start at zero.
 *
 * rkv_dense_decode with the weights: adds sum over the group's heads h of
 * softmax(scale * q[u][h] . K[u][g]^T)[j] to weights[u][g][j], j < len[u].
 *   q, k, v, len, out as rkv_dense_decode (0 <= len[u]: a unit without tokens gets zeros; a longer
 *   one than max_len sets RKV_DEV_LEN_OVER_CAP and counts as max_len). v finite and below 2^100 in
 *   magnitude in the unit's rows: sums of v come before the division by the softmax's sum, and an
 *   infinite value makes NaN of its outputs. Rows past len[u] may hold anything.
 *   weights [n][n_kv][max_len] fp32, 16-byte aligned; rows past len[u] left as they are
 *   (In the prompt call and the evictions 4 bytes are enough for weights and pos.) */
size_t rkv_dense_decode_weights_workspace_bytes(int n, int n_kv, int gqa, int max_len);
rkv_status rkv_dense_decode_weights(const void* q, const void* k, const void* v,
                                    const int32_t* len, int n, int n_kv, int gqa, int head_dim,
                                    int max_len, float scale, void* out, float* weights, void* ws,
                                    size_t ws_bytes, void* stream);

/* The weights of a prompt, or of a chunk of one behind cached tokens: query i < q_len[u] of every
 * head stands at position len[u] - q_len[u] + i and sees the keys up to its own; the softmax weight
 * that key j gets from all of them is added to weights[u][g][j]. (rkv_snapkv_scores without the
 * window's limits: any number of queries, and every key gets its weight.)
 *   q       [n][n_kv*gqa][max_q][128] bf16; rows q_len[u] and up are not used
 *   q_len   [n] int32, 0 <= q_len[u] <= min(max_q, len[u]) (else RKV_DEV_BAD_WINDOW, unit skipped)
 *   k       [n][n_kv][max_len][128] bf16, the chunk's own keys included; rows len[u] and up unused
 *   len     [n] int32, at most max_len (else RKV_DEV_LEN_OVER_CAP, unit skipped)
 *   gqa     1 .. 64
 *   weights [n][n_kv][max_len] fp32
 *   1 <= max_q <= max_len; n * n_kv * gqa * max_q and n * n_kv * max_len at most 2^31 - 513
 *   (RKV_ERR_TOO_LARGE; rkv_prompt_weights_workspace_bytes is 0 for what the call refuses) */
size_t rkv_prompt_weights_workspace_bytes(int n, int n_kv, int gqa, int max_q, int max_len);
rkv_status rkv_prompt_weights(const void* q, const int32_t* q_len, const void* k,
                              const int32_t* len, int n, int n_kv, int gqa, int head_dim,
                              int max_q, int max_len, float scale, float* weights, void* ws,
                              size_t ws_bytes, void* stream);

/* Shrink every unit of more than `keep` rows to `keep`, per KV head: the tokens of the last
 * `recent` positions stay, and of the others those with the largest weights (ties -> lower row;
 * NaN counts as largest). Kept rows below `keep` do not move; the i-th free row below `keep`
 * takes the i-th kept row at or past `keep`, so a step that evicts few rows moves few, and rows
 * are in no particular order of position (attention does not depend on it; page summaries have
 * to be rebuilt). A unit of at most `keep` rows is left as it is.
 *   k, v     [n][n_kv][cap][128] bf16, or the 4-bit arrays: moved in place
 *   len      [n] int32; len_out [n] int32: min(len[u], keep); may be the same array, or seen
 *   weights  [n][n_kv][cap] fp32, pos [n][n_kv][cap] int32: a row's position in its sequence, or -1
 *            for a row appended since the last eviction (its position is then
 *            seen[u] - (len[u] - row)); all -1 at first
 *   seen     [n] int32: tokens the sequence has had so far (the position of the next one)
 *   weights_out, pos_out: the arrays after the move (may be the same arrays): rows below
 *            len_out[u] belong to the rows now there (of an evicted unit, every position is
 *            known), rows from len_out[u] to len[u] - 1 are reset (0 and -1), later rows are left
 *            as they were
 *   src_rows NULL or [n][n_kv][keep] int32: the row each row came from, -1 past len_out[u]
 *   0 <= recent <= keep, 1 <= keep. len[u] outside [0, cap]: RKV_DEV_LEN_OVER_CAP, unit left as it
 *   was (len_out[u] = len[u]; weights_out, pos_out and src_rows not written). */
size_t rkv_evict_workspace_bytes(int n, int n_kv, int cap, int keep);
rkv_status rkv_evict(void* k, void* v, const int32_t* len, int32_t* len_out, const float* weights,
                     float* weights_out, const int32_t* pos, int32_t* pos_out,
                     const int32_t* seen, int n, int n_kv, int head_dim, int cap, int keep,
                     int recent, int32_t* src_rows, void* ws, size_t ws_bytes, void* stream);
rkv_status rkv_evict_kv4(void* k_codes, void* k_scales, void* v_codes, void* v_scales,
                         const int32_t* len, int32_t* len_out, const float* weights,
                         float* weights_out, const int32_t* pos, int32_t* pos_out,
                         const int32_t* seen, int n, int n_kv, int head_dim, int cap, int keep,
                         int recent, int32_t* src_rows, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------------------ */
/* A serving step around the cache: places, rotary positions, attention of packed tokens        */
/* ------------------------------------------------------------------------------------------ */
/* What fills the caches that the calls above compress and read, and the steps that have more than
 * one query per request. A step's new tokens of all units lie packed, token-major: unit u has the
 * tokens q_start[u] .. q_start[u+1]-1 of arrays [tokens][heads][128] (q_start [n+1] int32). q, k
 * and v may be slices of one projection's output: their tokens are `*_stride` elements apart (a
 * multiple of 8, at least heads * 128), the heads of one token contiguous.
 * A slot names a row of every KV head: slot = b * block + r is row r of block b of pools
 * [num_blocks][n_kv][block][128]; a contiguous cache [n][n_kv][cap][128] is the pool of n blocks of
 * cap rows (any block size >= 1 is taken here). A negative slot is no place. n is at most 2^30.
 * No *_workspace_bytes of this part falls when one of its arguments grows (0 for what is refused).
 *
 * Block tables and slots on the device. The free blocks are a stack: free_blocks [num_blocks]
 * int32, entries 0 .. free_count[0]-1, the top last.
 *
 * rkv_reserve_slots: a place for new_len[u] more tokens of every unit behind its len[u] ones.
 *   new_len, len, held [n] int32: held[u] blocks of block_table [n][max_blocks] are the unit's
 *            already, ceil(len / block) at least (blocks kept after a sequence was cut are used
 *            first); entries from held[u] on are not read
 *   block    tokens of a block; n, block, num_blocks, max_blocks, max_tokens >= 1; num_blocks * block,
 *            max_blocks * block and max_tokens at most 2^30
 *   block_table  entries held[u] .. of a unit that needs more blocks are written: they come off the
 *            top of the stack in the order of the units. free_blocks itself is only read.
 *   q_start  [n+1] int32: prefix sums of new_len (a negative one counts as 0)
 *   slots, positions [max_tokens] int32: slot and position (len[u] + i) of every new token; -1 and
 *            0 for tokens of units not served, and behind the last token (so a batch padded to
 *            max_tokens stores nothing there)
 *   len_out, held_out, free_count_out: the values after the call (may be the input arrays)
 * A unit is served or left as it was. Not served: len, new_len or held out of range, or len + new_len
 * above max_blocks * block, or tokens that do not fit in max_tokens (RKV_DEV_LEN_OVER_CAP); fewer
 * blocks held than its tokens need, or a block outside [0, num_blocks) among those that its new
 * tokens go to (RKV_DEV_BAD_INDEX; in the latter case those tokens alone have no place); blocks
 * needed, and more needed by it and the units before it, served or not, than are free
 * (RKV_DEV_NO_BLOCKS). free_count outside [0, num_blocks]: RKV_DEV_BAD_INDEX, none is free.
 * q_start counts the tokens of a unit that is not served too, where they lie in the packed arrays. With their
 * slots of -1 rkv_rope_append leaves them out (nothing is stored, q_out stays), but the attentions below know
 * q_start and len alone: they take the last rows of the unit's old length for those of the new tokens and write
 * outputs that mean nothing, and report nothing themselves unless the unit has fewer rows than that. So the status
 * of this call is to be checked before a step's outputs are used (one workspace for the step's calls gathers
 * their statuses); the units concerned are those whose new tokens' slots are all -1. */
size_t rkv_reserve_slots_workspace_bytes(int n);
rkv_status rkv_reserve_slots(const int32_t* new_len, const int32_t* len, const int32_t* held,
                             int32_t* block_table, const int32_t* free_blocks,
                             const int32_t* free_count, int n, int num_blocks, int block,
                             int max_blocks, int max_tokens, int32_t* q_start, int32_t* slots,
                             int32_t* positions, int32_t* len_out, int32_t* held_out,
                             int32_t* free_count_out, void* ws, size_t ws_bytes, void* stream);

/* The way back: every unit keeps the ceil(len[u] / block) blocks that its tokens need (none with
 * len[u] = 0), the others of its held[u] go to the stack, in the order of units and of the table.
 * held_out, free_count_out may be the input arrays; block_table is only read. A unit with len < 0 or
 * held outside [0, max_blocks] sets RKV_DEV_LEN_OVER_CAP and keeps all. If more would come back than
 * the pool can lack (num_blocks - free_count), RKV_DEV_BAD_INDEX is set and nothing is released; a
 * table entry outside [0, num_blocks) sets it too and goes to the stack as it is. */
size_t rkv_release_blocks_workspace_bytes(int n);
rkv_status rkv_release_blocks(const int32_t* len, const int32_t* held, const int32_t* block_table,
                              int32_t* free_blocks, const int32_t* free_count, int n,
                              int num_blocks, int block, int max_blocks, int32_t* held_out,
                              int32_t* free_count_out, void* ws, size_t ws_bytes, void* stream);

/* Rotary positions. rkv_rope_frequencies (host): inv_freq[i] of the rot_dim / 2 pairs, and mscale.
 *   RKV_ROPE_PLAIN    base^(-2 i / rot_dim)
 *   RKV_ROPE_LINEAR   divided by factor (positions as if interpolated)
 *   RKV_ROPE_BASE     plain with base * factor^(rot_dim / (rot_dim - 2)): the slowest pair is slower
 *                     by factor, the fastest unchanged (rot_dim >= 4)
 *   RKV_ROPE_BY_PARTS pairs that turn more than `fast` times within the original context `ctx` keep
 *                     their frequency, those that turn fewer than `slow` times are divided by
 *                     factor, linear in the pair's number between the (real) numbers of these two;
 *                     mscale = 0.1 ln(factor) + 1 (factor > 1)
 *   RKV_ROPE_SMOOTH   the same with a ramp linear in the number of turns; mscale 1
 *   RKV_ROPE_BY_WHOLE_PARTS  RKV_ROPE_BY_PARTS with the ramp's ends rounded outward, down to a whole pair's number
 *                     for `fast` and up for `slow`, both brought into [0, rot_dim - 1] (the ramp of equal ends is
 *                     0.001 long). Models that were scaled by parts were made with one or the other: with 128
 *                     dimensions, base 1e6, ctx 32768, fast 32 and slow 1 the ends are 23.6 and 39.7, or 23 and 40,
 *                     and frequencies on the ramp are some per cent apart
 * factor >= 1; ctx > 0, fast > slow > 0 for the last three (ignored by the others). rot_dim even,
 * 2 .. 128; base > 1. Errors: RKV_ERR_INVALID_ARG. */
#define RKV_ROPE_PLAIN 0
#define RKV_ROPE_LINEAR 1
#define RKV_ROPE_BASE 2
#define RKV_ROPE_BY_PARTS 3
#define RKV_ROPE_SMOOTH 4
#define RKV_ROPE_BY_WHOLE_PARTS 5
rkv_status rkv_rope_frequencies(int kind, int rot_dim, double base, double factor, int ctx,
                                double fast, double slow, float* inv_freq, float* mscale);

/* Turn the queries and keys of the new tokens to their positions and store the keys and values.
 * For every token t with slots[t] >= 0, pair i < rot_dim / 2 of each head of q and k,
 *   (a, b) -> mscale (a cos w - b sin w, b cos w + a sin w),   w = positions[t] * inv_freq[i],
 * (a, b) being dimensions (i, i + rot_dim / 2), or (2 i, 2 i + 1) if interleaved; dimensions from
 * rot_dim on stay as they are. fp32 arithmetic, rounded once; w is reduced exactly, however far
 * the position (any int32).
 *   q [tokens][hq][128], k, v [tokens][n_kv][128] bf16 with strides as above; inv_freq
 *   [rot_dim / 2] fp32; positions, slots [tokens] int32
 *   q_out    [tokens][hq][128] bf16, contiguous; may be q (then q_stride = hq * 128)
 *   k_pool, v_pool [num_blocks][n_kv][block][128] bf16: row slots[t] of every KV head
 *   rot_dim  a multiple of 16, 16 .. 128; hq >= 1 (hq need not be a multiple of n_kv)
 * A token with a negative slot is left out: none of its rows is written. A slot at or past
 * num_blocks * block sets RKV_DEV_BAD_INDEX, and the token is left out. Two tokens with one slot
 * leave rows of either of them there, or pieces of both. */
size_t rkv_rope_append_workspace_bytes(void);
rkv_status rkv_rope_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                           const void* v, int64_t v_stride, const int32_t* positions,
                           const float* inv_freq, const int32_t* slots, int tokens, int hq,
                           int n_kv, int head_dim, int rot_dim, int interleaved, float mscale,
                           void* q_out, void* k_pool, void* v_pool, int num_blocks, int block,
                           void* ws, size_t ws_bytes, void* stream);

/* Attention of a prompt, or of a chunk of one behind cached tokens: out[t][h] = softmax(scale *
 * q[t][h] . K^T) V of KV head h / gqa of t's unit over the keys up to t's own. The unit's rows in the
 * cache (len[u]) include those of its T = q_start[u+1] - q_start[u] new tokens, which are its last
 * ones: token i stands at position len[u] - T + i. (One token each is a decode step.)
 *   q        [tokens][n_kv*gqa][128] bf16, tokens q_stride elements apart
 *   q_start  [n+1] int32 (device), ascending, within [0, tokens]
 *   k, v     [n][n_kv][max_len][128] bf16, or pools with a block table as for the paged calls above
 *            (block a power of two). Rows from len[u] on may hold anything; rows before that have
 *            finite values, v below 2^80 in magnitude (sums of v come before the division by the
 *            softmax's sum; an infinite or NaN value of v makes NaN of outputs that do not see it).
 *   len      [n] int32 (device), T <= len[u] <= max_len (paged: max_blocks * block)
 *   out      [tokens][n_kv*gqa][128] bf16, contiguous; may not overlap q. Rows of tokens that belong
 *            to no unit are left as they were.
 *   gqa      1 .. 64
 *   scores   scale log2(e) q . k below 2^28 in magnitude for every row that a token sees (beyond that, fp32
 *            numbers are 16 and more apart, and numerators relative to a rounded score may overflow)
 * len out of range: RKV_DEV_LEN_OVER_CAP; q_start out of order or range, or T > len[u]:
 * RKV_DEV_BAD_WINDOW; the unit is skipped, its rows left as they were. A table entry outside the pool
 * among the unit's blocks: RKV_DEV_BAD_INDEX, block 0 is read. RKV_ERR_TOO_LARGE where tokens * n_kv *
 * gqa, or the rows of k, exceed 2^31 - 513. The softmax's numerators are rounded to bf16 for the
 * product with V; everything else is fp32. */
size_t rkv_prompt_attention_workspace_bytes(int n, int n_kv, int gqa, int tokens);
rkv_status rkv_prompt_attention(const void* q, int64_t q_stride, const int32_t* q_start,
                                const void* k, const void* v, const int32_t* len, int n, int n_kv,
                                int gqa, int head_dim, int tokens, int max_len, float scale,
                                void* out, void* ws, size_t ws_bytes, void* stream);
rkv_status rkv_prompt_attention_paged(const void* q, int64_t q_stride, const int32_t* q_start,
                                      const void* k_pool, const void* v_pool,
                                      const int32_t* block_table, const int32_t* len, int n,
                                      int n_kv, int gqa, int head_dim, int tokens, int num_blocks,
                                      int block, int max_blocks, float scale, void* out, void* ws,
                                      size_t ws_bytes, void* stream);

/* The same for a tree of drafted tokens: the unit's T new tokens see all of the len[u] - T rows before
 * theirs, and among theirs those that a bit mask names: token t sees row len[u] - T + j iff bit j % 32
 * of mask[t][j / 32] is set (its ancestors and itself; any mask is taken, bits from T on are ignored).
 *   mask     [tokens][mask_words] int32, 1 <= mask_words <= 32; T <= 32 * mask_words (else
 *            RKV_DEV_BAD_WINDOW, unit skipped)
 * A token that sees nothing gets zeros. The drafted rows are in the cache in the tokens' order,
 * whatever their positions (a token's position is the number of its ancestors behind the cached ones);
 * the rows of those that were accepted are stored again in place (rkv_rope_append), the length then
 * covers them only. Workspace rkv_prompt_attention_workspace_bytes; the rest as above. */
rkv_status rkv_tree_attention(const void* q, int64_t q_stride, const int32_t* q_start,
                              const int32_t* mask, int mask_words, const void* k, const void* v,
                              const int32_t* len, int n, int n_kv, int gqa, int head_dim,
                              int tokens, int max_len, float scale, void* out, void* ws,
                              size_t ws_bytes, void* stream);
rkv_status rkv_tree_attention_paged(const void* q, int64_t q_stride, const int32_t* q_start,
                                    const int32_t* mask, int mask_words, const void* k_pool,
                                    const void* v_pool, const int32_t* block_table,
                                    const int32_t* len, int n, int n_kv, int gqa, int head_dim,
                                    int tokens, int num_blocks, int block, int max_blocks,
                                    float scale, void* out, void* ws, size_t ws_bytes,
                                    void* stream);

#ifdef __cplusplus
}
#endif

#endif /* RKV_H_ */
