/*
 * kv_cache.h -- C ABI of a paged key/value cache and the operators on it: the
 * attention of new (drafted) tokens over the cache, appending accepted tokens,
 * accumulating the attention weight of cached keys, and evicting the lightest
 * ones. Same library (libgemm_tn.so), status codes and conventions as
 * gemm_tn.h.
 *
 * The cache. K and V live in pools of pages. Slot s of sequence b is row
 * s % page_size of page page_table[b][s / page_size]; its row of KV head h is
 * head_dim contiguous 16-bit elements at
 *     page * page_stride + row * slot_stride + h * head_stride
 * in either pool (strides in elements, the same for K and V; multiples of 8:
 * every row starts on a 16-byte boundary). Both [page][row][head] and
 * [page][head][row] orders are such strides. A sequence uses slots 0 ..
 * lens[b] - 1; what lies behind them, in its last page or in other pages, is
 * never read into a result and may hold anything, NaN included. lens, the
 * page table and the per-sequence counts below are read on the device, in
 * stream order: a captured launch follows them from replay to replay.
 *
 * Query heads are grouped: KV head h serves the `group` = heads / kv_heads
 * query heads h * group .. h * group + group - 1.
 *
 * Conventions beside those of gemm_tn.h:
 *   - Pools, inputs and outputs of 16-bit elements are 16-byte aligned; int32
 *     and fp32 arrays 4-byte, the mask 8-byte.
 *   - Values on the device that the host cannot check are made safe there:
 *     lengths and counts are clamped to [0, what the arrays hold], and an entry
 *     of the page table (or of `rows`) in use that is out of range is not
 *     followed: GEMM_TN_ERR_INVALID_VALUE is stored in *d_status if d_status
 *     is not NULL (the first error wins, as for the watchdog's timeout), reads
 *     through it count as zeros and writes through it are left out.
 *   - The device watchdog (GEMM_TN_WATCHDOG_MS) bounds every wait of
 *     tree_attn_fwd and kv_cache_weigh. GEMM_TN_TEST_DROP_LOAD=<tile> is their
 *     test hook: the first CTA skips the K load of its tile of that number.
 *   - Pages that a call writes (append, evict) belong to one sequence only;
 *     pages that are only read may be shared.
 *   - An output (the pools, weight and pos too where they are written, and the
 *     status word) overlaps no other array of the call, used by it or not
 *     (INVALID_VALUE), except that it may be, exactly, the cache's array that it
 *     replaces. The K and V pools of append and evict may lie between one
 *     another's rows (K and V of a page or of a slot side by side) but share none.
 *   - Results are repeatable to the bit: no atomics touch them.
 *   - Serving only: there are no gradients.
 */
#ifndef KV_CACHE_H_
#define KV_CACHE_H_

#include <stdint.h>

#include "gemm_tn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct kv_cache {
  void* k;                    /* device pools */
  void* v;
  int64_t num_pages;          /* pages in each pool, < 2^31 */
  int64_t page_size;          /* rows per page: 8, 16, 32, 64 or a multiple of 128 up to 2^20 */
  int64_t kv_heads;
  int64_t head_dim;           /* 64 or 128 */
  int64_t page_stride;        /* elements, multiples of 8, below 2^39 */
  int64_t slot_stride;
  int64_t head_stride;
  const int32_t* page_table;  /* device [batch] rows of max_pages entries, table_stride apart */
  int64_t table_stride;
  int64_t max_pages;          /* max_pages * page_size = capacity, the most slots a sequence can use, < 2^31 */
  int32_t* lens;              /* device [batch]: slots in use */
  /* The next three are needed where an operator says so, and NULL otherwise. */
  float* weight;              /* device [batch][kv_heads][capacity]: accumulated attention weight */
  int32_t* pos;               /* device [batch][kv_heads][capacity]: position of the token in the slot */
  int32_t* seen;              /* device [batch]: tokens appended so far = the next token's position */
} kv_cache;

/* A [batch][tokens][heads] array of head_dim-long rows: strides in elements, multiples of 8. */
typedef struct kv_rows {
  const void* data;
  int64_t batch_stride;
  int64_t token_stride;
  int64_t head_stride;
} kv_rows;

/*
 * tree_attn_fwd -- attention of `tokens` new tokens per sequence over the
 * sequence's cached keys and over one another:
 *
 *   s(i, k) = scale * q_i . k     k over slots 0 .. lens[b]-1, all seen by every
 *                                 new token, then over the new tokens i sees
 *   o[b][i][x] = sum_k softmax(s)_k v_k        lse[b][i][x] = log sum_k exp(s_k)
 *
 * for i < token_lens[b] (NULL: tokens); rows of o and lse from there on are
 * left as they were. k_new and v_new hold the new tokens' keys and values
 * [batch][tokens][kv_heads]; they need not be (and are not put) in the cache.
 * NULL for both: the new tokens see the cache only (append first, then attend).
 * mask: device [batch][tokens][mask_words] 64-bit words, mask_words =
 * ceil(tokens / 64): new token i sees new token j when bit j % 64 of word
 * j / 64 of mask[b][i] is set, and j < token_lens[b]. A drafted tree sets each
 * token's ancestors and itself. NULL: the causal chain, j <= i. A new token
 * that sees no key gives o = 0 and lse = -inf. The values of a new token that
 * another one must not see have to be finite all the same (its probability is
 * a zero in a matrix product).
 *
 * One token per sequence is a decode step; many tokens with a NULL mask are
 * the next chunk of a prompt. Scores, softmax statistics, the accumulated
 * output and lse are fp32; probabilities are rounded to the input type before
 * the product with V, o to nearest-even at the end. Against the exact result
 * |o - ref| <= 1e-2 * sum_k p_k |v_k| + 1e-3.
 * o: device [batch][tokens][heads][head_dim], contiguous; lse: device fp32
 * [batch][tokens][heads] or NULL. softmax_scale: 0 selects 1/sqrt(head_dim).
 * Limits: heads a multiple of kv_heads, group <= 128; sizes below 2^31.
 * Parts of long sequences go through a workspace from the library's pool
 * (gemm_tn_workspace_pool), allocated and freed on `stream`.
 * Errors: GEMM_TN_ERR_INVALID_VALUE, _UNSUPPORTED_DTYPE, _MISALIGNED,
 * _UNSUPPORTED_DEVICE, _CUDA; nothing is enqueued on error.
 */
GEMM_TN_API int tree_attn_fwd(int dtype, int64_t batch, int64_t tokens, int64_t heads, const kv_cache* cache,
                              const kv_rows* q, const kv_rows* k_new, const kv_rows* v_new, const uint64_t* mask,
                              const int32_t* token_lens, void* o, float* lse, float softmax_scale, int* d_status,
                              gemm_tn_stream_t stream);

/*
 * kv_cache_append -- puts tokens into the cache: for i < counts[b] (NULL:
 * max_rows) row rows[b][i] of k_new and v_new (NULL: row i; [batch][max_rows])
 * goes to slot lens[b] + i; where the cache has them, weight is zeroed and pos
 * set to seen[b] + i (lens[b] + i without seen) for every KV head. Then
 * lens_out[b] = lens[b] + counts[b] and seen_out[b] = seen[b] + counts[b];
 * lens_out and seen_out may be lens and seen (a second small kernel then
 * writes them). seen_out: NULL without seen. Slots past the capacity are not
 * written, lens_out stops there and the status word is set.
 */
GEMM_TN_API int kv_cache_append(int dtype, int64_t batch, int64_t tokens, const kv_cache* cache, const kv_rows* k_new,
                                const kv_rows* v_new, const int32_t* rows, const int32_t* counts, int64_t max_rows,
                                int32_t* lens_out, int32_t* seen_out, int* d_status, gemm_tn_stream_t stream);

/*
 * kv_cache_weigh -- accumulates attention weight: for every slot s < lens[b]
 *
 *   weight_out[b][h][s] = weight[b][h][s]
 *       + sum_{i < counts[b]} sum_{x of h} exp(scale * q_(row i, x) . k_s - lse[b][row i][x])
 *
 * over the counted rows rows[b][i] of q and lse ([batch][tokens][heads], lse as
 * tree_attn_fwd writes it). causal non-zero: the counted rows are the queries of
 * the newest counts[b] slots, in order, and row i counts for slots s <
 * lens[b] - counts[b] + i + 1 only; zero: every row counts for every slot.
 * A counted row adds nothing where its lse is infinite (-inf: it saw no key) or
 * its entry of rows is out of range, whatever the keys hold; neither does a row
 * to a slot that it does not count for.
 * weight_out may be cache->weight; entries from lens[b] on are left as they
 * were. Sums are fp32. The same limits and errors as tree_attn_fwd.
 */
GEMM_TN_API int kv_cache_weigh(int dtype, int64_t batch, int64_t tokens, int64_t heads, const kv_cache* cache,
                               const kv_rows* q, const float* lse, const int32_t* rows, const int32_t* counts,
                               int64_t max_rows, int causal, float softmax_scale, float* weight_out, int* d_status,
                               gemm_tn_stream_t stream);

/*
 * kv_cache_evict -- cuts every sequence longer than `keep` down to `keep`
 * slots, for each KV head by its own weights: the slots with pos >= seen[b] -
 * recent stay, then those with the largest weight (NaN counts above
 * everything else, equal weights stay in slot order, lowest first). Kept
 * slots below `keep` stay in place; the kept slots behind, in ascending order,
 * fill the holes in ascending order, in K, V, weight and pos. The order of
 * slots is therefore not the order of positions afterwards: pos tells.
 * weight_out, pos_out and lens_out (slots of longer sequences from `keep` on
 * and of shorter ones from lens[b] on are left as they were; lens_out[b] =
 * min(lens[b], keep)) may be the cache's own weight, pos and lens. pos and
 * seen may be NULL when recent is 0; pos_out is NULL exactly when pos is.
 * 0 <= recent <= keep. K and V behind the new length keep their old contents.
 * Limits: capacity <= 2^31 - 2^16, batch * kv_heads <= 2^30.
 * The list of moves is a workspace from the library's pool.
 */
GEMM_TN_API int kv_cache_evict(int dtype, int64_t batch, const kv_cache* cache, int64_t keep, int64_t recent,
                               float* weight_out, int32_t* pos_out, int32_t* lens_out, int* d_status,
                               gemm_tn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KV_CACHE_H_ */
