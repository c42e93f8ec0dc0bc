/*
 * specverify_kv.h — C ABI of the paged key-value cache around a verify step, on GB300.
 *
 *   paged_attention       attention of the n_r + 1 new positions of each request over its
 *                         paged cache (n_r drafts and the token ahead of them; n_r = 0 is
 *                         plain decoding), split over the cache's length and joined.
 *   attention_weight_sum  adds to each cached key the softmax weight that the accepted
 *                         positions of a step gave it.
 *   kv_cache_evict        keeps the most recent and the heaviest keys of each cache.
 *
 * A step chains them: paged_attention per layer, the verify call, whose accept_len then tells
 * attention_weight_sum which rows count; kv_cache_evict once a cache passes its budget.
 *
 * The conventions of specverify.h hold.
 */
#ifndef SPECVERIFY_KV_H_
#define SPECVERIFY_KV_H_

#include "specverify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Types of queries, keys, values and outputs. */
typedef enum {
  SV_KV_BF16 = 1, /* bfloat16 (the value of SV_BF16) */
  SV_KV_F16 = 2   /* IEEE binary16 */
} sv_kv_dtype;

/* A pool of pages holding keys or values: element d of kv head h of the token in slot s of
 * page p is at data[p * page_stride + s * token_stride + h * head_stride + d] (strides in
 * elements, so both [pages, page_size, heads, D] and [pages, heads, page_size, D] fit).
 * data must be 16-byte aligned and every stride a positive multiple of 8 elements. This
 * struct is HOST memory, read during the call. */
typedef struct {
  void* data;
  int64_t page_stride, token_stride, head_stride;
} sv_kv_pool;

/* Sizes shared by the calls below. HOST memory, read during the call.
 *   dtype       of queries, keys, values and outputs.
 *   B           requests, B >= 0 (0 is a no-op).
 *   P           query positions per request, 1 <= P <= SV_MAX_K + 1.
 *   Hq, Hkv     query and key-value heads, Hq a multiple of Hkv; query heads h*G .. h*G+G-1
 *               (G = Hq / Hkv) read kv head h. G <= 64, Hkv <= 1024, else SV_ERR_UNSUPPORTED.
 *   D           head width: 64, 128 or 256, else SV_ERR_UNSUPPORTED.
 *   page_size   slots per page: a power of two from 8 to 1024, else SV_ERR_UNSUPPORTED.
 *   num_pages   pages in the pool.
 *   max_pages   columns of the page table; max_pages * page_size < 2^30.  */
typedef struct {
  sv_kv_dtype dtype;
  int B, P, Hq, Hkv, D, page_size, num_pages, max_pages;
} sv_kv_shape;

/* How a row scores a key. HOST memory, read during the call.
 *   scale    multiplies q.k; finite.
 *   softcap  0 for none, else c >= 1e-6: the scaled score s becomes c * tanh(s / c).
 *   window   0 for none, else a row at position p sees keys p - window + 1 .. p only.
 *   slopes   DEVICE [Hq] fp32 or NULL: the capped score of a key at position j falls by
 *            slopes[h] * (p - j).
 * Positions are cache slots: after an eviction distances count kept keys. */
typedef struct {
  float scale, softcap;
  int window;
  const float* slopes;
} sv_score_rule;

/* ------------------------------------------------------------------------------------------
 * Attention over the paged cache. Request r holds n = seq_len[r] tokens, those of its
 * n_r + 1 new positions (their keys and values already in the pool) included. Row i
 * (0 <= i <= n_r) of head h is the token at position p_i = n - 1 - n_r + i:
 *   s_j  = score of key j under the rule, for the keys 0 <= j <= p_i it sees
 *   lse  = log(sum_j exp(s_j)),  out = sum_j exp(s_j - lse) v_j
 * A row that sees no key (p_i < 0) gets out = 0 and lse = -inf.
 *
 * Arguments
 *   q            [B, P, Hq, D]; element strides q_req, q_row, q_head (multiples of 8), D
 *                contiguous, 16-byte aligned. What rows past n_r hold reaches no output.
 *   k, v         pools of num_pages pages.
 *   page_table   [B, max_pages] int32: page t of request r holds tokens t*page_size on. Only
 *                pages that hold a key some row sees are looked up.
 *   seq_len      [B] int32 in [0, max_pages * page_size].
 *   num_draft    [B] int32 in [0, P-1], or NULL for all P-1.
 *   out          [B, P, Hq, D] contiguous. Rows past n_r are not written.
 *   out_lse      [B, P, Hq] fp32, or NULL.
 *   workspace    >= paged_attention_workspace(shape) bytes; needs no initialisation.
 * What slots past n hold never reaches an output (NaN included), nor does a drafted token's
 * value reach the rows ahead of it. A value that is infinite or NaN makes what it enters infinite or
 * NaN: the sum, over the keys a row sees, of that component's values that are not finite.
 * A request with seq_len or num_draft out of range gets NaN in out and out_lse in all its P
 * rows; one whose page table names a page outside [0, num_pages) for a key that is seen, NaN
 * at least in the rows that see such a key.
 * Scores, their softmax and the sums over values are fp32; the weights exp(s_j - max) enter the
 * product with the values as a sum of numbers of the values' type: off by 2^-22 of a weight (fp16),
 * or 2^-24 (bf16, up to 32 query rows per kv head and pass) or 2^-16 (bf16, more). The work is split
 * over the SMs by a rule on the lengths alone and joined in order: equal calls give equal bits.
 * ---------------------------------------------------------------------------------------- */
size_t paged_attention_workspace(const sv_kv_shape* shape);

sv_status paged_attention(const sv_kv_shape* shape, const sv_score_rule* rule, const void* q,
                          int64_t q_req, int64_t q_row, int64_t q_head, const sv_kv_pool* k,
                          const sv_kv_pool* v, const int32_t* page_table,
                          const int32_t* seq_len, const int32_t* num_draft, void* out,
                          float* out_lse, void* workspace, size_t workspace_bytes,
                          sv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * Self-tests of the bounded waits inside paged_attention and attention_weight_sum: the same calls
 * with each wait limited to wait_us microseconds (1 .. 100000) instead of 2 s, so that ordinary
 * waits run out. No fault and no hang: a CTA whose wait ran out waits for its own copies and
 * instructions, writes NaN to everything in its share of the work and ends. Every row, and every
 * key weight, is then either what the call gives or NaN, and the device stays usable.
 * Returns SV_ERR_INVALID_ARG for wait_us out of range, else what the call returns.
 * ---------------------------------------------------------------------------------------- */
sv_status paged_attention_wait_selftest(
    const sv_kv_shape* shape, const sv_score_rule* rule, const void* q, int64_t q_req,
    int64_t q_row, int64_t q_head, const sv_kv_pool* k, const sv_kv_pool* v,
    const int32_t* page_table, const int32_t* seq_len, const int32_t* num_draft, void* out,
    float* out_lse, void* workspace, size_t workspace_bytes, unsigned int wait_us,
    sv_stream_t stream);

sv_status attention_weight_sum_wait_selftest(
    const sv_kv_shape* shape, const sv_score_rule* rule, const void* q, int64_t q_req,
    int64_t q_row, int64_t q_head, const sv_kv_pool* k, const int32_t* page_table,
    const int32_t* seq_len, const int32_t* num_draft, const float* lse, int64_t lse_req,
    int64_t lse_row, int64_t lse_head, const int32_t* accept_len, const float* prior, float* out,
    int64_t stride, unsigned int wait_us, sv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * The weight each key received. With rows and scores as in paged_attention, for every slot
 * j < seq_len[r] of kv head h:
 *   out[r, h, j] = prior[r, h, j] + sum over rows i <= accept_len[r] and the G query heads of
 *                  h of exp(s_j - lse[r, i, head])   where the row sees key j
 * Rows of rejected drafts do not count. Where lse is -inf the row counts for nothing.
 *
 * Arguments
 *   q, k, page_table, seq_len, num_draft   as in paged_attention.
 *   lse          [B, P, Hq] fp32, as paged_attention returned it; element strides lse_req,
 *                lse_row, lse_head (>= 0).
 *   accept_len   [B] int32, a verify call's accept_len (-1: no row of the request counts), or
 *                NULL: all n_r + 1 rows count.
 *   prior        [B, Hkv, stride] fp32 or NULL for zero; may be `out`.
 *   out          [B, Hkv, stride] fp32; slots at or past seq_len[r] are not written.
 *   stride       slots per (request, head) in prior and out, >= max_pages * page_size or at
 *                least every seq_len; a request whose seq_len is above it is out of range.
 * A request with seq_len, num_draft or accept_len (above num_draft) out of range is left
 * unwritten but for out[r, :, 0] = NaN (stride >= 1); a page outside [0, num_pages) gives NaN
 * in those of its slots that a counted row sees.
 * No workspace.
 * ---------------------------------------------------------------------------------------- */
sv_status attention_weight_sum(const sv_kv_shape* shape, const sv_score_rule* rule,
                               const void* q, int64_t q_req, int64_t q_row, int64_t q_head,
                               const sv_kv_pool* k, const int32_t* page_table,
                               const int32_t* seq_len, const int32_t* num_draft,
                               const float* lse, int64_t lse_req, int64_t lse_row,
                               int64_t lse_head, const int32_t* accept_len,
                               const float* prior, float* out, int64_t stride,
                               sv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * Eviction. For each request r of n = seq_len[r] tokens and each kv head h, m = min(n,
 * budget) slots are kept: all of them when n <= budget, else the last `recent` and, of the
 * others, the budget - recent of largest weight (equal weights: the lower slots; NaN counts
 * as -inf). Kept slots are copied in ascending order to slots 0 .. m-1 of new pages: a
 * cache's old pages may be shared with other requests and are only read.
 *
 * Arguments
 *   shape        dtype, B, Hkv, D, page_size, num_pages, max_pages (P and Hq are not used).
 *   k, v         the pools the pages are read from.
 *   page_table   [B, max_pages] int32; seq_len [B] int32 in [0, max_pages * page_size].
 *   weights      [B, Hkv, stride] fp32, stride as above.
 *   budget       1 <= budget <= new_max_pages * page_size and < 2^30.
 *   recent       0 <= recent <= budget.
 *   new_k, new_v pools of new_num_pages pages of the same page_size, which may be the pools k
 *                and v: the new pages must then be none of the pages read in this call.
 *   new_table    [B, new_max_pages] int32: distinct pages for the kept slots.
 *   out_len      [B] int32: m, or -1 for a request with a data error.
 *   out_index    [B, Hkv, budget] int32: the old slot of each kept one, then -1.
 *   out_weights  [B, Hkv, budget] fp32: the kept slots' weights, then 0; or NULL.
 * B * Hkv is at most 65535, else SV_ERR_UNSUPPORTED. out_len must not overlap seq_len, nor
 * out_weights weights, else SV_ERR_INVALID_ARG.
 * A request with seq_len out of range (or above stride) or with a page outside its pool's
 * range among those it needs, in either table, gets out_len = -1, out_index all -1 and
 * out_weights all 0, and nothing of it is copied.
 * ---------------------------------------------------------------------------------------- */
sv_status kv_cache_evict(const sv_kv_shape* shape, const sv_kv_pool* k, const sv_kv_pool* v,
                         const int32_t* page_table, const int32_t* seq_len,
                         const float* weights, int64_t stride, int budget, int recent,
                         const sv_kv_pool* new_k, const sv_kv_pool* new_v, int new_num_pages,
                         const int32_t* new_table, int new_max_pages, int32_t* out_len,
                         int32_t* out_index, float* out_weights, sv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_KV_H_ */
