/*
 * specverify_kv8.h — C ABI of the paged key-value cache held in 8 bits, on GB300.
 *
 *   kv_cache_append_q8   rounds the keys and values of new tokens to 8 bits, with a scale for each
 *                        block of tokens and kv head, and puts them into their slots.
 *   paged_attention_q8   attention of the new positions over such a cache.
 *
 * Half the bytes of the cache of specverify_kv.h, so about twice its tokens. Its attention takes 0.57 of
 * the other's time with 4 query rows per kv head, 0.62 with 12, 0.8 with 24 to 32 and 0.9 with 48, and
 * from 49 to 64 more time for less memory (64 requests of 200 .. 8192 keys).
 * Codes are e4m3 (sign, 4 exponent bits of bias 7, 3 mantissa bits; largest
 * 448, no infinity; 0x7f and 0xff are NaN). The element a code stands for is code * scale.
 *
 * A pool is an sv_kv_pool of codes: strides in elements (bytes), positive multiples of 16, data
 * 16-byte aligned, D contiguous. Its scales are [num_pages, page_size / block, Hkv] fp32,
 * contiguous: slots b*block .. b*block + block-1 of a page share one. `block` is a power of two,
 * at most 128 and at most page_size. Scales lie in [2^-40, 2^40], or are 0.
 *
 * The conventions of specverify.h and specverify_kv.h hold.
 */
#ifndef SPECVERIFY_KV8_H_
#define SPECVERIFY_KV8_H_

#include "specverify_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------------------------
 * Append. Row t of k and v goes to slot slots[t] (page * page_size + slot in page) of both pools.
 * For each block of slots that new rows fall into, each kv head, and keys and values apart:
 *   need  = the smallest power of two with  max |x| of the block's new rows <= 448 * need,
 *           at least 2^-40
 *   scale = need where the first new row takes the block's first slot, else max(need, the block's
 *           scale so far)
 *   code  = x / scale, rounded to nearest even, for the new rows
 * and where the scale rises the codes of the block's slots below its first new one are rounded
 * again: code * old / new (exact but for codes that become subnormal). Slots past the first new one that
 * take no row are left as they are, and count for nothing: what they held is under the new scale.
 * Powers of two cost a code nothing but where it becomes subnormal, and they make a cache filled token
 * by token equal, but for those, to one filled at once.
 *
 * Arguments
 *   shape      dtype (of k and v), Hkv, D, page_size, num_pages; B = 1, and P, Hq and max_pages 1
 *              (not used).
 *   rows       0 <= T <= 2^30 (0 is a no-op).
 *   k, v       [T, Hkv, D]; element strides row and head (multiples of 8), D contiguous, 16-byte
 *              aligned.
 *   slots      [T] int64. A row whose slot is negative or past the pools is left out. Rows of one
 *              block stand side by side in ascending order of slots, and no other rows of the call
 *              fall into that block: a request's new positions in order. Where a block's rows stand
 *              side by side but not in ascending order, the scales of the block become NaN. Where
 *              they do not stand side by side (a page shared by two requests that both append to
 *              it), what the block holds is one of the ways of writing them at once; nothing
 *              outside the block is touched.
 *   k_pool, v_pool, k_scale, v_scale, block   as above; written in place. The two pools share no
 *              element and the two scales none; what starts at the same address, scales that share
 *              bytes and strides below D (of a dimension of two or more) are SV_ERR_INVALID_ARG.
 * A row's element that is infinite, NaN or above 448 * 2^40 becomes the NaN code and does not count
 * for the scale. A block whose earlier slots have a scale that is negative, above 2^40 or NaN keeps
 * NaN. No workspace.
 * ---------------------------------------------------------------------------------------- */
sv_status kv_cache_append_q8(const sv_kv_shape* shape, int rows, const void* k, int64_t k_row,
                             int64_t k_head, const void* v, int64_t v_row, int64_t v_head,
                             const int64_t* slots, const sv_kv_pool* k_pool,
                             const sv_kv_pool* v_pool, float* k_scale, float* v_scale, int block,
                             sv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * Attention over the cache. As paged_attention of specverify_kv.h, over keys and values code *
 * scale: the same rows, rule, page table, lengths, outputs, errors and guarantees, but:
 *   k, v         pools of codes, with k_scale, v_scale and block as above.
 *   G            at most 64, and at most 32 where D is 256, else SV_ERR_UNSUPPORTED.
 *   values       a NaN code makes the component NaN in the rows that see it.
 *   scales       a value scale that is negative, above 2^40 or NaN, or a key scale that is not
 *                finite, makes the rows that see the block NaN. (Value scales below 2^-40 count as
 *                they are, but lose digits beside others.)
 *   queries      a row that is not finite gets NaN. An element below 2^-6 of its row's largest may
 *                be off by 2^-17 of that.
 * Scores, their softmax and the sums are fp32. The weights exp(s_j - max) * scale enter the product
 * with the codes rounded to fp16, to nearest: off by 2^-11 of a weight and 2^-27 of the row's largest.
 * Equal calls give equal bits. The cache is read once for as many whole positions as 64 query rows per kv
 * head hold (32 where D is 256): ceil(P / floor(64 / G)) times, P times from G = 33 (17) on.
 * ---------------------------------------------------------------------------------------- */
size_t paged_attention_q8_workspace(const sv_kv_shape* shape);

sv_status paged_attention_q8(const sv_kv_shape* shape, const sv_score_rule* rule, const void* q,
                             int64_t q_req, int64_t q_row, int64_t q_head, const sv_kv_pool* k,
                             const sv_kv_pool* v, const float* k_scale, const float* v_scale,
                             int block, const int32_t* page_table, const int32_t* seq_len,
                             const int32_t* num_draft, void* out, float* out_lse, void* workspace,
                             size_t workspace_bytes, sv_stream_t stream);

/* The self-test of its bounded waits, as paged_attention_wait_selftest. */
sv_status paged_attention_q8_wait_selftest(
    const sv_kv_shape* shape, const sv_score_rule* rule, const void* q, int64_t q_req,
    int64_t q_row, int64_t q_head, const sv_kv_pool* k, const sv_kv_pool* v, const float* k_scale,
    const float* v_scale, int block, const int32_t* page_table, const int32_t* seq_len,
    const int32_t* num_draft, void* out, float* out_lse, void* workspace, size_t workspace_bytes,
    unsigned int wait_us, sv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_KV8_H_ */
