/*
 * specverify_step.h — C ABI of what a step does around the cache before its attention, on GB300.
 *
 *   kv_page_map      the pages and slots of the new positions, from the requests' lengths.
 *   qk_norm_rotate   the norm of each query and key head and the rotation by its position.
 *
 * The conventions of specverify.h hold.
 */
#ifndef SPECVERIFY_STEP_H_
#define SPECVERIFY_STEP_H_

#include "specverify_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------------------------
 * Page tables and slots. Request r holds the pages of old_len[r] tokens: have = ceil(old_len /
 * page_size) entries of its row of page_table. After the step it has n = seq_len[r] tokens, the last
 * num_new[r] of them new (0 tokens: it has ended), so it needs need = ceil(n / page_size) pages.
 * (After a verify, old_len is the last step's seq_len, rejected drafts included, and seq_len what was
 * kept and the new positions: the pages of rejected drafts are reused or go back.)
 *
 * Free pages wait in a ring of ring_size places: `count` of them from place `head` on.
 *   need > have   takes need - have pages from the ring's front, in the order of the requests, if
 *                 the growth of requests 0 .. r adds up to at most count; entries have .. need-1.
 *   need < have   its entries need .. have-1 go to the ring's end, in the order of the requests
 *                 (they are free from the next call on; the table keeps the stale entries).
 * A request that is left without pages keeps what it holds: out_len = old_len, its slots -1.
 * A page has one owner: one that stands in two rows (a common prefix) goes back with each of them, and is
 * then given out twice. Rows that share pages are the caller's to keep apart.
 * Row i of request r is its token at position p = n - num_new + i, in slot
 *   page_table[r][p / page_size] * page_size + p % page_size
 * or -1 where that page is outside [0, num_pages).
 *
 * Arguments
 *   B            requests, 0 <= B <= 8192, else SV_ERR_UNSUPPORTED. With none the ring is kept:
 *                out_state is ring_state (or {-1, -1}, as below), out_first[0] 0, all rows -1, and
 *                the requests' arrays may be NULL. (With none and an out_state that is no memory of
 *                CUDA's, as NULL, the call is a no-op.)
 *   page_size    a power of two from 8 to 1024. num_pages >= 0.
 *   page_table   [B, max_pages] int32, updated in place; max_pages * page_size < 2^30.
 *   old_len, seq_len   [B] int32 in [0, max_pages * page_size].
 *   num_new      [B] int32 in [0, seq_len], and in [0, P] where P > 0.
 *   ring         [ring_size] int32, updated in place; ring_size >= 1.
 *   ring_state   [2] int32: head in [0, ring_size), count in [0, ring_size].
 *   P            row layout: P > 0 for P rows per request (row r * P + i), 0 for packed rows
 *                (request r's from out_first[r] on).
 *   rows         rows of slots and positions: B * P, or any number for packed ones.
 *   out_slots    [rows] int64, out_positions [rows] int32: -1 in rows of no new token.
 *   out_len      [B] int32: seq_len, old_len (no pages), or -1 for a request with a length out of
 *                range, or whose packed rows pass `rows`: nothing of it is changed.
 *   out_first    [B + 1] int32: the requests' first rows, and the number of rows used.
 *   out_state    [2] int32: the ring's state after the call.
 * No output, nor page_table or ring, may overlap another of these or an input, else
 * SV_ERR_INVALID_ARG. A ring whose state is out of range, or that has no room for its pages and
 * those given back (a ring of as many places as there are pages always has), is a data error of the
 * call: out_len and rows are all -1, out_state is {-1, -1}, and nothing is changed. No workspace.
 * Called again with the same inputs, a call does the same again.
 * ---------------------------------------------------------------------------------------- */
sv_status kv_page_map(int B, int page_size, int num_pages, int32_t* page_table, int max_pages,
                      const int32_t* old_len, const int32_t* seq_len, const int32_t* num_new,
                      int32_t* ring, int ring_size, const int32_t* ring_state, int P, int rows,
                      int64_t* out_slots, int32_t* out_positions, int32_t* out_len,
                      int32_t* out_first, int32_t* out_state, sv_stream_t stream);

/* Queries or keys of qk_norm_rotate: element d of head h of row (r, i) is at
 * data[r * req + i * row + h * head + d] (strides in elements, multiples of 8; data 16-byte
 * aligned). `out` likewise; it may be `data` with the same strides, and has no other element of the
 * call's inputs or outputs in it: data at other strides, an out that starts where the other rows' out
 * or data does, and out strides below D (of a dimension of two or more) are SV_ERR_INVALID_ARG.
 * HOST memory. */
typedef struct {
  const void* data;
  int64_t req, row, head;
  void* out;
  int64_t out_req, out_row, out_head;
  int heads;
  const void* weight; /* DEVICE [D], or NULL for ones */
} sv_head_rows;

/* ------------------------------------------------------------------------------------------
 * For each row at a position p >= 0, and each head x of its queries and keys:
 *   y = x / sqrt(mean(x^2) + eps) * weight                 (norm = 0: y = x * weight)
 *   (a, b) = (y_i, y_{i + R/2}), or (y_2i, y_{2i+1}) where interleaved, for 0 <= i < R/2:
 *   out    = (a cos t - b sin t, a sin t + b cos t),  t = p * inv_freq[i]
 * and y in the components from R on. Angles are reduced in 64 bits, the rest is fp32, rounded once.
 *
 * Arguments
 *   dtype        of q, k and their outputs.
 *   B, P         rows are [B, P], B * P < 2^31 (0 is a no-op).
 *   D            64, 128 or 256; R a multiple of 16 in [0, D], else SV_ERR_UNSUPPORTED.
 *   q, k         as above; heads >= 0 (0: none of them).
 *   weight_f32   whether the weights are fp32, else of dtype.
 *   positions    [B, P] int32; rows at a negative position are left as they are.
 *   inv_freq     [R / 2], fp32, or fp64 where freq_f64.
 *   eps          >= 0. A head's squares are summed in fp32; bf16 heads that pass its range there are
 *                scaled by a power of two first.
 * No workspace.
 * ---------------------------------------------------------------------------------------- */
sv_status qk_norm_rotate(sv_kv_dtype dtype, int B, int P, int D, int R, const sv_head_rows* q,
                         const sv_head_rows* k, int weight_f32, const int32_t* positions,
                         const void* inv_freq, int freq_f64, int norm, float eps, int interleaved,
                         sv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_STEP_H_ */
