/*
 * specverify_logits.h — C ABI of the logits' adjustment ahead of a verify, on GB300.
 *
 *   logit_adjust   penalties for repeated tokens, per-token biases and an allowed-token mask
 *                  (a grammar's) over the logit rows of P = k+1 positions per request, each
 *                  position counting the drafted tokens ahead of it.
 *
 * The conventions of specverify.h hold.
 */
#ifndef SPECVERIFY_LOGITS_H_
#define SPECVERIFY_LOGITS_H_

#include "specverify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------------------------
 * Adjust the logits of request r at position i (0 <= i <= n_r, n_r = num_draft[r]): with
 * the tokens h = history[r, 0 .. hist_len[r]) and x = draft_tokens[r, 0 .. i) ahead of it,
 *   seen(v) = v occurs in h or x
 *   c(v)    = occurrences of v in history[r, prompt_len[r] .. hist_len[r]) plus those in x
 *   y(v)    = z(v) > 0 ? z(v) / rho_r : z(v) * rho_r     where seen(v), else z(v)
 *   y(v)   -= f_r * c(v) + pi_r * [c(v) > 0]
 *   y(v)   += the bias listed for v
 *   y(v)    = -inf                                       where v is not allowed at (r, i)
 * in fp32, rounded once to the output's type. z * (1 / rho) stands for z / rho (one more
 * fp32 rounding). A masked logit is -inf whatever it held (NaN included); a row whose mask
 * allows nothing comes out all -inf, which the verify calls report as a data error.
 *
 * Arguments
 *   logits         [B, P, V] dtype (SV_F32 or SV_BF16), each row contiguous; rows lie
 *                  in_row_stride and requests in_req_stride elements apart. Rows past n_r of a
 *                  request are not read.
 *   history        [B, L_max] int32, or NULL (then hist_len and prompt_len are NULL and
 *                  L_max is 0). Tokens outside [0, V) count for nothing (padding).
 *                  L_max < 2^30, else SV_ERR_UNSUPPORTED.
 *   hist_len       [B] int32, in [0, L_max].
 *   prompt_len     [B] int32, in [0, hist_len[r]], or NULL for no prompt.
 *   draft_tokens   [B, P-1] int32, or NULL: no drafts count. Tokens outside [0, V) count for
 *                  nothing.
 *   num_draft      [B] int32 in [0, P-1], or NULL for all P-1.
 *   repetition, presence, frequency   [B] fp32 rho, pi and f, each NULL for 1, 0 and 0. rho
 *                  is meant to be positive; other values go through the formula as they are.
 *   bias_tokens    [B, n_bias] int32, bias_values [B, n_bias] fp32, or both NULL with
 *                  n_bias = 0. Tokens outside [0, V) are padding; of a token listed more
 *                  than once the first entry counts.
 *   allowed        [B, P, ceil(V/32)] uint32, bit v % 32 of word v / 32 set where token v is
 *                  allowed, or NULL for all.
 *   B, P, V        B >= 0 (0 is a no-op), 1 <= P <= SV_MAX_K + 1, V >= 1.
 *   out            [B, P, V] dtype, with its own strides; `out` may be `logits` with the
 *                  same strides, and must not overlap it otherwise. Rows past n_r are not
 *                  written.
 * A request with hist_len, prompt_len or num_draft out of range gets NaN in all its P rows.
 * Any alignment of the rows works. Rows move in 16-byte pieces where logits and out, their strides
 * and V are all multiples of 16 bytes (4 fp32 or 8 bf16 elements); else element by element, which is
 * slower. No workspace; one launch.
 * ---------------------------------------------------------------------------------------- */
sv_status logit_adjust(const void* logits, int64_t in_req_stride, int64_t in_row_stride,
                       sv_dtype dtype, const int32_t* history, const int32_t* hist_len,
                       const int32_t* prompt_len, int L_max, const int32_t* draft_tokens,
                       const int32_t* num_draft, const float* repetition,
                       const float* presence, const float* frequency,
                       const int32_t* bias_tokens, const float* bias_values, int n_bias,
                       const uint32_t* allowed, int B, int P, int V, void* out,
                       int64_t out_req_stride, int64_t out_row_stride, sv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * Self-test of the bounded waits inside logit_adjust: the same call, except that each wait for a
 * copy is limited to wait_us microseconds (1000 .. 100000: the copies have landed by then) instead of
 * 2 s and that those for the third row of a request cannot be over. Where rows move in 16-byte pieces,
 * rows 0 and 1 come out as ever and the others are NaN, with no fault and no hang; other calls are as
 * logit_adjust's. Returns SV_ERR_INVALID_ARG for wait_us out of range, else what the call returns.
 * ---------------------------------------------------------------------------------------- */
sv_status logit_adjust_wait_selftest(
    const void* logits, int64_t in_req_stride, int64_t in_row_stride, sv_dtype dtype,
    const int32_t* history, const int32_t* hist_len, const int32_t* prompt_len,
    int L_max, const int32_t* draft_tokens, const int32_t* num_draft,
    const float* repetition, const float* presence, const float* frequency,
    const int32_t* bias_tokens, const float* bias_values, int n_bias,
    const uint32_t* allowed, int B, int P, int V, void* out,
    int64_t out_req_stride, int64_t out_row_stride, unsigned int wait_us,
    sv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPECVERIFY_LOGITS_H_ */
