/*
 * pkv_softmax.h - what stands around the packed causal attention of
 * pkv_mixers.h in a softmax layer, for training and for serving (C ABI of
 * libpkv, AMD Instinct MI355X).
 *
 *   pkv_qk_norm_rope, pkv_qk_norm_rope_backward
 *       RMS norm of every query and key head and the rotation by position,
 *       one pass (RFC-0026 section 3.6: positions restart at every document;
 *       pkv_eod_to_segment_ids gives them)
 *   pkv_attn_window_varlen, pkv_attn_window_varlen_backward
 *       pkv_attn_varlen through a sliding window, with a few first tokens of
 *       each segment that stay visible (sinks)
 *   pkv_paged_kv_append, pkv_attn_paged
 *       for serving: new tokens' keys and values into a paged cache, and
 *       attention of the new tokens (one of each request, or chunks of
 *       prompts) over it
 *
 * The conventions of pkv.h and pkv_mixers.h hold: device pointers, the caller
 * owns every buffer, nothing is allocated or kept between calls, nothing
 * synchronizes, host-visible errors are returned before any launch and
 * data-dependent ones go to the device `flags` word. Tensors in `dtype` are
 * 16-byte aligned; fp32 and int32 ones are aligned to their element size. No
 * output overlaps an input or another output (but see pkv_paged_kv_append).
 * Equal calls give equal bits; the order of a sum may go by the call's sizes,
 * over a paged cache also by the lengths of the call's requests.
 * Workspaces are scratch: calls that share one must be ordered on one stream.
 * What a call reads, lengths and tables among it, must not change while it runs.
 */
#ifndef PKV_SOFTMAX_H
#define PKV_SOFTMAX_H

#include "pkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bits of the device flags word: a page that a request needs is not in
   [0, num_pages); a length of kv_lens is negative or more than its row of the
   page table holds. */
#define PKV_FLAG_BAD_PAGE 32
#define PKV_FLAG_BAD_LENGTH 64

/* Bit of pkv_qk_norm_rope's `options`: channels 2 i and 2 i + 1 make a rotated
   pair, instead of i and i + rot_dim / 2. */
#define PKV_OPT_ROPE_INTERLEAVED 2

/*
 * Per token n with position p = positions[n], and per head of q and of k:
 *   u_d = w_d x_d / sqrt(mean_d x_d^2 + eps)
 *   (y_a, y_b) = (u_a cos t - u_b sin t, u_a sin t + u_b cos t),
 *   t = p * inv_freq[i], for pair i < rot_dim / 2; other channels: y = u.
 * The angle is reduced in fp64, so far positions lose nothing; norm and
 * rotation are fp32 with one rounding to `dtype`.
 *
 * q, k       [N, Hq, D], [N, Hkv, D] in `dtype`, heads dense, consecutive
 *            tokens q_stride / k_stride elements apart (views of one
 *            projection's result): at least the heads' size, multiples of 16
 *            bytes, N of them at most 2^46 bytes. k's tokens may lie between
 *            q's.
 * q_weight, k_weight  float32 [D] or NULL (1).
 * positions  int32 [N] or NULL (0 .. N - 1). A negative one marks a row to
 *            leave out (padding): its outputs and gradients are 0, and its
 *            values reach nothing.
 * inv_freq   float32 [rot_dim / 2]; NULL with rot_dim 0.
 * q_out, k_out  dense [N, Hq, D], [N, Hkv, D].
 * options    0 or PKV_OPT_ROPE_INTERLEAVED.
 * Supported: D in {32, 64, 128}, rot_dim a multiple of 16 in [0, D]. Errors:
 * PKV_ERR_INVALID_ARGUMENT for a NULL tensor, N < 1, N > 2^25, heads < 1
 * or > 65536, a bad stride, eps < 0 or not finite, a misaligned or overlapping
 * tensor; PKV_ERR_UNSUPPORTED for another D, rot_dim, dtype or option.
 */
pkv_status pkv_qk_norm_rope(const void* q, const void* k, int64_t q_stride, int64_t k_stride,
                            const float* q_weight, const float* k_weight, const int32_t* positions,
                            const float* inv_freq, int64_t N, int32_t Hq, int32_t Hkv, int32_t D,
                            int32_t rot_dim, float eps, int32_t dtype, int32_t options, void* q_out,
                            void* k_out, void* stream);

/*
 * Reverse pass on the same inputs: dq_out, dk_out (dense, in `dtype`) are the
 * gradients of q_out and k_out. With r = 1 / sqrt(mean x^2 + eps) and du the
 * rotation's transpose applied to dy:
 *   dx = r (w du - r x mean(w du r x)),  dw = sum over rows of du r x
 * dq, dk     dense [N, Hq, D], [N, Hkv, D].
 * dq_weight, dk_weight  float32 [D] or NULL (not written).
 * workspace  at least pkv_qk_norm_rope_backward_workspace_size() bytes,
 *            256-byte aligned; not needed (NULL) without the weights'
 *            gradients.
 * Errors: as pkv_qk_norm_rope; PKV_ERR_WORKSPACE.
 */
size_t pkv_qk_norm_rope_backward_workspace_size(int64_t N, int32_t Hq, int32_t Hkv, int32_t D,
                                                int32_t dtype);
pkv_status pkv_qk_norm_rope_backward(const void* q, const void* k, int64_t q_stride, int64_t k_stride,
                                     const void* dq_out, const void* dk_out, const float* q_weight,
                                     const float* k_weight, const int32_t* positions,
                                     const float* inv_freq, int64_t N, int32_t Hq, int32_t Hkv,
                                     int32_t D, int32_t rot_dim, float eps, int32_t dtype,
                                     int32_t options, void* dq, void* dk, float* dq_weight,
                                     float* dk_weight, void* workspace, size_t workspace_bytes,
                                     void* stream);

/*
 * pkv_attn_varlen in which token t of a segment [a, e) attends to s <= t only
 * if t - s < window or s - a < sinks. Everything else is as for
 * pkv_attn_varlen: layouts, lse, flags, what is rounded; a row's values go by
 * the keys and values that it sees alone (NaN and infinities in others leave
 * its bits as they are).
 * Errors: as pkv_attn_varlen; PKV_ERR_INVALID_ARGUMENT for window < 1 or
 * sinks < 0; PKV_ERR_UNSUPPORTED for sinks > 64.
 */
pkv_status pkv_attn_window_varlen(const void* q, const void* k, const void* v,
                                  const int32_t* cu_seqlens, int32_t max_segs, int64_t N, int32_t Hq,
                                  int32_t Hkv, int32_t D, float scale, int32_t dtype, int32_t window,
                                  int32_t sinks, void* o, float* lse, int32_t* flags, void* stream);

/*
 * Reverse pass, as pkv_attn_varlen_backward with the window's pairs. The
 * workspace also holds partial sums of the sinks' gradients: 8 sinks D Hkv
 * bytes for every chunk of 128 to 512 tokens (of `window` tokens if that is
 * less; windows below 64: for every chunk and every segment slot).
 */
size_t pkv_attn_window_varlen_backward_workspace_size(int64_t N, int32_t Hq, int32_t Hkv, int32_t D,
                                                      int32_t max_segs, int32_t dtype, int32_t window,
                                                      int32_t sinks);
pkv_status pkv_attn_window_varlen_backward(const void* q, const void* k, const void* v, const void* o,
                                           const float* lse, const void* dout,
                                           const int32_t* cu_seqlens, int32_t max_segs, int64_t N,
                                           int32_t Hq, int32_t Hkv, int32_t D, float scale,
                                           int32_t dtype, int32_t window, int32_t sinks, void* dq,
                                           void* dk, void* dv, int32_t* flags, void* workspace,
                                           size_t workspace_bytes, void* stream);

/*
 * The paged cache: k_pages and v_pages are [num_pages, page_size, Hkv, D] in
 * `dtype`. Token i of request r lies at
 *   page page_table[r, i / page_size], place i % page_size.
 * page_table  int32 [R, max_pages]; entries that no token needs may hold
 *             anything.
 * kv_lens     int32 [R]: tokens of each request, its new ones included. 0
 *             with new tokens is an idle row of a batch.
 * cu_seqlens  int32 [R + 1]: request r's new tokens are [cu[r], cu[r + 1]) of
 *             the N packed ones; they are its last tokens. NULL: one new
 *             token for each request, N = R.
 * page_size   a multiple of 16, at most 65536; num_pages * page_size at
 *             most 2^30, max_pages * page_size at most 2^29.
 *
 * pkv_paged_kv_append writes the new tokens' k and v [N, Hkv, D] (dense, or
 * with k_stride / v_stride elements from token to token as for
 * pkv_qk_norm_rope) to their places; all else in the pages keeps its bits. New
 * tokens before the request's first place (more new ones than kv_lens) and
 * those of a bad length or page are left out; the bad ones set their flag. Two
 * requests may share pages that no new token goes to; where two new tokens of
 * a call have one place, either's values may be there.
 * Supported: D in {32, 64, 128}. Errors: PKV_ERR_INVALID_ARGUMENT for a NULL
 * tensor, sizes out of range, R < 1, N < 1, (N / 16 + R) heads >= 2^23, N != R
 * without cu_seqlens, a misaligned or overlapping tensor; PKV_ERR_UNSUPPORTED for another D, dtype
 * or page_size.
 */
pkv_status pkv_paged_kv_append(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                               const int32_t* page_table, const int32_t* kv_lens,
                               const int32_t* cu_seqlens, int64_t N, int32_t R, int32_t Hkv, int32_t D,
                               int32_t page_size, int32_t num_pages, int32_t max_pages, int32_t dtype,
                               void* k_pages, void* v_pages, int32_t* flags, void* stream);

/*
 * Attention of the new tokens (whose keys and values are in the pages already)
 * over their request's tokens: the new token at place t attends to the places
 * s <= t, and with window > 0 only if t - s < window or s < sinks.
 *
 * q, o   [N, Hq, D] in `dtype`; query head h reads kv head h / (Hq / Hkv).
 * lse    float32 [Hq, N] or NULL (not written).
 * window 0 (no window; sinks, 0 or more, are ignored) or more.
 * A row that sees nothing (an idle request, a place before the first) and the
 * rows behind cu_seqlens[R] get o = 0, lse = -inf. A bad length or a malformed
 * cu_seqlens sets its flag and leaves its requests' rows undefined; so does a
 * bad page. What pages hold outside a request's tokens reaches nothing, nor
 * does a token reach a row that does not see it (NaN, infinities). Scores,
 * statistics and sums are fp32; with bf16 and D in {64, 128} the weights are
 * rounded to bf16 for the product with v.
 * workspace  at least pkv_attn_paged_workspace_size() bytes, 256-byte aligned
 *            (NULL where that is 0): in bf16 85 MB at D 128 and 43 at D 64 if
 *            a request can have more than 32 rows (N Hq / Hkv > 32), 17 and 9
 *            if not, else at most 5 MB. Without cu_seqlens a request has one
 *            token: those bf16 calls need what the function says for
 *            N = R = 1.
 * Errors: as pkv_paged_kv_append; Hq not a multiple of Hkv, a scale that is
 * not finite, window < 0, sinks < 0 (PKV_ERR_INVALID_ARGUMENT); with a window
 * sinks > 64 (PKV_ERR_UNSUPPORTED); PKV_ERR_WORKSPACE.
 */
size_t pkv_attn_paged_workspace_size(int64_t N, int32_t R, int32_t Hq, int32_t Hkv, int32_t D,
                                     int32_t dtype);
pkv_status pkv_attn_paged(const void* q, const void* k_pages, const void* v_pages,
                          const int32_t* page_table, const int32_t* kv_lens,
                          const int32_t* cu_seqlens, int64_t N, int32_t R, int32_t Hq, int32_t Hkv,
                          int32_t D, int32_t page_size, int32_t num_pages, int32_t max_pages,
                          float scale, int32_t dtype, int32_t window, int32_t sinks, void* o, float* lse,
                          int32_t* flags, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_SOFTMAX_H */
