/*
 * pkv_mixers.h - the packed token mixers that stand next to KDA in a model, and
 * the recurrences' single-token steps (C ABI of libpkv, AMD Instinct MI355X).
 *
 *   pkv_attn_varlen, pkv_attn_varlen_backward
 *       causal softmax attention with grouped heads over packed segments
 *       ("Drill: Sequence Packing from scratch", The math: a token attends to
 *       the earlier tokens of its own document)
 *   pkv_linear_attn_varlen, pkv_linear_attn_varlen_backward
 *       S_t = e^{g_h} S_{t-1} + k_t v_t^T, o_t = scale * S_t^T q_t: linear
 *       attention with one decay per head, S reset per segment
 *   pkv_linear_attn_step, pkv_kda_step
 *       one token of each of R requests on per-slot states (the final states
 *       of the packed calls), for decoding
 *
 * The conventions of pkv.h hold: device pointers, dense row-major layouts, the
 * caller owns every buffer, nothing is allocated or kept between calls,
 * nothing synchronizes, host-visible errors are returned before any launch and
 * data-dependent ones go to the device `flags` word. q, k, v, o, their
 * gradients and the fp32 states are 16-byte aligned; lse, beta, g and slots
 * are aligned to their element size. No output overlaps an input or another
 * output.
 *
 * Packed calls take cu_seqlens int32 [max_segs + 1] (cu[0] = 0, non-decreasing,
 * cu[max_segs] <= N; empty slots are allowed) or NULL: one segment [0, N).
 * Outputs of positions p >= cu[max_segs] are zero (lse: -inf). A malformed
 * cu_seqlens sets PKV_FLAG_BAD_CU_SEQLENS and leaves the outputs undefined;
 * nothing outside the tensors is read or written. No result of a segment
 * depends on the values of another segment, NaN and infinities included, and
 * equal calls give equal bits. The order of a sum may go by the call's sizes
 * (N, max_segs, heads), so the same segment in another call may differ in its
 * last bits.
 */
#ifndef PKV_MIXERS_H
#define PKV_MIXERS_H

#include "pkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bit of the device flags word: a step's row named a slot that does not exist
   or that an earlier row of the call names too. */
#define PKV_FLAG_BAD_SLOT 16

/*
 * Packed causal softmax attention with grouped heads.
 *
 *   o_t = sum_{s <= t, same segment} softmax_s(scale q_t.k_s) v_s
 *   lse_t = ln sum_{s <= t, same segment} exp(scale q_t.k_s)
 * Query head h reads kv head h / (Hq / Hkv).
 *
 * q, o   [1, N, Hq, D]; k, v [1, N, Hkv, D], in `dtype`.
 * lse    float32 [Hq, N] or NULL (not written); the reverse pass needs it.
 * flags  int32 [1] or NULL; PKV_FLAG_BAD_CU_SEQLENS is OR-ed in.
 * Scores, softmax statistics and sums are fp32; with bf16 and D in {64, 128}
 * the weights are rounded to bf16 for the product with v. A row goes by the
 * tokens up to its own alone: NaN, infinities and large values in later ones
 * leave its bits as they are.
 * Supported: D in {32, 64, 128}. Errors: PKV_ERR_INVALID_ARGUMENT for a NULL
 * tensor, N < 1, N > INT32_MAX, Hq or Hkv < 1 or > 65536, Hq not a multiple of
 * Hkv, max_segs < 1 (with cu_seqlens), (N / 32 + max_segs) Hq >= 2^23, a
 * misaligned or overlapping tensor, a scale that is not finite;
 * PKV_ERR_UNSUPPORTED for another D or dtype.
 */
pkv_status pkv_attn_varlen(const void* q, const void* k, const void* v, const int32_t* cu_seqlens,
                           int32_t max_segs, int64_t N, int32_t Hq, int32_t Hkv, int32_t D,
                           float scale, int32_t dtype, void* o, float* lse, int32_t* flags,
                           void* stream);

/*
 * Reverse pass of pkv_attn_varlen on the same inputs, with its o and lse and
 * dout = dL/do. With P_ts = exp(scale q_t.k_s - lse_t):
 *   delta_t = do_t.o_t,  dS_ts = P_ts (do_t.v_s - delta_t)
 *   dq_t = scale sum_s dS_ts k_s
 *   dk_s = scale sum_t dS_ts q_t,  dv_s = sum_t P_ts do_t,
 * dk and dv summed over the query heads of their kv head, in an order that the
 * sizes and the segments' lengths fix. Sums, delta and dS are fp32; with bf16 and
 * D in {64, 128} P and dS are rounded to bf16 for their products (dv; dq, dk).
 * A segment with NaN or infinities may have them anywhere in its gradients.
 * workspace  at least pkv_attn_varlen_backward_workspace_size() bytes, 256-byte
 *            aligned; scratch.
 * Errors: as pkv_attn_varlen; PKV_ERR_WORKSPACE for a missing, small,
 * misaligned or overlapping workspace.
 */
size_t pkv_attn_varlen_backward_workspace_size(int64_t N, int32_t Hq, int32_t Hkv, int32_t D,
                                               int32_t max_segs, int32_t dtype);
pkv_status pkv_attn_varlen_backward(const void* q, const void* k, const void* v, const void* o,
                                    const float* lse, const void* dout, const int32_t* cu_seqlens,
                                    int32_t max_segs, int64_t N, int32_t Hq, int32_t Hkv, int32_t D,
                                    float scale, int32_t dtype, void* dq, void* dk, void* dv,
                                    int32_t* flags, void* workspace, size_t workspace_bytes,
                                    void* stream);

/*
 * Packed linear attention with one decay per head.
 *
 * For every segment i and head h, from S = initial_state[i, h] (0 when NULL):
 *   S_t = e^{g[h]} S_{t-1} + k_t v_t^T,  o_t = scale * S_t^T q_t
 * final_state[i, h] = S after the last token (the initial state, or 0, for an
 * empty slot).
 *
 * q, k   [1, N, H, Dk]; v, o [1, N, H, Dv], in `dtype`.
 * g      float32 [H]: log decays (<= 0; -inf keeps nothing). A constant of the layer: the reverse
 *        pass has no gradient for it. Above 0 the state grows; up to
 *        64 g = 80 ln 2 the weights inside a chunk stay finite.
 * initial_state, final_state  float32 [max_segs, H, Dk, Dv] or NULL.
 * workspace  at least pkv_linear_attn_varlen_workspace_size() bytes, 256-byte
 *        aligned (NULL where that is 0); scratch: calls that share it must be
 *        ordered on one stream.
 * With bf16 and Dk, Dv in {64, 128} the call works in chunks of 32 tokens:
 * states and sums are fp32, the in-chunk weights and, for the readout, the
 * state are rounded to bf16; NaN and infinities reach no other segment, but
 * may reach earlier tokens of their own chunk, and an infinity may become NaN.
 * Decay weights below 2^-126 are 0.
 * Asking for the states or not changes no bit of the other results.
 * Supported: Dk, Dv in {32, 64, 128}. Errors: as pkv_attn_varlen with H in
 * place of the heads, max_segs * H > 2^22; PKV_ERR_WORKSPACE.
 */
size_t pkv_linear_attn_varlen_workspace_size(int64_t N, int32_t H, int32_t Dk, int32_t Dv,
                                             int32_t max_segs, int32_t dtype);
pkv_status pkv_linear_attn_varlen(const void* q, const void* k, const void* v, const float* g,
                                  const int32_t* cu_seqlens, int32_t max_segs, int64_t N, int32_t H,
                                  int32_t Dk, int32_t Dv, float scale, int32_t dtype,
                                  const float* initial_state, void* o, float* final_state,
                                  int32_t* flags, void* workspace, size_t workspace_bytes,
                                  void* stream);

/*
 * Reverse pass of pkv_linear_attn_varlen on the same inputs, with dout = dL/do
 * and (optionally) dfinal_state = dL/dfinal_state. Per segment and head:
 *   dS (after the last token) = dfinal_state (0 when NULL)
 *   dS_t = [dS_t+1 e^{g}, or the line above] + scale * q_t do_t^T
 *   dq_t = scale * S_t do_t,  dk_t = dS_t v_t,  dv_t = dS_t^T k_t
 *   d_initial_state = e^{g} dS_first (dfinal_state for an empty slot)
 * d_initial_state  float32 [max_segs, H, Dk, Dv] or NULL (not written).
 * Roundings as in the forward call, the adjoint state dS like the state.
 */
size_t pkv_linear_attn_varlen_backward_workspace_size(int64_t N, int32_t H, int32_t Dk, int32_t Dv,
                                                      int32_t max_segs, int32_t dtype);
pkv_status pkv_linear_attn_varlen_backward(const void* q, const void* k, const void* v,
                                           const float* g, const int32_t* cu_seqlens,
                                           int32_t max_segs, int64_t N, int32_t H, int32_t Dk,
                                           int32_t Dv, float scale, int32_t dtype,
                                           const float* initial_state, const void* dout,
                                           const float* dfinal_state, void* dq, void* dk, void* dv,
                                           float* d_initial_state, int32_t* flags, void* workspace,
                                           size_t workspace_bytes, void* stream);

/*
 * One token of each of R requests; request r's state is
 * state[slots[r]] (state[r] when slots is NULL, and then R <= S), updated in
 * place:
 *   pkv_linear_attn_step   S = e^{g[h]} S + k v^T
 *   pkv_kda_step           S = diag(e^{g}) S + beta k v^T (pkv.h's recurrence)
 *   o = scale * S^T q
 *
 * q, k   [R, H, Dk]; v, o [R, H, Dv], in `dtype`.
 * g      linear: float32 [H]; KDA: [R, H, Dk] in `dtype`. beta [R, H].
 * slots  int32 [R] or NULL. A negative slot is an idle row: o = 0 and no state
 *        is touched. A slot >= S, or one that an earlier row of the call
 *        names, is treated the same and sets PKV_FLAG_BAD_SLOT.
 * state  float32 [S, H, Dk, Dv]; all arithmetic is fp32.
 * options  0 or PKV_OPT_QK_L2NORM, as for pkv_chunk_kda_varlen.
 * Supported: Dk, Dv in {32, 64, 128}, R <= 2^20, H <= 65535. Errors:
 * PKV_ERR_INVALID_ARGUMENT for a NULL tensor, sizes out of range, R > S
 * without slots, a misaligned or overlapping tensor; PKV_ERR_UNSUPPORTED for
 * other head dimensions, dtypes or options.
 */
pkv_status pkv_linear_attn_step(const void* q, const void* k, const void* v, const float* g,
                                const int32_t* slots, int64_t R, int32_t S, int32_t H, int32_t Dk,
                                int32_t Dv, float scale, int32_t dtype, float* state, void* o,
                                int32_t* flags, void* stream);
pkv_status pkv_kda_step(const void* q, const void* k, const void* v, const void* g, const void* beta,
                        const int32_t* slots, int64_t R, int32_t S, int32_t H, int32_t Dk,
                        int32_t Dv, float scale, int32_t dtype, int32_t options, float* state,
                        void* o, int32_t* flags, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_MIXERS_H */
