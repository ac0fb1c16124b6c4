// Argument validation and dispatch of the calls in include/pkv_softmax.h.

#include "pkv_softmax.h"

#include "api_check.h"
#include "common.h"

namespace {

using namespace pkv;

constexpr int32_t kMaxSinks = 64;
constexpr int64_t kMaxPlaces = int64_t(1) << 30;  // of a cache; of a request half of it

Span f32_span(const float* p, int64_t n) { return {p, n * 4, 4}; }
Span i32_span(const int32_t* p, int64_t n) { return {p, n * 4, 4}; }

pkv_status check_norm_rope(int64_t q_stride, int64_t k_stride, const float* inv_freq, int64_t N, int32_t Hq,
                           int32_t Hkv, int32_t D, int32_t rot, float eps, int32_t dtype, int32_t options) {
  // (four tokens a work-group at least)
  if (N < 1 || N > 4 * kMaxGroups || !heads_ok(Hq, Hkv) || !(eps >= 0.f) || !std::isfinite(eps))
    return PKV_ERR_INVALID_ARGUMENT;
  if (!known_dtype(dtype) || !supported_head_dim(D) || rot < 0 || rot > D || rot % 16 != 0 ||
      (options & ~PKV_OPT_ROPE_INTERLEAVED) != 0)
    return PKV_ERR_UNSUPPORTED;
  const int64_t es = elem_size(dtype);
  if (!stride_ok(N, q_stride, Hq, D, es) || !stride_ok(N, k_stride, Hkv, D, es) || (rot > 0 && inv_freq == nullptr))
    return PKV_ERR_INVALID_ARGUMENT;
  return PKV_OK;
}

pkv_status check_window(const int32_t* cu, int32_t& max_segs, int64_t N, int32_t Hq, int32_t Hkv, int32_t D,
                        float scale, int32_t dtype, int32_t window, int32_t sinks) {
  if (N < 1 || N > kInt32Max || !std::isfinite(scale)) return PKV_ERR_INVALID_ARGUMENT;
  if (cu == nullptr) max_segs = 1;
  if (max_segs < 1 || max_segs >= kInt32Max || !heads_ok(Hq, Hkv) || Hq % Hkv != 0 || window < 1 || sinks < 0)
    return PKV_ERR_INVALID_ARGUMENT;
  if (!known_dtype(dtype) || !supported_head_dim(D) || sinks > kMaxSinks) return PKV_ERR_UNSUPPORTED;
  if ((N / 32 + max_segs) * Hq >= kMaxGroups) return PKV_ERR_INVALID_ARGUMENT;
  return PKV_OK;
}

// Statistics and delta of every row, 256 bytes aligned, then the sinks' partial sums.
size_t stats_bytes(int64_t N, int32_t Hq) { return (size_t(N) * Hq * 8 + 16 + 255) / 256 * 256; }

pkv_status check_paged(const int32_t* cu, int64_t N, int32_t R, int32_t Hq, int32_t Hkv, int32_t D,
                       int32_t page_size, int32_t num_pages, int32_t max_pages, int32_t dtype) {
  if (N < 1 || N > kInt32Max || R < 1 || R >= kInt32Max || (cu == nullptr && N != R) || !heads_ok(Hq, Hkv) ||
      Hq % Hkv != 0 || num_pages < 1 || max_pages < 1)
    return PKV_ERR_INVALID_ARGUMENT;
  if (!known_dtype(dtype) || !supported_head_dim(D) || page_size < 16 || page_size > 65536 || page_size % 16 != 0)
    return PKV_ERR_UNSUPPORTED;
  if (int64_t(num_pages) * page_size > kMaxPlaces || int64_t(max_pages) * page_size > kMaxPlaces / 2 ||
      (N / 16 + R) * Hq >= kMaxGroups)
    return PKV_ERR_INVALID_ARGUMENT;
  return PKV_OK;
}

// chunks: with cu_seqlens.
size_t paged_workspace(int64_t N, int32_t R, int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype, bool chunks) {
  return attn_mfma_supported(D, dtype) ? attn_paged_workspace_bytes(N, Hq, Hkv, D, chunks)
                                       : attn_paged_simple_workspace_bytes(N, R, Hq, Hkv, D);
}

}  // namespace

extern "C" {

pkv_status pkv_qk_norm_rope(const void* q, const void* k, int64_t q_stride, int64_t k_stride, const float* q_weight,
                            const float* k_weight, const int32_t* positions, const float* inv_freq, int64_t N,
                            int32_t Hq, int32_t Hkv, int32_t D, int32_t rot_dim, float eps, int32_t dtype,
                            int32_t options, void* q_out, void* k_out, void* stream) {
  if (any_null({q, k, q_out, k_out})) return PKV_ERR_INVALID_ARGUMENT;
  const pkv_status st =
      check_norm_rope(q_stride, k_stride, inv_freq, N, Hq, Hkv, D, rot_dim, eps, dtype, options);
  if (st != PKV_OK) return st;
  const int64_t es = elem_size(dtype);
  if (!spans_ok({{q, strided_bytes(N, q_stride, Hq, D, es), 16}, {k, strided_bytes(N, k_stride, Hkv, D, es), 16},
                 f32_span(q_weight, D), f32_span(k_weight, D), i32_span(positions, N), f32_span(inv_freq, rot_dim / 2)},
                {{q_out, N * Hq * D * es, 16}, {k_out, N * Hkv * D * es, 16}}))
    return PKV_ERR_INVALID_ARGUMENT;
  const NormRopeArgs x{q,   k,  q_stride, k_stride, q_weight, k_weight, positions, inv_freq,
                       N,   Hq, Hkv,      D,        rot_dim,  eps,      (options & PKV_OPT_ROPE_INTERLEAVED) != 0,
                       q_out, k_out};
  return from_hip(launch_norm_rope(x, dtype, static_cast<hipStream_t>(stream)));
}

size_t pkv_qk_norm_rope_backward_workspace_size(int64_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype) {
  if (N < 1 || N > 4 * kMaxGroups || !heads_ok(Hq, Hkv) || !known_dtype(dtype) || !supported_head_dim(D)) return 0;
  return norm_rope_workspace_bytes(N, D);
}

pkv_status pkv_qk_norm_rope_backward(const void* q, const void* k, int64_t q_stride, int64_t k_stride,
                                     const void* dq_out, const void* dk_out, const float* q_weight,
                                     const float* k_weight, const int32_t* positions, const float* inv_freq,
                                     int64_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t rot_dim, float eps,
                                     int32_t dtype, int32_t options, void* dq, void* dk, float* dq_weight,
                                     float* dk_weight, void* workspace, size_t workspace_bytes, void* stream) {
  if (any_null({q, k, dq_out, dk_out, dq, dk})) return PKV_ERR_INVALID_ARGUMENT;
  const pkv_status st =
      check_norm_rope(q_stride, k_stride, inv_freq, N, Hq, Hkv, D, rot_dim, eps, dtype, options);
  if (st != PKV_OK) return st;
  const bool weights = dq_weight != nullptr || dk_weight != nullptr;
  const size_t need = weights ? norm_rope_workspace_bytes(N, D) : 0;
  if (!workspace_ok(workspace, workspace_bytes, need)) return PKV_ERR_WORKSPACE;
  const int64_t es = elem_size(dtype), qb = N * Hq * D * es, kb = N * Hkv * D * es;
  const Span qs{q, strided_bytes(N, q_stride, Hq, D, es), 16}, ks{k, strided_bytes(N, k_stride, Hkv, D, es), 16};
  if (!spans_ok({qs, ks, {dq_out, qb, 16}, {dk_out, kb, 16}, f32_span(q_weight, D), f32_span(k_weight, D),
                 i32_span(positions, N), f32_span(inv_freq, rot_dim / 2)},
                {{dq, qb, 16}, {dk, kb, 16}, f32_span(dq_weight, D), f32_span(dk_weight, D),
                 {need > 0 ? workspace : nullptr, int64_t(need), 16}}))
    return PKV_ERR_INVALID_ARGUMENT;
  const NormRopeArgs x{q, k,  q_stride, k_stride, q_weight, k_weight, positions, inv_freq,
                       N, Hq, Hkv,      D,        rot_dim,  eps,      (options & PKV_OPT_ROPE_INTERLEAVED) != 0,
                       nullptr, nullptr};
  const NormRopeGradArgs y{dq_out, dk_out, dq, dk, dq_weight, dk_weight, static_cast<float*>(workspace)};
  return from_hip(launch_norm_rope_backward(x, y, dtype, static_cast<hipStream_t>(stream)));
}

pkv_status pkv_attn_window_varlen(const void* q, const void* k, const void* v, const int32_t* cu_seqlens,
                                  int32_t max_segs, int64_t N, int32_t Hq, int32_t Hkv, int32_t D, float scale,
                                  int32_t dtype, int32_t window, int32_t sinks, void* o, float* lse, int32_t* flags,
                                  void* stream) {
  if (any_null({q, k, v, o})) return PKV_ERR_INVALID_ARGUMENT;
  const pkv_status st = check_window(cu_seqlens, max_segs, N, Hq, Hkv, D, scale, dtype, window, sinks);
  if (st != PKV_OK) return st;
  const int64_t es = elem_size(dtype), qb = N * Hq * D * es, kb = N * Hkv * D * es;
  if (!spans_ok({{q, qb, 16}, {k, kb, 16}, {v, kb, 16}, i32_span(cu_seqlens, int64_t(max_segs) + 1)},
                {{o, qb, 16}, f32_span(lse, N * Hq), i32_span(flags, 1)}))
    return PKV_ERR_INVALID_ARGUMENT;
  const AttnArgs a{q, k, v, cu_seqlens, max_segs, N, Hq, Hkv, D, scale, o, lse, flags, window, sinks};
  if (attn_mfma_supported(D, dtype)) return from_hip(launch_attn_fwd(a, static_cast<hipStream_t>(stream)));
  return from_hip(launch_attn_simple(a, dtype, static_cast<hipStream_t>(stream)));
}

size_t pkv_attn_window_varlen_backward_workspace_size(int64_t N, int32_t Hq, int32_t Hkv, int32_t D,
                                                      int32_t max_segs, int32_t dtype, int32_t window,
                                                      int32_t sinks) {
  // (a call without cu_seqlens has one segment, which a larger max_segs only adds to)
  const int32_t one = 1;
  if (check_window(&one, max_segs, N, Hq, Hkv, D, 1.f, dtype, window, sinks) != PKV_OK) return 0;
  return stats_bytes(N, Hq) +
         (attn_mfma_supported(D, dtype) ? attn_far_bytes(N, max_segs, Hkv, D, window, sinks) : 0);
}

pkv_status pkv_attn_window_varlen_backward(const void* q, const void* k, const void* v, const void* o,
                                           const float* lse, const void* dout, const int32_t* cu_seqlens,
                                           int32_t max_segs, int64_t N, int32_t Hq, int32_t Hkv, int32_t D,
                                           float scale, int32_t dtype, int32_t window, int32_t sinks, void* dq,
                                           void* dk, void* dv, int32_t* flags, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  if (any_null({q, k, v, o, lse, dout, dq, dk, dv})) return PKV_ERR_INVALID_ARGUMENT;
  const pkv_status st = check_window(cu_seqlens, max_segs, N, Hq, Hkv, D, scale, dtype, window, sinks);
  if (st != PKV_OK) return st;
  const size_t need =
      pkv_attn_window_varlen_backward_workspace_size(N, Hq, Hkv, D, max_segs, dtype, window, sinks);
  if (!workspace_ok(workspace, workspace_bytes, need)) return PKV_ERR_WORKSPACE;
  const int64_t es = elem_size(dtype), qb = N * Hq * D * es, kb = N * Hkv * D * es;
  const Span cs = i32_span(cu_seqlens, int64_t(max_segs) + 1), ls = f32_span(lse, N * Hq);
  if (!spans_ok({{q, qb, 16}, {k, kb, 16}, {v, kb, 16}, {o, qb, 16}, {dout, qb, 16}, ls, cs},
                {{dq, qb, 16}, {dk, kb, 16}, {dv, kb, 16}, i32_span(flags, 1)}))
    return PKV_ERR_INVALID_ARGUMENT;
  if (!spans_ok({{q, qb, 16}, {k, kb, 16}, {v, kb, 16}, {o, qb, 16}, {dout, qb, 16}, ls, cs, {dq, qb, 16},
                 {dk, kb, 16}, {dv, kb, 16}, i32_span(flags, 1)},
                {{workspace, int64_t(need), 256}}))
    return PKV_ERR_WORKSPACE;
  const AttnArgs a{q,     k, v, cu_seqlens, max_segs, N, Hq, Hkv, D, scale, const_cast<void*>(o), const_cast<float*>(lse),
                   flags, window, sinks};
  char* ws = static_cast<char*>(workspace);
  const AttnGradArgs g{dout, reinterpret_cast<float*>(ws), dq, dk, dv,
                       sinks > 0 ? reinterpret_cast<float*>(ws + stats_bytes(N, Hq)) : nullptr};
  if (attn_mfma_supported(D, dtype)) return from_hip(launch_attn_bwd(a, g, static_cast<hipStream_t>(stream)));
  return from_hip(launch_attn_simple_backward(a, g, dtype, static_cast<hipStream_t>(stream)));
}

pkv_status pkv_paged_kv_append(const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                               const int32_t* page_table, const int32_t* kv_lens, const int32_t* cu_seqlens,
                               int64_t N, int32_t R, int32_t Hkv, int32_t D, int32_t page_size, int32_t num_pages,
                               int32_t max_pages, int32_t dtype, void* k_pages, void* v_pages, int32_t* flags,
                               void* stream) {
  if (any_null({k, v, page_table, kv_lens, k_pages, v_pages})) return PKV_ERR_INVALID_ARGUMENT;
  const pkv_status st = check_paged(cu_seqlens, N, R, Hkv, Hkv, D, page_size, num_pages, max_pages, dtype);
  if (st != PKV_OK) return st;
  const int64_t es = elem_size(dtype), pb = int64_t(num_pages) * page_size * Hkv * D * es;
  if (!stride_ok(N, k_stride, Hkv, D, es) || !stride_ok(N, v_stride, Hkv, D, es)) return PKV_ERR_INVALID_ARGUMENT;
  if (!spans_ok({{k, strided_bytes(N, k_stride, Hkv, D, es), 16}, {v, strided_bytes(N, v_stride, Hkv, D, es), 16},
                 i32_span(page_table, int64_t(R) * max_pages), i32_span(kv_lens, R),
                 i32_span(cu_seqlens, int64_t(R) + 1)},
                {{k_pages, pb, 16}, {v_pages, pb, 16}, i32_span(flags, 1)}))
    return PKV_ERR_INVALID_ARGUMENT;
  const PagedArgs c{page_table, kv_lens, cu_seqlens, N, R, Hkv, D, page_size, num_pages, max_pages, flags};
  const AppendArgs x{k, v, k_stride, v_stride, k_pages, v_pages};
  return from_hip(launch_paged_append(c, x, dtype, static_cast<hipStream_t>(stream)));
}

size_t pkv_attn_paged_workspace_size(int64_t N, int32_t R, int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype) {
  const int32_t one = 1;
  if (check_paged(&one, N, R, Hq, Hkv, D, 16, 1, 1, dtype) != PKV_OK) return 0;
  return paged_workspace(N, R, Hq, Hkv, D, dtype, true);
}

pkv_status pkv_attn_paged(const void* q, const void* k_pages, const void* v_pages, const int32_t* page_table,
                          const int32_t* kv_lens, const int32_t* cu_seqlens, int64_t N, int32_t R, int32_t Hq,
                          int32_t Hkv, int32_t D, int32_t page_size, int32_t num_pages, int32_t max_pages,
                          float scale, int32_t dtype, int32_t window, int32_t sinks, void* o, float* lse,
                          int32_t* flags, void* workspace, size_t workspace_bytes, void* stream) {
  if (any_null({q, k_pages, v_pages, page_table, kv_lens, o})) return PKV_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(scale) || window < 0 || sinks < 0) return PKV_ERR_INVALID_ARGUMENT;
  const pkv_status st = check_paged(cu_seqlens, N, R, Hq, Hkv, D, page_size, num_pages, max_pages, dtype);
  if (st != PKV_OK) return st;
  if (window > 0 && sinks > kMaxSinks) return PKV_ERR_UNSUPPORTED;
  const size_t need = paged_workspace(N, R, Hq, Hkv, D, dtype, cu_seqlens != nullptr);
  if (!workspace_ok(workspace, workspace_bytes, need)) return PKV_ERR_WORKSPACE;
  const int64_t es = elem_size(dtype), qb = N * Hq * D * es, pb = int64_t(num_pages) * page_size * Hkv * D * es;
  const Span ws{need > 0 ? workspace : nullptr, int64_t(need), 256};
  if (!spans_ok({{q, qb, 16}, {k_pages, pb, 16}, {v_pages, pb, 16}, i32_span(page_table, int64_t(R) * max_pages),
                 i32_span(kv_lens, R), i32_span(cu_seqlens, int64_t(R) + 1)},
                {{o, qb, 16}, f32_span(lse, N * Hq), i32_span(flags, 1), ws}))
    return PKV_ERR_INVALID_ARGUMENT;
  const PagedArgs c{page_table, kv_lens, cu_seqlens, N, R, Hkv, D, page_size, num_pages, max_pages, flags};
  const AttnPagedArgs x{q, k_pages, v_pages, Hq, scale, window, window > 0 ? sinks : 0, o, lse, workspace};
  if (attn_mfma_supported(D, dtype)) return from_hip(launch_attn_paged(c, x, static_cast<hipStream_t>(stream)));
  return from_hip(launch_attn_paged_simple(c, x, dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
