// Argument validation and dispatch of the calls in include/pkv_mixers.h. Every
// check runs before any HIP call, so invalid arguments are reported
// synchronously and nothing is enqueued.

#include "pkv_mixers.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <initializer_list>

#include "common.h"

namespace {

constexpr int64_t kInt32Max = 2147483647;
// Work-groups of a launch: a grid holds less than 2^32 work-items, of at most 512
// a group.
constexpr int64_t kMaxGroups = int64_t(1) << 23;

bool supported_head_dim(int32_t d) { return d == 32 || d == 64 || d == 128; }
bool known_dtype(int32_t dt) { return dt == PKV_BF16 || dt == PKV_F32; }
int64_t elem_size(int32_t dt) { return dt == PKV_BF16 ? 2 : 4; }
pkv_status from_hip(hipError_t e) { return e == hipSuccess ? PKV_OK : PKV_ERR_HIP; }

struct Span {
  const void* p;
  int64_t bytes;
  int64_t align;
};

bool overlap(const Span& a, const Span& b) {
  if (a.p == nullptr || b.p == nullptr) return false;
  const char *x = static_cast<const char*>(a.p), *y = static_cast<const char*>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}

// Alignment of every span, and no output on an input or another output.
bool spans_ok(std::initializer_list<Span> ins, std::initializer_list<Span> outs) {
  for (const Span& s : ins)
    if (reinterpret_cast<uintptr_t>(s.p) % s.align != 0) return false;
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    if (reinterpret_cast<uintptr_t>(o->p) % o->align != 0) return false;
    for (const Span& s : ins)
      if (overlap(*o, s)) return false;
    for (const Span* p = outs.begin(); p != o; ++p)
      if (overlap(*o, *p)) return false;
  }
  return true;
}

bool any_null(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (p == nullptr) return true;
  return false;
}

// N, max_segs (set to 1 without cu) and scale of a packed call.
bool packed_sizes_ok(const int32_t* cu, int32_t& max_segs, int64_t N, float scale) {
  if (N < 1 || N > kInt32Max || !std::isfinite(scale)) return false;
  if (cu == nullptr) max_segs = 1;
  return max_segs >= 1 && max_segs < kInt32Max;
}

Span cu_span(const int32_t* cu, int32_t max_segs) { return {cu, (int64_t(max_segs) + 1) * 4, 4}; }

pkv_status check_attn(const int32_t* cu, int32_t& max_segs, int64_t N, int32_t Hq, int32_t Hkv, int32_t D,
                      float scale, int32_t dtype) {
  if (!packed_sizes_ok(cu, max_segs, N, scale) || Hq < 1 || Hkv < 1 || Hq > 65536 || Hkv > 65536 ||
      Hq % Hkv != 0)
    return PKV_ERR_INVALID_ARGUMENT;
  if (!known_dtype(dtype) || !supported_head_dim(D)) return PKV_ERR_UNSUPPORTED;
  if ((N / 32 + max_segs) * Hq >= kMaxGroups) return PKV_ERR_INVALID_ARGUMENT;
  return PKV_OK;
}

pkv_status check_linear(const int32_t* cu, int32_t& max_segs, int64_t N, int32_t H, int32_t Dk, int32_t Dv,
                        float scale, int32_t dtype) {
  if (!packed_sizes_ok(cu, max_segs, N, scale) || H < 1 || H > 65536 ||
      int64_t(max_segs) * H > (int64_t(1) << 22))
    return PKV_ERR_INVALID_ARGUMENT;
  if (!known_dtype(dtype) || !supported_head_dim(Dk) || !supported_head_dim(Dv)) return PKV_ERR_UNSUPPORTED;
  if (pkv::linear_chunk_supported(Dk, Dv, dtype) && pkv::linear_chunk_grid(N, max_segs, H) >= kMaxGroups)
    return PKV_ERR_INVALID_ARGUMENT;
  return PKV_OK;
}

size_t linear_workspace(int64_t N, int32_t H, int32_t Dk, int32_t Dv, int32_t dtype, bool reverse) {
  if (N < 1 || N > kInt32Max || H < 1 || H > 65536 || !pkv::linear_chunk_supported(Dk, Dv, dtype)) return 0;
  return pkv::linear_chunk_workspace_bytes(N, H, Dk, Dv, reverse);
}

bool workspace_ok(const void* ws, size_t bytes, size_t need) {
  return need == 0 || (ws != nullptr && bytes >= need && reinterpret_cast<uintptr_t>(ws) % 256 == 0);
}

}  // namespace

extern "C" {

pkv_status pkv_attn_varlen(const void* q, const void* k, const void* v, const int32_t* cu_seqlens,
                           int32_t max_segs, int64_t N, int32_t Hq, int32_t Hkv, int32_t D, float scale,
                           int32_t dtype, void* o, float* lse, int32_t* flags, void* stream) {
  if (any_null({q, k, v, o})) return PKV_ERR_INVALID_ARGUMENT;
  const pkv_status st = check_attn(cu_seqlens, max_segs, N, Hq, Hkv, D, scale, dtype);
  if (st != PKV_OK) return st;
  const int64_t qb = N * Hq * D * elem_size(dtype), kb = N * Hkv * D * elem_size(dtype);
  if (!spans_ok({{q, qb, 16}, {k, kb, 16}, {v, kb, 16}, cu_span(cu_seqlens, max_segs)},
                {{o, qb, 16}, {lse, N * Hq * 4, 4}, {flags, 4, 4}}))
    return PKV_ERR_INVALID_ARGUMENT;
  const pkv::AttnArgs a{q, k, v, cu_seqlens, max_segs, N, Hq, Hkv, D, scale, o, lse, flags};
  if (pkv::attn_mfma_supported(D, dtype))
    return from_hip(pkv::launch_attn_fwd(a, static_cast<hipStream_t>(stream)));
  return from_hip(pkv::launch_attn_simple(a, dtype, static_cast<hipStream_t>(stream)));
}

size_t pkv_attn_varlen_backward_workspace_size(int64_t N, int32_t Hq, int32_t Hkv, int32_t D,
                                               int32_t max_segs, int32_t dtype) {
  if (check_attn(nullptr, max_segs, N, Hq, Hkv, D, 1.f, dtype) != PKV_OK) return 0;
  return size_t(N) * Hq * 8 + 16;  // two numbers per row; the form of the keys pass
}

pkv_status pkv_attn_varlen_backward(const void* q, const void* k, const void* v, const void* o,
                                    const float* lse, const void* dout, const int32_t* cu_seqlens,
                                    int32_t max_segs, int64_t N, int32_t Hq, int32_t Hkv, int32_t D,
                                    float scale, int32_t dtype, void* dq, void* dk, void* dv, int32_t* flags,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  if (any_null({q, k, v, o, lse, dout, dq, dk, dv})) return PKV_ERR_INVALID_ARGUMENT;
  const pkv_status st = check_attn(cu_seqlens, max_segs, N, Hq, Hkv, D, scale, dtype);
  if (st != PKV_OK) return st;
  const size_t need = pkv_attn_varlen_backward_workspace_size(N, Hq, Hkv, D, max_segs, dtype);
  if (!workspace_ok(workspace, workspace_bytes, need)) return PKV_ERR_WORKSPACE;
  const int64_t qb = N * Hq * D * elem_size(dtype), kb = N * Hkv * D * elem_size(dtype);
  const std::initializer_list<Span> ins = {{q, qb, 16},    {k, kb, 16},       {v, kb, 16}, {o, qb, 16},
                                           {dout, qb, 16}, {lse, N * Hq * 4, 4}, cu_span(cu_seqlens, max_segs)};
  if (!spans_ok(ins, {{dq, qb, 16}, {dk, kb, 16}, {dv, kb, 16}, {flags, 4, 4}}))
    return PKV_ERR_INVALID_ARGUMENT;
  if (!spans_ok({{q, qb, 16}, {k, kb, 16}, {v, kb, 16}, {o, qb, 16}, {dout, qb, 16}, {lse, N * Hq * 4, 4},
                 cu_span(cu_seqlens, max_segs), {dq, qb, 16}, {dk, kb, 16}, {dv, kb, 16}, {flags, 4, 4}},
                {{workspace, int64_t(need), 256}}))
    return PKV_ERR_WORKSPACE;
  const pkv::AttnArgs a{q,   k,   v, cu_seqlens, max_segs, N, Hq, Hkv, D, scale, const_cast<void*>(o),
                        const_cast<float*>(lse), flags};
  const pkv::AttnGradArgs g{dout, static_cast<float*>(workspace), dq, dk, dv};
  if (pkv::attn_mfma_supported(D, dtype))
    return from_hip(pkv::launch_attn_bwd(a, g, static_cast<hipStream_t>(stream)));
  return from_hip(pkv::launch_attn_simple_backward(a, g, dtype, static_cast<hipStream_t>(stream)));
}

size_t pkv_linear_attn_varlen_workspace_size(int64_t N, int32_t H, int32_t Dk, int32_t Dv, int32_t max_segs,
                                             int32_t dtype) {
  return linear_workspace(N, H, Dk, Dv, dtype, false);
}

pkv_status pkv_linear_attn_varlen(const void* q, const void* k, const void* v, const float* g,
                                  const int32_t* cu_seqlens, int32_t max_segs, int64_t N, int32_t H,
                                  int32_t Dk, int32_t Dv, float scale, int32_t dtype,
                                  const float* initial_state, void* o, float* final_state, int32_t* flags,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  if (any_null({q, k, v, g, o})) return PKV_ERR_INVALID_ARGUMENT;
  const pkv_status st = check_linear(cu_seqlens, max_segs, N, H, Dk, Dv, scale, dtype);
  if (st != PKV_OK) return st;
  const size_t need = pkv_linear_attn_varlen_workspace_size(N, H, Dk, Dv, max_segs, dtype);
  if (!workspace_ok(workspace, workspace_bytes, need)) return PKV_ERR_WORKSPACE;
  const int64_t kb = N * H * Dk * elem_size(dtype), vb = N * H * Dv * elem_size(dtype);
  const int64_t sb = int64_t(max_segs) * H * Dk * Dv * 4;
  if (!spans_ok({{q, kb, 16}, {k, kb, 16}, {v, vb, 16}, {g, int64_t(H) * 4, 4}, cu_span(cu_seqlens, max_segs),
                 {initial_state, sb, 16}},
                {{o, vb, 16}, {final_state, sb, 16}, {flags, 4, 4},
                 {need > 0 ? workspace : nullptr, int64_t(need), 16}}))
    return PKV_ERR_INVALID_ARGUMENT;
  const pkv::LinearArgs x{q,  k,  v,     g,             cu_seqlens, max_segs,    N,     H,
                          Dk, Dv, scale, initial_state, o,          final_state, flags, workspace};
  if (pkv::linear_chunk_supported(Dk, Dv, dtype))
    return from_hip(pkv::launch_linear_chunk(x, static_cast<hipStream_t>(stream)));
  return from_hip(pkv::launch_linear_serial(x, dtype, static_cast<hipStream_t>(stream)));
}

size_t pkv_linear_attn_varlen_backward_workspace_size(int64_t N, int32_t H, int32_t Dk, int32_t Dv,
                                                      int32_t max_segs, int32_t dtype) {
  return linear_workspace(N, H, Dk, Dv, dtype, true);
}

pkv_status pkv_linear_attn_varlen_backward(const void* q, const void* k, const void* v, const float* g,
                                           const int32_t* cu_seqlens, int32_t max_segs, int64_t N, int32_t H,
                                           int32_t Dk, int32_t Dv, float scale, int32_t dtype,
                                           const float* initial_state, const void* dout,
                                           const float* dfinal_state, void* dq, void* dk, void* dv,
                                           float* d_initial_state, int32_t* flags, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  if (any_null({q, k, v, g, dout, dq, dk, dv})) return PKV_ERR_INVALID_ARGUMENT;
  const pkv_status st = check_linear(cu_seqlens, max_segs, N, H, Dk, Dv, scale, dtype);
  if (st != PKV_OK) return st;
  const size_t need = pkv_linear_attn_varlen_backward_workspace_size(N, H, Dk, Dv, max_segs, dtype);
  if (!workspace_ok(workspace, workspace_bytes, need)) return PKV_ERR_WORKSPACE;
  const int64_t kb = N * H * Dk * elem_size(dtype), vb = N * H * Dv * elem_size(dtype);
  const int64_t sb = int64_t(max_segs) * H * Dk * Dv * 4;
  if (!spans_ok({{q, kb, 16}, {k, kb, 16}, {v, vb, 16}, {dout, vb, 16}, {g, int64_t(H) * 4, 4},
                 cu_span(cu_seqlens, max_segs), {initial_state, sb, 16}, {dfinal_state, sb, 16}},
                {{dq, kb, 16}, {dk, kb, 16}, {dv, vb, 16}, {d_initial_state, sb, 16}, {flags, 4, 4},
                 {need > 0 ? workspace : nullptr, int64_t(need), 16}}))
    return PKV_ERR_INVALID_ARGUMENT;
  const pkv::LinearArgs x{q,  k,  v,     g,             cu_seqlens, max_segs, N,     H,
                          Dk, Dv, scale, initial_state, nullptr,    nullptr,  flags, workspace};
  const pkv::LinearGradArgs y{dout, dfinal_state, dq, dk, dv, d_initial_state};
  if (pkv::linear_chunk_supported(Dk, Dv, dtype))
    return from_hip(pkv::launch_linear_chunk_backward(x, y, static_cast<hipStream_t>(stream)));
  return from_hip(pkv::launch_linear_serial_backward(x, y, dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

namespace {

pkv_status step(const void* q, const void* k, const void* v, const void* g, int64_t g_bytes, int64_t g_align,
                const void* beta, const int32_t* slots, int64_t R, int32_t S, int32_t H, int32_t Dk, int32_t Dv,
                float scale, int32_t dtype, bool l2, float* state, void* o, int32_t* flags, void* stream) {
  if (any_null({q, k, v, g, state, o})) return PKV_ERR_INVALID_ARGUMENT;
  if (R < 1 || R > (int64_t(1) << 20) || S < 1 || H < 1 || H > 65535 || !std::isfinite(scale) ||
      (slots == nullptr && R > S))
    return PKV_ERR_INVALID_ARGUMENT;
  if (!known_dtype(dtype) || !supported_head_dim(Dk) || !supported_head_dim(Dv)) return PKV_ERR_UNSUPPORTED;
  const int64_t es = elem_size(dtype), kb = R * H * Dk * es, vb = R * H * Dv * es;
  if (!spans_ok({{q, kb, 16}, {k, kb, 16}, {v, vb, 16}, {g, g_bytes, g_align}, {beta, R * H * es, es},
                 {slots, R * 4, 4}},
                {{state, int64_t(S) * H * Dk * Dv * 4, 16}, {o, vb, 16}, {flags, 4, 4}}))
    return PKV_ERR_INVALID_ARGUMENT;
  const pkv::StepArgs a{q, k, v, g, beta, slots, R, S, H, Dk, Dv, scale, l2, state, o, flags};
  return from_hip(pkv::launch_step(a, dtype, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

pkv_status pkv_linear_attn_step(const void* q, const void* k, const void* v, const float* g,
                                const int32_t* slots, int64_t R, int32_t S, int32_t H, int32_t Dk, int32_t Dv,
                                float scale, int32_t dtype, float* state, void* o, int32_t* flags,
                                void* stream) {
  return step(q, k, v, g, int64_t(H) * 4, 4, nullptr, slots, R, S, H, Dk, Dv, scale, dtype, false, state, o,
              flags, stream);
}

pkv_status pkv_kda_step(const void* q, const void* k, const void* v, const void* g, const void* beta,
                        const int32_t* slots, int64_t R, int32_t S, int32_t H, int32_t Dk, int32_t Dv,
                        float scale, int32_t dtype, int32_t options, float* state, void* o, int32_t* flags,
                        void* stream) {
  if (beta == nullptr) return PKV_ERR_INVALID_ARGUMENT;
  if ((options & ~PKV_OPT_QK_L2NORM) != 0) return PKV_ERR_UNSUPPORTED;
  return step(q, k, v, g, R * H * Dk * (known_dtype(dtype) ? elem_size(dtype) : 4), 16, beta, slots, R, S, H,
              Dk, Dv, scale, dtype, (options & PKV_OPT_QK_L2NORM) != 0, state, o, flags, stream);
}

}  // extern "C"
