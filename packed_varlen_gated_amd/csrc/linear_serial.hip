// Linear attention with one decay per head, token by token in fp32 (fp32
// tensors, and bf16 tensors with a head dimension of 32).
//
//   S_t = e^{g_h} S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t
// with S reset (or set to the slot's initial state) at every segment start: the
// recurrence of RFC-0026 Background with one decay in place of a gate per
// channel and no beta.
//
// One kernel runs the recurrence in either direction of time, and the reverse
// pass is three runs of it with the tensors in other roles:
//   dq_t = scale S_t do_t                      (a, b, c) = (do, v, k), forward, on S^T;
//   dv_t = dS_t^T k_t                          (k, q, do), backward, on dS;
//   dk_t = dS_t v_t                            (v, do, q), backward, on dS^T,
// where dS_t = e^{g} dS_{t+1} + scale q_t do_t^T and dS after the last token is
// the final state's cotangent. out_t = out_scale X_t^T a_t, X <- X + in_scale b_t c_t^T;
// forward the decay comes before a token's update, backward after its readout,
// so the state that leaves the walk backwards is the initial state's cotangent.
//
// One work-group of 256 threads per (slot, head): thread (rg, e) keeps column e,
// rows [rg R, rg R + R) of X in registers, tokens are staged through LDS in
// blocks of 16 and each block's partial readouts are reduced over the 256 / DB
// row groups.

#include "segments.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kTB = 16;
constexpr int kTail = 64;

template <typename T, int DA, int DB>
__global__ __launch_bounds__(kThreads) void linear_serial_kernel(
    const T* __restrict__ a, const T* __restrict__ b, const T* __restrict__ c, const float* __restrict__ g,
    const int32_t* __restrict__ cu, int32_t max_segs, int64_t N, int32_t H, float in_scale, float out_scale,
    bool reverse, bool transposed, const float* __restrict__ init, T* __restrict__ out,
    float* __restrict__ fin, int32_t* __restrict__ flags) {
  constexpr int RG = kThreads / DB, R = DA / RG;
  static_assert(RG * DB == kThreads && R * RG == DA, "bad tile");
  __shared__ float sa[kTB][DA], sb[kTB][DA], sc[kTB][DB], part[kTB][RG][DB];
  const int tid = threadIdx.x;
  const int64_t items = int64_t(max_segs) * H;
  if (int64_t(blockIdx.x) >= items) {
    const int64_t j = blockIdx.x - items;
    zero_tail(out, covered_tokens(cu, max_segs, N), N, int64_t(H) * DB * sizeof(T), j, kTail);
    if (j == 0) check_cu(cu, max_segs, N, flags);
    return;
  }
  const int32_t slot = int32_t(blockIdx.x / H), h = int32_t(blockIdx.x % H);
  const int64_t start = cu ? cu[slot] : 0, end = cu ? cu[slot + 1] : N;
  if (!segment_ok(slot, start, end, N)) return;

  const int e = tid % DB, rg = tid / DB;
  const float decay = expf(g[h]);
  const int64_t state0 = (int64_t(slot) * H + h) * DA * DB;
  float X[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int d = rg * R + r;
    X[r] = init == nullptr ? 0.f : init[state0 + (transposed ? e * DA + d : d * DB + e)];
  }
  for (int64_t t0 = 0; t0 < end - start; t0 += kTB) {
    const int nt = end - start - t0 < kTB ? int(end - start - t0) : kTB;
    __syncthreads();
    for (int i = tid; i < nt * DA; i += kThreads) {
      const int64_t t = reverse ? end - 1 - (t0 + i / DA) : start + t0 + i / DA;
      const int64_t off = (t * H + h) * DA + i % DA;
      sa[i / DA][i % DA] = to_f32(a[off]) * out_scale;
      sb[i / DA][i % DA] = to_f32(b[off]) * in_scale;
    }
    for (int i = tid; i < nt * DB; i += kThreads) {
      const int64_t t = reverse ? end - 1 - (t0 + i / DB) : start + t0 + i / DB;
      sc[i / DB][i % DB] = to_f32(c[(t * H + h) * DB + i % DB]);
    }
    __syncthreads();
    for (int tt = 0; tt < nt; ++tt) {
      const float y = sc[tt][e];
      float p = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (!reverse) X[r] *= decay;
        X[r] += sb[tt][rg * R + r] * y;
        p += X[r] * sa[tt][rg * R + r];
        if (reverse) X[r] *= decay;
      }
      part[tt][rg][e] = p;
    }
    __syncthreads();
    for (int i = tid; i < nt * DB; i += kThreads) {
      float p = 0.f;
#pragma unroll
      for (int j = 0; j < RG; ++j) p += part[i / DB][j][i % DB];
      const int64_t t = reverse ? end - 1 - (t0 + i / DB) : start + t0 + i / DB;
      out[(t * H + h) * DB + i % DB] = from_f32<T>(p);
    }
  }
  if (fin != nullptr) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int d = rg * R + r;
      fin[state0 + (transposed ? e * DA + d : d * DB + e)] = X[r];
    }
  }
}

template <typename T, int DA, int DB>
void run(const void* a, const void* b, const void* c, const LinearArgs& x, float in_scale, float out_scale,
         bool reverse, bool transposed, const float* init, void* out, float* fin, hipStream_t stream) {
  const int64_t grid = int64_t(x.max_segs) * x.H + kTail;
  linear_serial_kernel<T, DA, DB><<<dim3(uint32_t(grid)), dim3(kThreads), 0, stream>>>(
      static_cast<const T*>(a), static_cast<const T*>(b), static_cast<const T*>(c), x.g, x.cu, x.max_segs,
      x.N, x.H, in_scale, out_scale, reverse, transposed, init, static_cast<T*>(out), fin, x.flags);
}

template <typename T, int DK, int DV>
hipError_t fwd(const LinearArgs& x, hipStream_t s) {
  run<T, DK, DV>(x.q, x.k, x.v, x, 1.f, x.scale, false, false, x.initial_state, x.o, x.final_state, s);
  return hipGetLastError();
}

template <typename T, int DK, int DV>
hipError_t bwd(const LinearArgs& x, const LinearGradArgs& y, hipStream_t s) {
  run<T, DV, DK>(y.dout, x.v, x.k, x, 1.f, x.scale, false, true, x.initial_state, y.dq, nullptr, s);
  run<T, DV, DK>(x.v, y.dout, x.q, x, x.scale, 1.f, true, true, y.dfinal_state, y.dk, nullptr, s);
  run<T, DK, DV>(x.k, x.q, y.dout, x, x.scale, 1.f, true, false, y.dfinal_state, y.dv, y.d_initial_state, s);
  return hipGetLastError();
}

#define PKV_LINEAR_DISPATCH(fn, T, ...)                           \
  if (x.Dk == 32 && x.Dv == 32) return fn<T, 32, 32>(__VA_ARGS__);    \
  if (x.Dk == 32 && x.Dv == 64) return fn<T, 32, 64>(__VA_ARGS__);    \
  if (x.Dk == 32 && x.Dv == 128) return fn<T, 32, 128>(__VA_ARGS__);  \
  if (x.Dk == 64 && x.Dv == 32) return fn<T, 64, 32>(__VA_ARGS__);    \
  if (x.Dk == 64 && x.Dv == 64) return fn<T, 64, 64>(__VA_ARGS__);    \
  if (x.Dk == 64 && x.Dv == 128) return fn<T, 64, 128>(__VA_ARGS__);  \
  if (x.Dk == 128 && x.Dv == 32) return fn<T, 128, 32>(__VA_ARGS__);  \
  if (x.Dk == 128 && x.Dv == 64) return fn<T, 128, 64>(__VA_ARGS__);  \
  return fn<T, 128, 128>(__VA_ARGS__)

}  // namespace

hipError_t launch_linear_serial(const LinearArgs& x, int32_t dtype, hipStream_t stream) {
  if (dtype == 1) { PKV_LINEAR_DISPATCH(fwd, float, x, stream); }
  PKV_LINEAR_DISPATCH(fwd, bf16, x, stream);
}

hipError_t launch_linear_serial_backward(const LinearArgs& x, const LinearGradArgs& y, int32_t dtype,
                                         hipStream_t stream) {
  if (dtype == 1) { PKV_LINEAR_DISPATCH(bwd, float, x, y, stream); }
  PKV_LINEAR_DISPATCH(bwd, bf16, x, y, stream);
}

}  // namespace pkv
