// Single-token steps of the recurrences for serving: one token of each of R
// requests, the state of request r in slot slots[r] (slot r without slots),
// updated in place.
//   linear attention:  S = e^{g_h} S + k v^T
//   KDA (RFC-0026 Background):  S = diag(e^{g}) S + beta k v^T
//   o = scale S^T q  (readout after the update)
//
// Bound by the state's bytes: 4 Dk Dv read and written per (request, head)
// against 4 Dk Dv operations. A work-group takes a slice of the value columns
// of one (request, head); a thread reads 16 bytes of a row at a time, all its
// rows before the first use, and the readout is summed over the row groups
// through LDS. 123 rows, H 32, 128 x 128: 107 us for 516 MB (4.8 TB/s; a copy
// reaches 5.2); KDA with 48 rows: 39.6 us (5.1 TB/s); one row, H 16: 3.8 us, a
// launch. A slice is 32 columns, so that one row of 16 heads has 64 work-groups.
//
// A row whose slot is negative is idle: o = 0 and no state is touched. A slot
// past the last one, or one that an earlier row of the call names too, is
// treated the same way and sets kFlagBadSlot: the rows of a call never race.

#include "common.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr float kL2NormEps = 1e-6f;  // added to a squared norm (the q/k L2 normalisation option)

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <typename T, int DK, int DV, int CW, bool kKda>
__global__ __launch_bounds__(kThreads) void step_kernel(
    const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, const void* __restrict__ gv,
    const T* __restrict__ beta, const int32_t* __restrict__ slots, int32_t S, int32_t H, float scale,
    bool qk_l2norm, float* __restrict__ state, T* __restrict__ o, int32_t* __restrict__ flags) {
  constexpr int TC = CW / 4;             // threads per row of the slice
  constexpr int RG = kThreads / TC;      // row groups
  constexpr int R = DK / RG > 0 ? DK / RG : 1;  // rows per thread
  constexpr int USED = DK / R * TC;      // threads that hold rows
  __shared__ float sq[DK], sk[DK], sg[DK], part[DK / R][CW], norm[2];
  const int tid = threadIdx.x;
  const int32_t h = blockIdx.y;
  const int64_t r = blockIdx.x / (DV / CW);
  const int c0 = int(blockIdx.x % (DV / CW)) * CW;
  const int64_t slot = slots == nullptr ? r : slots[r];
  const int64_t row = r * H + h;

  bool bad = slots != nullptr && slot >= S;
  const bool live = !bad && slot >= 0;
  const int rg = tid / TC, c = c0 + tid % TC * 4;
  float* p = state + ((slot * H + h) * DK + rg * R) * DV + c;
  f32x4 x[R];
  if (live && tid < USED) {
#pragma unroll
    for (int i = 0; i < R; ++i) x[i] = *reinterpret_cast<const f32x4*>(p + i * DV);
  }
  if (live && slots != nullptr) {
    // while the state comes: the earlier rows' slots, 16 bytes a load
    typedef int32_t i32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
    const int64_t quads = r / 4;
#pragma unroll 4
    for (int64_t i = tid; i < quads; i += kThreads) {
      const i32x4_a4 y = *reinterpret_cast<const i32x4_a4*>(slots + 4 * i);
      bad |= (y[0] == slot) | (y[1] == slot) | (y[2] == slot) | (y[3] == slot);
    }
    if (tid < r % 4) bad |= slots[4 * quads + tid] == slot;
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0 && h == 0 && c0 == 0 && flags != nullptr) atomicOr(flags, kFlagBadSlot);
  if (bad || !live) {
    if (tid < CW) o[row * DV + c0 + tid] = from_f32<T>(0.f);
    return;
  }

  if (tid < DK) {
    sq[tid] = to_f32(q[row * DK + tid]);
    const float kk = to_f32(k[row * DK + tid]);
    if constexpr (kKda) {
      sk[tid] = kk;
      sg[tid] = expf(to_f32(static_cast<const T*>(gv)[row * DK + tid]));
    } else {
      sk[tid] = kk;
      sg[tid] = expf(static_cast<const float*>(gv)[h]);
    }
  }
  __syncthreads();
  float nq = scale, nk = kKda ? to_f32(beta[row]) : 1.f;
  if (kKda && qk_l2norm) {
    if (tid < 128) {
      const float* s = tid < 64 ? sq : sk;
      float y = 0.f;
      for (int d = tid & 63; d < DK; d += 64) y += s[d] * s[d];
      for (int d = 32; d; d >>= 1) y += __shfl_xor(y, d, 64);
      if ((tid & 63) == 0) norm[tid >> 6] = rsqrtf(y + kL2NormEps);
    }
    __syncthreads();
    nq *= norm[0];
    nk *= norm[1];
  }
  if (tid < USED) {
    f32x4 y = {0.f, 0.f, 0.f, 0.f}, w;
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = to_f32(v[row * DV + c + j]) * nk;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int d = rg * R + i;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[i][j] = x[i][j] * sg[d] + sk[d] * w[j];
        y[j] += x[i][j] * sq[d];
      }
      *reinterpret_cast<f32x4*>(p + i * DV) = x[i];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) part[rg][tid % TC * 4 + j] = y[j];
  }
  __syncthreads();
  if (tid < CW) {
    float y = 0.f;
    for (int i = 0; i < DK / R; ++i) y += part[i][tid];
    o[row * DV + c0 + tid] = from_f32<T>(y * nq);
  }
}

template <typename T, int DK, int DV, bool kKda>
hipError_t run(const StepArgs& a, hipStream_t stream) {
  constexpr int CW = 32;
  const dim3 grid(uint32_t(a.R * (DV / CW)), uint32_t(a.H));
  step_kernel<T, DK, DV, CW, kKda><<<grid, dim3(kThreads), 0, stream>>>(
      static_cast<const T*>(a.q), static_cast<const T*>(a.k), static_cast<const T*>(a.v), a.g,
      static_cast<const T*>(a.beta), a.slots, a.S, a.H, a.scale, a.qk_l2norm, a.state, static_cast<T*>(a.o),
      a.flags);
  return hipGetLastError();
}

template <typename T, bool kKda>
hipError_t shapes(const StepArgs& a, hipStream_t s) {
  if (a.Dk == 32) {
    if (a.Dv == 32) return run<T, 32, 32, kKda>(a, s);
    if (a.Dv == 64) return run<T, 32, 64, kKda>(a, s);
    return run<T, 32, 128, kKda>(a, s);
  }
  if (a.Dk == 64) {
    if (a.Dv == 32) return run<T, 64, 32, kKda>(a, s);
    if (a.Dv == 64) return run<T, 64, 64, kKda>(a, s);
    return run<T, 64, 128, kKda>(a, s);
  }
  if (a.Dv == 32) return run<T, 128, 32, kKda>(a, s);
  if (a.Dv == 64) return run<T, 128, 64, kKda>(a, s);
  return run<T, 128, 128, kKda>(a, s);
}

}  // namespace

hipError_t launch_step(const StepArgs& a, int32_t dtype, hipStream_t stream) {
  if (a.beta != nullptr) return dtype == 1 ? shapes<float, true>(a, stream) : shapes<bf16, true>(a, stream);
  return dtype == 1 ? shapes<float, false>(a, stream) : shapes<bf16, false>(a, stream);
}

}  // namespace pkv
