// Packed causal softmax attention with grouped heads, and its reverse pass, on
// the vector units in fp32: fp32 tensors, and bf16 tensors at D = 32.
//
// Token t of a segment attends to the tokens s <= t of the same segment
// ("Drill: Sequence Packing from scratch", The math: doc(s) = doc(t), s <= t):
//   P_ts = exp(scale q_t.k_s - lse_t),  lse_t = ln sum_s exp(scale q_t.k_s),
//   o_t = sum_s P_ts v_s.
// Reverse pass, with delta_t = do_t.o_t and dS_ts = P_ts (do_t.v_s - delta_t):
//   dq_t = scale sum_s dS_ts k_s, dk_s = scale sum_t dS_ts q_t,
//   dv_s = sum_t P_ts do_t, the last two also summed over the query heads that
//   share the kv head, in a fixed order (no atomics).
// Query head h reads kv head h / (Hq / Hkv).
//
// A work-group of 256 threads takes 32 rows (queries, or keys in the dk/dv
// pass) of one head and walks the other side in tiles of 32 staged in LDS as
// fp32. Thread (r, c) = (tid / 8, tid % 8) holds row r's scores of columns
// c + 8 j and its output channels c + 8 j; the softmax runs in one pass with a
// running maximum and sum. These shapes serve fp32 batches that models are
// debugged on; the MFMA kernels serve bf16 at D = 64 and 128.

#include "segments.h"

namespace pkv {
namespace {

constexpr int kT = 32;        // tokens per tile, both sides
constexpr int kThreads = 256;
constexpr int kTail = 64;     // work-groups that zero the rows no segment has

// 32 rows of a [N, H, D] tensor from `row` on, fp32, zero past `end`.
template <typename T, int D>
__device__ __forceinline__ void stage(float (&dst)[kT][D + 1], const T* __restrict__ src, int64_t row,
                                      int64_t end, int32_t H, int32_t h) {
  for (int i = threadIdx.x; i < kT * D; i += kThreads) {
    const int r = i / D, d = i % D;
    dst[r][d] = row + r < end ? to_f32(src[((row + r) * H + h) * D + d]) : 0.f;
  }
}

// Over the 8 threads of a row.
__device__ __forceinline__ float row_max(float x) {
  for (int d = 4; d; d >>= 1) x = fmaxf(x, __shfl_xor(x, d, 8));
  return x;
}
__device__ __forceinline__ float row_sum(float x) {
  for (int d = 4; d; d >>= 1) x += __shfl_xor(x, d, 8);
  return x;
}

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_simple_fwd(
    const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
    const int32_t* __restrict__ cu, int32_t max_segs, int64_t N, int32_t H, int32_t Hkv, float scale,
    T* __restrict__ o, float* __restrict__ lse, int32_t* __restrict__ flags, int64_t slots) {
  __shared__ float sq[kT][D + 1], sk[kT][D + 1], sv[kT][D + 1], sp[kT][kT + 1];
  const int64_t b = blockIdx.x;
  if (b >= slots * H) {
    const int64_t j = b - slots * H, c = covered_tokens(cu, max_segs, N);
    zero_tail(o, c, N, int64_t(H) * D * sizeof(T), j, kTail);
    if (lse != nullptr)
      for (int64_t i = j * kThreads + threadIdx.x; i < (N - c) * H; i += int64_t(kTail) * kThreads)
        lse[(i / (N - c)) * N + c + i % (N - c)] = -INFINITY;
    if (j == 0) check_cu(cu, max_segs, N, flags);
    return;
  }
  const int32_t h = int32_t(b % H);
  SegTile t;
  if (!find_tile(cu, max_segs, N, kT, int32_t(b / H), t)) return;
  const int32_t hk = h / (H / Hkv);
  const int r = threadIdx.x / 8, c = threadIdx.x % 8;
  const int64_t row = int64_t(t.start) + r;

  stage<T, D>(sq, q, t.start, t.e, H, h);
  float m = -INFINITY, l = 0.f, acc[D / 8] = {};
  for (int64_t s0 = t.a; s0 < t.start + kT && s0 < t.e; s0 += kT) {
    __syncthreads();
    stage<T, D>(sk, k, s0, t.e, Hkv, hk);
    stage<T, D>(sv, v, s0, t.e, Hkv, hk);
    __syncthreads();
    float x[kT / 8] = {};
    for (int d = 0; d < D; ++d) {
      const float y = sq[r][d];
#pragma unroll
      for (int j = 0; j < kT / 8; ++j) x[j] += y * sk[c + 8 * j][d];
    }
    float mt = m;
#pragma unroll
    for (int j = 0; j < kT / 8; ++j) {
      x[j] = s0 + c + 8 * j <= row ? x[j] * scale : -INFINITY;
      mt = fmaxf(mt, x[j]);
    }
    mt = row_max(mt);
    // a row whose scores so far are all -inf has no maximum to subtract
    const float ms = mt == -INFINITY ? 0.f : mt;
    const float f = expf(m - ms);
    float lt = 0.f;
#pragma unroll
    for (int j = 0; j < kT / 8; ++j) {
      const float p = expf(x[j] - ms);
      lt += p;
      sp[r][c + 8 * j] = p;
    }
    l = l * f + row_sum(lt);
    m = mt;
#pragma unroll
    for (int j = 0; j < D / 8; ++j) acc[j] *= f;
    __syncthreads();
    // only the keys the row attends to: a later key's value takes no part,
    // whatever it holds
    const int64_t last = row - s0 < kT - 1 ? row - s0 : kT - 1;
    for (int s = 0; s <= last; ++s) {
      const float p = sp[r][s];
#pragma unroll
      for (int j = 0; j < D / 8; ++j) acc[j] += p * sv[s][c + 8 * j];
    }
  }
  if (row >= t.e) return;
  const float inv = 1.f / l;
#pragma unroll
  for (int j = 0; j < D / 8; ++j) o[(row * H + h) * D + c + 8 * j] = from_f32<T>(acc[j] * inv);
  if (lse != nullptr && c == 0) lse[int64_t(h) * N + row] = m + logf(l);
}

// delta_t = do_t.o_t, fp32 [H, N].
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_delta(const T* __restrict__ o, const T* __restrict__ dout,
                                                       float* __restrict__ delta, int64_t N, int32_t H) {
  const int64_t i = int64_t(blockIdx.x) * (kThreads / 8) + threadIdx.x / 8;  // token * H + head
  const int c = threadIdx.x % 8;
  float x = 0.f;
  if (i < N * H)
    for (int d = c; d < D; d += 8) x += to_f32(o[i * D + d]) * to_f32(dout[i * D + d]);
  x = row_sum(x);
  if (i < N * H && c == 0) delta[(i % H) * N + i / H] = x;
}

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_simple_dq(
    const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, const T* __restrict__ dout,
    const float* __restrict__ lse, const float* __restrict__ delta, const int32_t* __restrict__ cu,
    int32_t max_segs, int64_t N, int32_t H, int32_t Hkv, float scale, T* __restrict__ dq,
    int32_t* __restrict__ flags, int64_t slots) {
  __shared__ float sq[kT][D + 1], sdo[kT][D + 1], sk[kT][D + 1], sv[kT][D + 1], sp[kT][kT + 1];
  const int64_t b = blockIdx.x;
  if (b >= slots * H) {
    zero_tail(dq, covered_tokens(cu, max_segs, N), N, int64_t(H) * D * sizeof(T), b - slots * H, kTail);
    if (b == slots * H) check_cu(cu, max_segs, N, flags);
    return;
  }
  const int32_t h = int32_t(b % H);
  SegTile t;
  if (!find_tile(cu, max_segs, N, kT, int32_t(b / H), t)) return;
  const int32_t hk = h / (H / Hkv);
  const int r = threadIdx.x / 8, c = threadIdx.x % 8;
  const int64_t row = int64_t(t.start) + r;
  const bool real = row < t.e;
  const float ls = real ? lse[int64_t(h) * N + row] : INFINITY;
  const float dl = real ? delta[int64_t(h) * N + row] : 0.f;

  stage<T, D>(sq, q, t.start, t.e, H, h);
  stage<T, D>(sdo, dout, t.start, t.e, H, h);
  float acc[D / 8] = {};
  for (int64_t s0 = t.a; s0 < t.start + kT && s0 < t.e; s0 += kT) {
    __syncthreads();
    stage<T, D>(sk, k, s0, t.e, Hkv, hk);
    stage<T, D>(sv, v, s0, t.e, Hkv, hk);
    __syncthreads();
    float x[kT / 8] = {}, y[kT / 8] = {};
    for (int d = 0; d < D; ++d) {
#pragma unroll
      for (int j = 0; j < kT / 8; ++j) {
        x[j] += sq[r][d] * sk[c + 8 * j][d];
        y[j] += sdo[r][d] * sv[c + 8 * j][d];
      }
    }
#pragma unroll
    for (int j = 0; j < kT / 8; ++j)
      sp[r][c + 8 * j] = s0 + c + 8 * j <= row ? expf(x[j] * scale - ls) * (y[j] - dl) : 0.f;
    __syncthreads();
    const int64_t last = row - s0 < kT - 1 ? row - s0 : kT - 1;
    for (int s = 0; s <= last; ++s) {
      const float p = sp[r][s];
#pragma unroll
      for (int j = 0; j < D / 8; ++j) acc[j] += p * sk[s][c + 8 * j];
    }
  }
  if (!real) return;
#pragma unroll
  for (int j = 0; j < D / 8; ++j) dq[(row * H + h) * D + c + 8 * j] = from_f32<T>(acc[j] * scale);
}

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_simple_dkv(
    const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, const T* __restrict__ dout,
    const float* __restrict__ lse, const float* __restrict__ delta, const int32_t* __restrict__ cu,
    int32_t max_segs, int64_t N, int32_t H, int32_t Hkv, float scale, T* __restrict__ dk,
    T* __restrict__ dv, int64_t slots) {
  // x of row r (a key) and column s (a query)
  __shared__ float sq[kT][D + 1], sdo[kT][D + 1], sk[kT][D + 1], sv[kT][D + 1];
  __shared__ float sp[kT][kT + 1], sd[kT][kT + 1], sl[kT], sdl[kT];
  const int64_t b = blockIdx.x;
  if (b >= slots * Hkv) {
    const int64_t j = b - slots * Hkv, cov = covered_tokens(cu, max_segs, N);
    zero_tail(dk, cov, N, int64_t(Hkv) * D * sizeof(T), j, kTail);
    zero_tail(dv, cov, N, int64_t(Hkv) * D * sizeof(T), j, kTail);
    return;
  }
  const int32_t hk = int32_t(b % Hkv);
  SegTile t;
  if (!find_tile(cu, max_segs, N, kT, int32_t(b / Hkv), t)) return;
  const int32_t rep = H / Hkv;
  const int r = threadIdx.x / 8, c = threadIdx.x % 8;
  const int64_t row = int64_t(t.start) + r;

  stage<T, D>(sk, k, t.start, t.e, Hkv, hk);
  stage<T, D>(sv, v, t.start, t.e, Hkv, hk);
  float ak[D / 8] = {}, av[D / 8] = {};
  for (int32_t h = hk * rep; h < (hk + 1) * rep; ++h) {
    for (int64_t s0 = t.start; s0 < t.e; s0 += kT) {
      __syncthreads();
      stage<T, D>(sq, q, s0, t.e, H, h);
      stage<T, D>(sdo, dout, s0, t.e, H, h);
      if (threadIdx.x < kT) {
        const int64_t s = s0 + threadIdx.x;
        sl[threadIdx.x] = s < t.e ? lse[int64_t(h) * N + s] : INFINITY;
        sdl[threadIdx.x] = s < t.e ? delta[int64_t(h) * N + s] : 0.f;
      }
      __syncthreads();
      float x[kT / 8] = {}, y[kT / 8] = {};
      for (int d = 0; d < D; ++d) {
#pragma unroll
        for (int j = 0; j < kT / 8; ++j) {
          x[j] += sk[r][d] * sq[c + 8 * j][d];
          y[j] += sv[r][d] * sdo[c + 8 * j][d];
        }
      }
#pragma unroll
      for (int j = 0; j < kT / 8; ++j) {
        const int s = c + 8 * j;
        const float p = expf(x[j] * scale - sl[s]);
        sp[r][s] = p;
        sd[r][s] = p * (y[j] - sdl[s]);
      }
      __syncthreads();
      // only the queries that attend to the row
      const int first = row > s0 ? int(row - s0) : 0;
      const int end = t.e - s0 < kT ? int(t.e - s0) : kT;
      for (int s = first; s < end; ++s) {
        const float p = sp[r][s], d = sd[r][s];
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          av[j] += p * sdo[s][c + 8 * j];
          ak[j] += d * sq[s][c + 8 * j];
        }
      }
    }
  }
  if (row >= t.e) return;
#pragma unroll
  for (int j = 0; j < D / 8; ++j) {
    const int64_t i = (row * Hkv + hk) * D + c + 8 * j;
    dk[i] = from_f32<T>(ak[j] * scale);
    dv[i] = from_f32<T>(av[j]);
  }
}

template <typename T, int D>
hipError_t fwd(const AttnArgs& a, hipStream_t stream) {
  const int64_t slots = tile_slots(a.N, a.max_segs, kT), grid = slots * a.H + kTail;
  attn_simple_fwd<T, D><<<dim3(uint32_t(grid)), dim3(kThreads), 0, stream>>>(
      static_cast<const T*>(a.q), static_cast<const T*>(a.k), static_cast<const T*>(a.v), a.cu, a.max_segs,
      a.N, a.H, a.Hkv, a.scale, static_cast<T*>(a.o), a.lse, a.flags, slots);
  return hipGetLastError();
}

template <typename T, int D>
hipError_t bwd(const AttnArgs& a, const AttnGradArgs& g, hipStream_t stream) {
  const T *q = static_cast<const T*>(a.q), *k = static_cast<const T*>(a.k), *v = static_cast<const T*>(a.v);
  const T* dout = static_cast<const T*>(g.dout);
  const int64_t slots = tile_slots(a.N, a.max_segs, kT), rows = kThreads / 8;
  attn_delta<T, D><<<dim3(uint32_t((a.N * a.H + rows - 1) / rows)), dim3(kThreads), 0, stream>>>(
      static_cast<const T*>(a.o), dout, g.stats, a.N, a.H);
  attn_simple_dq<T, D><<<dim3(uint32_t(slots * a.H + kTail)), dim3(kThreads), 0, stream>>>(
      q, k, v, dout, a.lse, g.stats, a.cu, a.max_segs, a.N, a.H, a.Hkv, a.scale, static_cast<T*>(g.dq),
      a.flags, slots);
  attn_simple_dkv<T, D><<<dim3(uint32_t(slots * a.Hkv + kTail)), dim3(kThreads), 0, stream>>>(
      q, k, v, dout, a.lse, g.stats, a.cu, a.max_segs, a.N, a.H, a.Hkv, a.scale, static_cast<T*>(g.dk),
      static_cast<T*>(g.dv), slots);
  return hipGetLastError();
}

}  // namespace

int64_t attn_simple_grid(int64_t N, int32_t max_segs, int32_t H) {
  const int64_t tiles = tile_slots(N, max_segs, kT) * H + kTail, delta = (N * H + 31) / 32;
  return tiles > delta ? tiles : delta;
}

hipError_t launch_attn_simple(const AttnArgs& a, int32_t dtype, hipStream_t stream) {
  if (dtype == 1) {
    if (a.D == 32) return fwd<float, 32>(a, stream);
    if (a.D == 64) return fwd<float, 64>(a, stream);
    return fwd<float, 128>(a, stream);
  }
  if (a.D == 32) return fwd<bf16, 32>(a, stream);
  if (a.D == 64) return fwd<bf16, 64>(a, stream);
  return fwd<bf16, 128>(a, stream);
}

hipError_t launch_attn_simple_backward(const AttnArgs& a, const AttnGradArgs& g, int32_t dtype,
                                       hipStream_t stream) {
  if (dtype == 1) {
    if (a.D == 32) return bwd<float, 32>(a, g, stream);
    if (a.D == 64) return bwd<float, 64>(a, g, stream);
    return bwd<float, 128>(a, g, stream);
  }
  if (a.D == 32) return bwd<bf16, 32>(a, g, stream);
  if (a.D == 64) return bwd<bf16, 64>(a, g, stream);
  return bwd<bf16, 128>(a, g, stream);
}

}  // namespace pkv
