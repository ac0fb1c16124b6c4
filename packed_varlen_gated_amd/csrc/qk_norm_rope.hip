// RMS norm of every query and key head with the rotation by position, and its
// reverse pass.
//
//   r = 1 / sqrt(mean_d x_d^2 + eps),  u = w r x,
//   (y_a, y_b) = (u_a cos t - u_b sin t, u_a sin t + u_b cos t),  t = p f_i
// Reverse pass, with du the transposed rotation of dy and z = r x:
//   dx = r (w du - z mean(w du z)),  dw = sum over rows of du z
//
// D / 16 lanes share a head's row of one token: a lane holds the two 16-byte
// chunks (bf16) whose channels are each other's partners, so the rotation needs no
// exchange and the norm D / 32 steps of one. A wave takes one token: it forms
// the token's 8 angles per lane once and walks the heads 1024 / D rows at a time,
// the loads of several steps going out together.
//
// An angle is p f / 2 pi turns, formed in fp64 and reduced to half a turn before it
// is rounded to fp32: at position 10^6 an fp32 product is off by 0.03 rad.
//
// Bound by memory: nothing is read twice, and the arithmetic is a third of the
// vector units' time at the copy's rate.

#include "common.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kAhead = 4;  // row groups of a wave that are loaded together

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct Chunk {  // 8 channels
  float x[8];
};
__device__ __forceinline__ Chunk load_chunk(const float* p) {
  const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
  return {{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
}
__device__ __forceinline__ void store_chunk(float* p, const Chunk& c) {
  reinterpret_cast<f32x4*>(p)[0] = f32x4{c.x[0], c.x[1], c.x[2], c.x[3]};
  reinterpret_cast<f32x4*>(p)[1] = f32x4{c.x[4], c.x[5], c.x[6], c.x[7]};
}
__device__ __forceinline__ void store_chunk(bf16* p, const Chunk& c) {
  bf16x8 v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = static_cast<bf16>(c.x[i]);
  *reinterpret_cast<bf16x8*>(p) = v;
}
// A chunk as it lies in memory, until it is used.
template <typename T>
struct Raw;
template <>
struct Raw<bf16> {
  bf16x8 v;
  __device__ __forceinline__ void load(const bf16* p) { v = *reinterpret_cast<const bf16x8*>(p); }
  __device__ __forceinline__ Chunk get() const {
    Chunk c;
#pragma unroll
    for (int i = 0; i < 8; ++i) c.x[i] = to_f32(v[i]);
    return c;
  }
};
template <>
struct Raw<float> {
  Chunk v;
  __device__ __forceinline__ void load(const float* p) { v = load_chunk(p); }
  __device__ __forceinline__ Chunk get() const { return v; }
};

// What a lane holds of a row, and its angles.
template <int D, bool kInter>
struct Lane {
  static constexpr int LPR = D / 16;     // lanes of a row
  static constexpr int ROWS = 64 / LPR;  // rows of a step
  int row;                               // of a step
  int at0, at1;                          // first channels of the two chunks
  int pair;                              // first pair, or -1: not rotated
  float cs[8], sn[8];
  __device__ __forceinline__ Lane(int lane, int rot) {
    const int j = lane % LPR;
    row = lane / LPR;
    const bool turns = 16 * j < rot;
    pair = turns ? 8 * j : -1;
    const bool split = !kInter && turns;  // partners are rot / 2 apart
    at0 = split ? 8 * j : 16 * j;
    at1 = split ? 8 * j + rot / 2 : 16 * j + 8;
  }
  __device__ __forceinline__ void turn(const float* __restrict__ freq, int32_t p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      cs[i] = 1.f;
      sn[i] = 0.f;
      if (pair >= 0) {
        const double t = double(p) * (double(freq[pair + i]) * 0.15915494309189533577);
        sincospif(2.f * float(t - rint(t)), &sn[i], &cs[i]);
      }
    }
  }
  // The rotation by the angles (dir 1) or back (dir -1).
  template <int dir>
  __device__ __forceinline__ void rotate(Chunk& a, Chunk& b) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float& x = kInter ? (i < 4 ? a.x[2 * i] : b.x[2 * i - 8]) : a.x[i];
      float& y = kInter ? (i < 4 ? a.x[2 * i + 1] : b.x[2 * i - 7]) : b.x[i];
      const float s = dir * sn[i], u = x * cs[i] - y * s, v = x * s + y * cs[i];
      x = u;
      y = v;
    }
  }
  // The sum over the row's lanes.
  static __device__ __forceinline__ float sum(float x) {
#pragma unroll
    for (int m = 1; m < LPR; m *= 2) x += __shfl_xor(x, m, 64);
    return x;
  }
};

struct Weight {
  Chunk a, b;
  __device__ __forceinline__ void load(const float* w, int at0, int at1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a.x[i] = w == nullptr ? 1.f : w[at0 + i];
      b.x[i] = w == nullptr ? 1.f : w[at1 + i];
    }
  }
};

template <typename T, int D, bool kInter>
__device__ __forceinline__ float inv_rms(const Chunk& a, const Chunk& b, float eps) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += a.x[i] * a.x[i] + b.x[i] * b.x[i];
  return 1.f / sqrtf(Lane<D, kInter>::sum(s) * (1.f / D) + eps);
}

// Steps [g0, g1) of one tensor's heads at one token; x, y: the token's rows.
template <typename T, int D, bool kInter>
__device__ __forceinline__ void forward_rows(const Lane<D, kInter>& ln, const Weight& w, const T* __restrict__ x,
                                             T* __restrict__ y, int heads, int g0, int g1, float eps) {
  for (int g = g0; g < g1; g += kAhead) {
    Raw<T> ra[kAhead], rb[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int h = (g + u) * ln.ROWS + ln.row;
      if (g + u < g1 && h < heads) {
        ra[u].load(x + h * D + ln.at0);
        rb[u].load(x + h * D + ln.at1);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int h = (g + u) * ln.ROWS + ln.row;
      if (g + u >= g1) break;
      if (h >= heads) continue;
      Chunk a = ra[u].get(), b = rb[u].get();
      const float r = inv_rms<T, D, kInter>(a, b, eps);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a.x[i] *= r * w.a.x[i];
        b.x[i] *= r * w.b.x[i];
      }
      ln.template rotate<1>(a, b);
      store_chunk(y + h * D + ln.at0, a);
      store_chunk(y + h * D + ln.at1, b);
    }
  }
}

template <typename T, int D>
__device__ __forceinline__ void zero_rows(T* y, int heads, int g0, int g1, int lane) {
  constexpr int ROWS = 1024 / D;
  const Chunk z = {};
  const int end = (g1 * ROWS < heads ? g1 * ROWS : heads) * (D / 8);
  for (int i = g0 * ROWS * (D / 8) + lane; i < end; i += 64) store_chunk(y + i * 8, z);
}

// Unit u of the call: token u / split, part u % split of its steps.
template <typename T, int D, bool kInter>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(const NormRopeArgs x, int split) {
  using L = Lane<D, kInter>;
  const int lane = threadIdx.x & 63;
  const int64_t unit = int64_t(blockIdx.x) * kWaves + (threadIdx.x >> 6);
  const int64_t n = unit / split;
  if (n >= x.N) return;
  const int part = int(unit % split);
  const int gq = (x.Hq + L::ROWS - 1) / L::ROWS, gk = (x.Hkv + L::ROWS - 1) / L::ROWS;
  const int per = (gq + gk + split - 1) / split, g0 = part * per, g1 = g0 + per < gq + gk ? g0 + per : gq + gk;
  const int32_t p = x.positions == nullptr ? int32_t(n) : x.positions[n];
  const int q1 = g1 < gq ? g1 : gq, k0 = g0 > gq ? g0 - gq : 0, k1 = g1 - gq;
  const T *q = static_cast<const T*>(x.q) + n * x.q_stride, *k = static_cast<const T*>(x.k) + n * x.k_stride;
  T *qo = static_cast<T*>(x.q_out) + n * x.Hq * D, *ko = static_cast<T*>(x.k_out) + n * x.Hkv * D;
  if (p < 0) {
    if (g0 < q1) zero_rows<T, D>(qo, x.Hq, g0, q1, lane);
    if (k0 < k1) zero_rows<T, D>(ko, x.Hkv, k0, k1, lane);
    return;
  }
  L ln(lane, x.rot);
  ln.turn(x.inv_freq, p);
  Weight w;
  if (g0 < q1) {
    w.load(x.q_weight, ln.at0, ln.at1);
    forward_rows<T, D, kInter>(ln, w, q, qo, x.Hq, g0, q1, x.eps);
  }
  if (k0 < k1) {
    w.load(x.k_weight, ln.at0, ln.at1);
    forward_rows<T, D, kInter>(ln, w, k, ko, x.Hkv, k0, k1, x.eps);
  }
}

// All heads of one tensor at one token; the row's part of dw is added to `dw`.
template <typename T, int D, bool kInter>
__device__ __forceinline__ void backward_rows(const Lane<D, kInter>& ln, const Weight& w, Weight& dw,
                                              const T* __restrict__ x, const T* __restrict__ dy, T* __restrict__ dx,
                                              int heads, float eps) {
  constexpr int kU = 2;
  const int groups = (heads + ln.ROWS - 1) / ln.ROWS;
  for (int g = 0; g < groups; g += kU) {
    Raw<T> ra[kU], rb[kU], rc[kU], rd[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int h = (g + u) * ln.ROWS + ln.row;
      if (h < heads) {
        ra[u].load(x + h * D + ln.at0);
        rb[u].load(x + h * D + ln.at1);
        rc[u].load(dy + h * D + ln.at0);
        rd[u].load(dy + h * D + ln.at1);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int h = (g + u) * ln.ROWS + ln.row;
      if (h >= heads) continue;
      Chunk a = ra[u].get(), b = rb[u].get(), c = rc[u].get(), d = rd[u].get();
      const float r = inv_rms<T, D, kInter>(a, b, eps);
      ln.template rotate<-1>(c, d);
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a.x[i] *= r;  // z
        b.x[i] *= r;
        dw.a.x[i] += c.x[i] * a.x[i];
        dw.b.x[i] += d.x[i] * b.x[i];
        c.x[i] *= w.a.x[i];
        d.x[i] *= w.b.x[i];
        s += c.x[i] * a.x[i] + d.x[i] * b.x[i];
      }
      s = Lane<D, kInter>::sum(s) * (1.f / D);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        c.x[i] = r * (c.x[i] - a.x[i] * s);
        d.x[i] = r * (d.x[i] - b.x[i] * s);
      }
      store_chunk(dx + h * D + ln.at0, c);
      store_chunk(dx + h * D + ln.at1, d);
    }
  }
}

// The sum of `dw` over the wave's rows and the work-group's waves, to out[D].
template <int D, bool kInter>
__device__ __forceinline__ void join_weight(const Lane<D, kInter>& ln, Weight& dw, float (*lds)[D], float* out) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int m = Lane<D, kInter>::LPR; m < 64; m *= 2) {
      dw.a.x[i] += __shfl_xor(dw.a.x[i], m, 64);
      dw.b.x[i] += __shfl_xor(dw.b.x[i], m, 64);
    }
  if (ln.row == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      lds[threadIdx.x >> 6][ln.at0 + i] = dw.a.x[i];
      lds[threadIdx.x >> 6][ln.at1 + i] = dw.b.x[i];
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += kThreads) {
    float s = lds[0][d];
    for (int v = 1; v < kWaves; ++v) s += lds[v][d];
    out[d] = s;
  }
  __syncthreads();
}

// Work-group b takes every gridDim.x-th group of kWaves tokens, a wave one token at
// a time; partial: [gridDim.x, 2, D] sums of dw, or null.
template <typename T, int D, bool kInter>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_bwd_kernel(const NormRopeArgs x, const NormRopeGradArgs y,
                                                                    float* __restrict__ partial) {
  __shared__ float lds[kWaves][D];
  using L = Lane<D, kInter>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  L ln(lane, x.rot);
  Weight wq, wk, dwq = {}, dwk = {};
  wq.load(x.q_weight, ln.at0, ln.at1);
  wk.load(x.k_weight, ln.at0, ln.at1);
  for (int64_t n = int64_t(blockIdx.x) * kWaves + wave; n < x.N; n += int64_t(gridDim.x) * kWaves) {
    const int32_t p = x.positions == nullptr ? int32_t(n) : x.positions[n];
    const int64_t qd = n * x.Hq * D, kd = n * x.Hkv * D;
    T *dq = static_cast<T*>(y.dq) + qd, *dk = static_cast<T*>(y.dk) + kd;
    if (p < 0) {
      zero_rows<T, D>(dq, x.Hq, 0, x.Hq, lane);
      zero_rows<T, D>(dk, x.Hkv, 0, x.Hkv, lane);
      continue;
    }
    ln.turn(x.inv_freq, p);
    backward_rows<T, D, kInter>(ln, wq, dwq, static_cast<const T*>(x.q) + n * x.q_stride,
                                static_cast<const T*>(y.dq_out) + qd, dq, x.Hq, x.eps);
    backward_rows<T, D, kInter>(ln, wk, dwk, static_cast<const T*>(x.k) + n * x.k_stride,
                                static_cast<const T*>(y.dk_out) + kd, dk, x.Hkv, x.eps);
  }
  if (partial == nullptr) return;
  join_weight<D, kInter>(ln, dwq, lds, partial + int64_t(blockIdx.x) * 2 * D);
  join_weight<D, kInter>(ln, dwk, lds, partial + int64_t(blockIdx.x) * 2 * D + D);
}

// Column sums of partial [groups, 2 D]: 32 columns a work-group, 8 slices of rows,
// joined in order.
template <int D>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_dw_kernel(const float* __restrict__ partial, int groups,
                                                                   float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ float lds[8][32];
  const int c = threadIdx.x % 32, s = threadIdx.x / 32, col = blockIdx.x * 32 + c;
  float x = 0.f;
  for (int g = s; g < groups; g += 8) x += partial[int64_t(g) * 2 * D + col];
  lds[s][c] = x;
  __syncthreads();
  if (s != 0) return;
  for (int i = 1; i < 8; ++i) x += lds[i][c];
  float* out = col < D ? dwq : dwk;
  if (out != nullptr) out[col % D] = x;
}

// Work-groups of the reverse pass: four waves a SIMD, and their partial sums stay few.
int64_t bwd_groups(int64_t N) {
  const int64_t g = (N + kWaves - 1) / kWaves;
  return g < 1024 ? g : 1024;
}

template <typename T, int D, bool kInter>
hipError_t forward(const NormRopeArgs& x, hipStream_t stream) {
  constexpr int ROWS = Lane<D, kInter>::ROWS;
  const int64_t steps = (x.Hq + ROWS - 1) / ROWS + (x.Hkv + ROWS - 1) / ROWS;
  // A few tokens: a token's steps go to waves of their own.
  int64_t split = 8192 / x.N;
  split = split < 1 ? 1 : (split < steps ? split : steps);
  const int64_t groups = (x.N * split + kWaves - 1) / kWaves;
  qk_norm_rope_kernel<T, D, kInter><<<dim3(uint32_t(groups)), dim3(kThreads), 0, stream>>>(x, int(split));
  return hipGetLastError();
}

template <typename T, int D, bool kInter>
hipError_t backward(const NormRopeArgs& x, const NormRopeGradArgs& y, hipStream_t stream) {
  const int64_t groups = bwd_groups(x.N);
  float* partial = y.dq_weight != nullptr || y.dk_weight != nullptr ? y.partial : nullptr;
  qk_norm_rope_bwd_kernel<T, D, kInter><<<dim3(uint32_t(groups)), dim3(kThreads), 0, stream>>>(x, y, partial);
  if (partial != nullptr)
    qk_norm_rope_dw_kernel<D><<<dim3(2 * D / 32), dim3(kThreads), 0, stream>>>(partial, int(groups), y.dq_weight,
                                                                             y.dk_weight);
  return hipGetLastError();
}

// f<T, D, kInter> for the call's type, head dimension and pairing.
#define PKV_NORM_ROPE_DISPATCH(f, ...)                                                                      \
  (dtype == 0 ? (x.D == 32   ? (x.interleaved ? f<bf16, 32, true>(__VA_ARGS__) : f<bf16, 32, false>(__VA_ARGS__))  \
                 : x.D == 64 ? (x.interleaved ? f<bf16, 64, true>(__VA_ARGS__) : f<bf16, 64, false>(__VA_ARGS__))  \
                             : (x.interleaved ? f<bf16, 128, true>(__VA_ARGS__) : f<bf16, 128, false>(__VA_ARGS__))) \
              : (x.D == 32   ? (x.interleaved ? f<float, 32, true>(__VA_ARGS__) : f<float, 32, false>(__VA_ARGS__)) \
                 : x.D == 64 ? (x.interleaved ? f<float, 64, true>(__VA_ARGS__) : f<float, 64, false>(__VA_ARGS__)) \
                             : (x.interleaved ? f<float, 128, true>(__VA_ARGS__) : f<float, 128, false>(__VA_ARGS__))))

}  // namespace

size_t norm_rope_workspace_bytes(int64_t N, int32_t D) { return size_t(bwd_groups(N)) * 2 * D * 4; }

hipError_t launch_norm_rope(const NormRopeArgs& x, int32_t dtype, hipStream_t stream) {
  return PKV_NORM_ROPE_DISPATCH(forward, x, stream);
}

hipError_t launch_norm_rope_backward(const NormRopeArgs& x, const NormRopeGradArgs& y, int32_t dtype,
                                     hipStream_t stream) {
  return PKV_NORM_ROPE_DISPATCH(backward, x, y, stream);
}

}  // namespace pkv
