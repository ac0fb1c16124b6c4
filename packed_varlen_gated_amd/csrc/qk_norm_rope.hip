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
// exchange and the norm log2(D / 16) steps of one. A wave takes one token: its lanes
// form an angle each, once, and it walks the heads 1024 / D rows at a time, the loads
// of several steps going out together, the first ones before the angles.
//
// An angle is p f / 2 pi turns, formed in fp64 and reduced to half a turn before it
// is rounded to fp32: at position 10^6 an fp32 product is off by 0.03 rad.
//
// Bound by memory where tokens are many: nothing is read twice. 65536 tokens of a fused
// projection, H 32, Hkv 8, D 128, all channels rotated: 253 us for 1.34 GB, 5.3 TB/s (a large
// copy 5.13), with vector instructions in 51 % of the cycles. 8192 tokens, H 16, Hkv 4, D 128,
// 64 channels rotated, forward and reverse pass: 61 us for 0.21 GB (41 at the copy's rate),
// three launches of 21, 29 and 4 us (the last sums the weights' gradients of the
// work-groups); vector instructions take 64 and 68 % of the first two: a token is two steps
// there, behind its position, fp64 product, sine and cosine and 16 exchanges. With the angles
// formed by every lane for itself and before the loads: 307 and 110 us.

#include "mfma.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
// Steps (1024 / D rows) of a wave that are loaded together, and in the reverse pass. Other
// waves hide most of a load. Forward, 1 / 2 / 4 steps, D 128 but where said:
//   bf16  65536 tokens, H 32, Hkv 8        254 / 258 / 254 us
//         8192, H 16, Hkv 4                23.7 / 24.8 / 24.9
//         16384, H 128, Hkv 8              223 / 222 / 220
//         16384, H 16, Hkv 16, D 64        27.5 / 29.6 / 30.3 (a token is one step)
//   fp32  32768, H 32, Hkv 8               259 / 256 / 249
//         16384, H 32, Hkv 8, D 64         71.5 / 69.1 / 72.6
//         2048, H 32, Hkv 8                17.0 / 17.8 / 17.6
// Reverse, 1 / 2 steps (2 do not fit the registers): bf16, 65536 tokens 432 / 1192, fp32,
// 32768 386 / 682.
template <typename T>
constexpr int kAhead = sizeof(T) == 2 ? 1 : 2;
template <typename T>
constexpr int kBack = 1;

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
  // The angles of position p: lane i of the wave forms that of pair i (there are at most
  // 64), and every lane fetches its 8.
  __device__ __forceinline__ void turn(const float* __restrict__ freq, int32_t p, int rot) {
    const int lane = threadIdx.x & 63;
    float c = 1.f, s = 0.f;
    if (2 * lane < rot) {
      const double t = double(p) * (double(freq[lane]) * 0.15915494309189533577);
      sincospif(2.f * float(t - rint(t)), &s, &c);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = __shfl(c, pair + i, 64), y = __shfl(s, pair + i, 64);
      cs[i] = pair < 0 ? 1.f : x;
      sn[i] = pair < 0 ? 0.f : y;
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

// kU steps of one tensor's heads at one token, from step g on. Rows past the last head
// are the last one again (a load under a condition costs registers), and not stored.
template <typename T, int D, bool kInter, int kU>
struct Batch {
  Raw<T> a[kU], b[kU];
  __device__ __forceinline__ void load(const Lane<D, kInter>& ln, const T* __restrict__ x, int heads, int g) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int i = (g + u) * ln.ROWS + ln.row, h = i < heads ? i : heads - 1;
      a[u].load(x + h * D + ln.at0);
      b[u].load(x + h * D + ln.at1);
    }
  }
};

// y of a batch's rows.
template <typename T, int D, bool kInter, int kU>
__device__ __forceinline__ void forward_batch(const Lane<D, kInter>& ln, const Weight& w,
                                              const Batch<T, D, kInter, kU>& x, T* __restrict__ y, int heads, int g,
                                              int g1, float eps) {
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int h = (g + u) * ln.ROWS + ln.row;
    if (g + u >= g1) break;
    Chunk a = x.a[u].get(), b = x.b[u].get();
    const float r = inv_rms<T, D, kInter>(a, b, eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a.x[i] *= r * w.a.x[i];
      b.x[i] *= r * w.b.x[i];
    }
    ln.template rotate<1>(a, b);
    if (h < heads) {
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
  // the first rows' loads go out before the position is used
  L ln(lane, x.rot);
  Batch<T, D, kInter, kAhead<T>> bq;
  Batch<T, D, kInter, kBack<T>> bk;
  if (g0 < q1) bq.load(ln, q, x.Hq, g0);
  if (k0 < k1) bk.load(ln, k, x.Hkv, k0);
  Weight w;
  w.load(g0 < q1 ? x.q_weight : x.k_weight, ln.at0, ln.at1);
  if (p < 0) {
    if (g0 < q1) zero_rows<T, D>(qo, x.Hq, g0, q1, lane);
    if (k0 < k1) zero_rows<T, D>(ko, x.Hkv, k0, k1, lane);
    return;
  }
  ln.turn(x.inv_freq, p, x.rot);
  if (g0 < q1) {
    for (int g = g0;;) {
      forward_batch<T, D, kInter, kAhead<T>>(ln, w, bq, qo, x.Hq, g, q1, x.eps);
      if ((g += kAhead<T>) >= q1) break;
      bq.load(ln, q, x.Hq, g);
    }
  }
  if (k0 < k1) {
    if (g0 < q1) w.load(x.k_weight, ln.at0, ln.at1);
    for (int g = k0;;) {
      forward_batch<T, D, kInter, kBack<T>>(ln, w, bk, ko, x.Hkv, g, k1, x.eps);
      if ((g += kBack<T>) >= k1) break;
      bk.load(ln, k, x.Hkv, g);
    }
  }
}

// dx of a batch's rows; their part of dw is added to `dw`.
template <typename T, int D, bool kInter, int kU>
__device__ __forceinline__ void backward_batch(const Lane<D, kInter>& ln, const float* w, Weight& dw,
                                               const Batch<T, D, kInter, kU>& x, const Batch<T, D, kInter, kU>& dy,
                                               T* __restrict__ dx, int heads, int g, float eps) {
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int h = (g + u) * ln.ROWS + ln.row;
    Chunk a = x.a[u].get(), b = x.b[u].get(), c = dy.a[u].get(), d = dy.b[u].get();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c.x[i] = h < heads ? c.x[i] : 0.f;
      d.x[i] = h < heads ? d.x[i] : 0.f;
    }
    const float r = inv_rms<T, D, kInter>(a, b, eps);
    ln.template rotate<-1>(c, d);
    const Chunk wa = load_chunk(w + fresh(ln.at0)), wb = load_chunk(w + fresh(ln.at1));
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a.x[i] *= r;  // z
      b.x[i] *= r;
      dw.a.x[i] += c.x[i] * a.x[i];
      dw.b.x[i] += d.x[i] * b.x[i];
      c.x[i] *= wa.x[i];
      d.x[i] *= wb.x[i];
      s += c.x[i] * a.x[i] + d.x[i] * b.x[i];
    }
    s = Lane<D, kInter>::sum(s) * (1.f / D);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c.x[i] = r * (c.x[i] - a.x[i] * s);
      d.x[i] = r * (d.x[i] - b.x[i] * s);
    }
    if (h < heads) {
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

// How the reverse pass's work-groups and their partial sums are shared out: by the steps
// of a token, at most one wave a token, four waves a SIMD in all.
struct Split {
  int q, k;
  Split(const NormRopeArgs& x) {
    const int64_t rows = 1024 / x.D, sq = (x.Hq + rows - 1) / rows, sk = (x.Hkv + rows - 1) / rows;
    const int64_t most = (x.N + kWaves - 1) / kWaves, k0 = kGroups * sk / (sq + sk);
    const int64_t k1 = k0 < 1 ? 1 : k0;
    k = int(k1 < most ? k1 : most);
    q = int(kGroups - k1 < most ? kGroups - k1 : most);
  }
  static constexpr int64_t kGroups = 1024;
};

// Work-groups [0, groups_q) have q, the others k: a tensor's work-group i takes every
// n-th group of kWaves tokens of its n, a wave one token at a time. partial: D sums of dw
// for each work-group, or null.
template <typename T, int D, bool kInter>
__global__ __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 3) void qk_norm_rope_bwd_kernel(
    const NormRopeArgs x, const NormRopeGradArgs y, float* __restrict__ partial, int groups_q) {
  __shared__ float lds[kWaves][D];
  __shared__ __attribute__((aligned(16))) float weight[D];  // (registers are for the sums)
  using L = Lane<D, kInter>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool isq = int(blockIdx.x) < groups_q;
  const int group = isq ? blockIdx.x : blockIdx.x - groups_q, groups = isq ? groups_q : gridDim.x - groups_q;
  const int heads = isq ? x.Hq : x.Hkv, steps = (heads + L::ROWS - 1) / L::ROWS;
  const int64_t stride = isq ? x.q_stride : x.k_stride, dense = int64_t(heads) * D;
  const T *xs = static_cast<const T*>(isq ? x.q : x.k), *dys = static_cast<const T*>(isq ? y.dq_out : y.dk_out);
  T* dxs = static_cast<T*>(isq ? y.dq : y.dk);
  const float* w = isq ? x.q_weight : x.k_weight;
  for (int d = threadIdx.x; d < D; d += kThreads) weight[d] = w == nullptr ? 1.f : w[d];
  __syncthreads();
  L ln(lane, x.rot);
  Weight dw = {};
  for (int64_t n = int64_t(group) * kWaves + wave; n < x.N; n += int64_t(groups) * kWaves) {
    const int32_t p = x.positions == nullptr ? int32_t(n) : x.positions[n];
    // the first rows' loads go out before the position is used
    Batch<T, D, kInter, kBack<T>> bx, by;
    bx.load(ln, xs + n * stride, heads, 0);
    by.load(ln, dys + n * dense, heads, 0);
    if (p < 0) {
      zero_rows<T, D>(dxs + n * dense, heads, 0, steps, lane);
      continue;
    }
    ln.turn(x.inv_freq, p, x.rot);
    for (int g = 0;;) {
      backward_batch<T, D, kInter, kBack<T>>(ln, weight, dw, bx, by, dxs + n * dense, heads, g, x.eps);
      if ((g += kBack<T>) >= steps) break;
      bx.load(ln, xs + n * stride, heads, g);
      by.load(ln, dys + n * dense, heads, g);
    }
  }
  if (partial != nullptr) join_weight<D, kInter>(ln, dw, lds, partial + int64_t(blockIdx.x) * D);
}

// Column sums of the partial sums [groups_q + groups_k, D]: 4 columns of one tensor a
// work-group, every 256th row a thread, joined in order.
template <int D>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_dw_kernel(const float* __restrict__ partial, int groups_q,
                                                                   int groups_k, float* __restrict__ dwq,
                                                                   float* __restrict__ dwk) {
  __shared__ f32x4 lds[kThreads];
  const bool isq = blockIdx.x < D / 4;
  const int col = blockIdx.x % (D / 4) * 4, end = isq ? groups_q : groups_q + groups_k;
  f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int g = (isq ? 0 : groups_q) + threadIdx.x; g < end; g += kThreads)
    x += *reinterpret_cast<const f32x4*>(partial + int64_t(g) * D + col);
  lds[threadIdx.x] = x;
  for (int n = kThreads / 2; n > 0; n /= 2) {
    __syncthreads();
    if (int(threadIdx.x) < n) lds[threadIdx.x] += lds[threadIdx.x + n];
  }
  float* out = isq ? dwq : dwk;
  if (threadIdx.x == 0 && out != nullptr) {
#pragma unroll
    for (int e = 0; e < 4; ++e) out[col + e] = lds[0][e];
  }
}

template <typename T, int D, bool kInter>
hipError_t forward(const NormRopeArgs& x, hipStream_t stream) {
  constexpr int ROWS = Lane<D, kInter>::ROWS;
  const int64_t steps = (x.Hq + ROWS - 1) / ROWS + (x.Hkv + ROWS - 1) / ROWS;
  // A few tokens: a token's steps go to waves of their own, up to 2048 waves in all; with
  // more, forming a token's angles again costs what it saves. bf16, D 128, H 32, Hkv 8 (5
  // steps), no split / up to 1024, 2048, 4096, 8192 waves:
  //   1 token                     5.3 / -, 4.0, 4.0, 4.0 us
  //   256 tokens                  7.4 / 4.9, 5.4, 5.4, 5.5
  //   768                            - / 8.3, 7.6, 8.0, 8.6
  //   1024                        8.5 / 8.7, 8.0, 9.0, 10.1
  //   1500                       10.8 / 10.8, 10.8, 9.8, 13.8
  //   2048                       12.3 / 12.3, 12.3, 12.3, 15.2
  //   4096                       18.4 / 18.4, 18.4, 18.4, 21.3
  // H 128, Hkv 8 (17 steps): 256 tokens 7.5, 7.6, 9.9, 9.9; 1024 19.1, 16.0, 15.8, 19.1.
  int64_t split = 2048 / x.N;
  split = split < 1 ? 1 : (split < steps ? split : steps);
  const int64_t groups = (x.N * split + kWaves - 1) / kWaves;
  qk_norm_rope_kernel<T, D, kInter><<<dim3(uint32_t(groups)), dim3(kThreads), 0, stream>>>(x, int(split));
  return hipGetLastError();
}

template <typename T, int D, bool kInter>
hipError_t backward(const NormRopeArgs& x, const NormRopeGradArgs& y, hipStream_t stream) {
  const Split g(x);
  float* partial = y.dq_weight != nullptr || y.dk_weight != nullptr ? y.partial : nullptr;
  qk_norm_rope_bwd_kernel<T, D, kInter><<<dim3(g.q + g.k), dim3(kThreads), 0, stream>>>(x, y, partial, g.q);
  if (partial != nullptr)
    qk_norm_rope_dw_kernel<D><<<dim3(2 * D / 4), dim3(kThreads), 0, stream>>>(partial, g.q, g.k, y.dq_weight,
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

size_t norm_rope_workspace_bytes(int64_t N, int32_t D) {
  const int64_t most = 2 * ((N + kWaves - 1) / kWaves);
  return size_t(most < Split::kGroups ? most : Split::kGroups) * D * 4;
}

hipError_t launch_norm_rope(const NormRopeArgs& x, int32_t dtype, hipStream_t stream) {
  return PKV_NORM_ROPE_DISPATCH(forward, x, stream);
}

hipError_t launch_norm_rope_backward(const NormRopeArgs& x, const NormRopeGradArgs& y, int32_t dtype,
                                     hipStream_t stream) {
  return PKV_NORM_ROPE_DISPATCH(backward, x, y, stream);
}

}  // namespace pkv
