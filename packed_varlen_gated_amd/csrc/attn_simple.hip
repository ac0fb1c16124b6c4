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
// fp32, the next tile's values on their way in registers. Thread (r, c) =
// (tid / 8, tid % 8) holds row r's scores of columns c + 8 j and its channels
// 4 (c + 8 j) .. + 3; LDS is read 16 bytes at a time. The softmax runs in one pass
// with a running maximum and sum. These shapes serve fp32 batches that models are
// debugged on, where latency counts; the MFMA kernels serve bf16 at D = 64 and 128.

#include "segments.h"

namespace pkv {
namespace {

constexpr int kT = 32;        // tokens per tile, both sides
constexpr int kThreads = 256;
constexpr int kTail = 64;     // work-groups that zero the rows no segment has

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <int D>
struct alignas(16) Tile {
  float x[kT][D + 4];  // (rows 16 bytes apart modulo the banks)
  __device__ __forceinline__ f32x4 at(int r, int d) const { return *reinterpret_cast<const f32x4*>(&x[r][d]); }
};
struct alignas(16) Weights {
  float x[kT][kT + 4];
  __device__ __forceinline__ f32x4 at(int r, int s) const { return *reinterpret_cast<const f32x4*>(&x[r][s]); }
};

__device__ __forceinline__ f32x4 load4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ f32x4 load4(const bf16* p) {
  typedef bf16 b16x4 __attribute__((ext_vector_type(4)));
  const b16x4 x = *reinterpret_cast<const b16x4*>(p);
  return f32x4{to_f32(x[0]), to_f32(x[1]), to_f32(x[2]), to_f32(x[3])};
}
__device__ __forceinline__ void store4(float* p, f32x4 x) { *reinterpret_cast<f32x4*>(p) = x; }
__device__ __forceinline__ void store4(bf16* p, f32x4 x) {
  typedef bf16 b16x4 __attribute__((ext_vector_type(4)));
  *reinterpret_cast<b16x4*>(p) = b16x4{from_f32<bf16>(x[0]), from_f32<bf16>(x[1]), from_f32<bf16>(x[2]), from_f32<bf16>(x[3])};
}

// The thread's part of 32 rows of a [N, H, D] tensor from `row` on, zero past `end`.
template <typename T, int D>
struct Stage {
  f32x4 v[D / 32];
  __device__ __forceinline__ void load(const T* __restrict__ src, int64_t row, int64_t end, int32_t H, int32_t h) {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int at = (i * kThreads + threadIdx.x) * 4, r = at / D, d = at % D;
      v[i] = row + r < end ? load4(src + ((row + r) * H + h) * D + d) : f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }
  __device__ __forceinline__ void put(Tile<D>& t) const {
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int at = (i * kThreads + threadIdx.x) * 4;
      *reinterpret_cast<f32x4*>(&t.x[at / D][at % D]) = v[i];
    }
  }
};

// Products of row r of a with rows c + 8 j of b, added to x.
template <int D>
__device__ __forceinline__ void dots(float (&x)[kT / 8], const Tile<D>& a, int r, const Tile<D>& b, int c) {
#pragma unroll 8
  for (int d = 0; d < D; d += 4) {
    const f32x4 y = a.at(r, d);
#pragma unroll
    for (int j = 0; j < kT / 8; ++j) {
      const f32x4 z = b.at(c + 8 * j, d);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[j] += y[e] * z[e];
    }
  }
}

// acc += sum over s in [first, end) of w[r][s] t[s][the thread's channels]; the
// rows of t outside take no part, whatever they hold.
template <int D>
__device__ __forceinline__ void combine(f32x4 (&acc)[D / 32], const Weights& w, int r, const Tile<D>& t, int c, int first,
                                        int end) {
#pragma unroll 2
  for (int s4 = first & ~3; s4 < end; s4 += 4) {
    const f32x4 p = w.at(r, s4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (s4 + e < first || s4 + e >= end) continue;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) acc[j] += p[e] * t.at(s4 + e, 4 * (c + 8 * j));
    }
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
  __shared__ Tile<D> sq, sk, sv;
  __shared__ Weights sp;
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

  Stage<T, D> gq, gk, gv;
  gq.load(q, t.start, t.e, H, h);
  gk.load(k, t.a, t.e, Hkv, hk);
  gv.load(v, t.a, t.e, Hkv, hk);
  gq.put(sq);
  float m = -INFINITY, l = 0.f;
  f32x4 acc[D / 32] = {};
  for (int64_t s0 = t.a; s0 < t.start + kT && s0 < t.e; s0 += kT) {
    __syncthreads();
    gk.put(sk);
    gv.put(sv);
    __syncthreads();
    gk.load(k, s0 + kT, t.e, Hkv, hk);
    gv.load(v, s0 + kT, t.e, Hkv, hk);
    float x[kT / 8] = {};
    dots<D>(x, sq, r, sk, c);
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
      sp.x[r][c + 8 * j] = p;
    }
    l = l * f + row_sum(lt);
    m = mt;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) acc[j] *= f;
    // (a row's weights are written and read by the same 8 lanes of a wave)
    asm volatile("" ::: "memory");
    combine<D>(acc, sp, r, sv, c, 0, row - s0 < kT ? int(row - s0) + 1 : kT);
  }
  if (row >= t.e) return;
  const float inv = 1.f / l;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) store4(o + (row * H + h) * D + 4 * (c + 8 * j), acc[j] * inv);
  if (lse != nullptr && c == 0) lse[int64_t(h) * N + row] = m + logf(l);
}

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_simple_dq(
    const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, const T* __restrict__ o,
    const T* __restrict__ dout, const float* __restrict__ lse, float* __restrict__ delta,
    const int32_t* __restrict__ cu, int32_t max_segs, int64_t N, int32_t H, int32_t Hkv, float scale,
    T* __restrict__ dq,
    int32_t* __restrict__ flags, int64_t slots) {
  __shared__ Tile<D> sq, sdo, sk, sv;
  __shared__ Weights sp;
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

  Stage<T, D> gq, gdo, gk, gv;
  gq.load(q, t.start, t.e, H, h);
  gdo.load(dout, t.start, t.e, H, h);
  gk.load(k, t.a, t.e, Hkv, hk);
  gv.load(v, t.a, t.e, Hkv, hk);
  const float ls = real ? lse[int64_t(h) * N + row] : INFINITY;
  // delta_t, which the keys pass reads
  float dl = 0.f;
  if (real)
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      const int64_t at = (row * H + h) * D + 4 * (c + 8 * j);
      const f32x4 x = load4(o + at), y = load4(dout + at);
      dl += x[0] * y[0] + x[1] * y[1] + x[2] * y[2] + x[3] * y[3];
    }
  dl = row_sum(dl);
  if (real && c == 0) delta[int64_t(h) * N + row] = dl;
  gq.put(sq);
  gdo.put(sdo);
  f32x4 acc[D / 32] = {};
  for (int64_t s0 = t.a; s0 < t.start + kT && s0 < t.e; s0 += kT) {
    __syncthreads();
    gk.put(sk);
    gv.put(sv);
    __syncthreads();
    gk.load(k, s0 + kT, t.e, Hkv, hk);
    gv.load(v, s0 + kT, t.e, Hkv, hk);
    float x[kT / 8] = {}, y[kT / 8] = {};
    dots<D>(x, sq, r, sk, c);
    dots<D>(y, sdo, r, sv, c);
#pragma unroll
    for (int j = 0; j < kT / 8; ++j)
      sp.x[r][c + 8 * j] = s0 + c + 8 * j <= row ? expf(x[j] * scale - ls) * (y[j] - dl) : 0.f;
    // (a row's weights are written and read by the same 8 lanes of a wave)
    asm volatile("" ::: "memory");
    combine<D>(acc, sp, r, sk, c, 0, row - s0 < kT ? int(row - s0) + 1 : kT);
  }
  if (!real) return;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) store4(dq + (row * H + h) * D + 4 * (c + 8 * j), acc[j] * scale);
}

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_simple_dkv(
    const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, const T* __restrict__ dout,
    const float* __restrict__ lse, const float* __restrict__ delta, const int32_t* __restrict__ cu,
    int32_t max_segs, int64_t N, int32_t H, int32_t Hkv, float scale, T* __restrict__ dk,
    T* __restrict__ dv, int64_t slots) {
  __shared__ Tile<D> sq, sdo, sk, sv;
  __shared__ Weights sp, sd;  // of row r (a key) and column s (a query)
  __shared__ float sl[kT], sdl[kT];
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

  Stage<T, D> gq, gdo;
  float gs = 0.f;
  auto load = [&](int32_t h, int64_t s0) {
    gq.load(q, s0, t.e, H, h);
    gdo.load(dout, s0, t.e, H, h);
    if (threadIdx.x < 2 * kT) {
      const int64_t s = s0 + threadIdx.x % kT;
      const bool first = threadIdx.x < kT;
      gs = s < t.e ? (first ? lse : delta)[int64_t(h) * N + s] : (first ? INFINITY : 0.f);
    }
  };
  {
    Stage<T, D> gk, gv;
    gk.load(k, t.start, t.e, Hkv, hk);
    gv.load(v, t.start, t.e, Hkv, hk);
    load(hk * rep, t.start);
    gk.put(sk);
    gv.put(sv);
  }
  f32x4 ak[D / 32] = {}, av[D / 32] = {};
  for (int32_t h = hk * rep; h < (hk + 1) * rep; ++h) {
    for (int64_t s0 = t.start; s0 < t.e; s0 += kT) {
      __syncthreads();
      gq.put(sq);
      gdo.put(sdo);
      if (threadIdx.x < 2 * kT) (threadIdx.x < kT ? sl : sdl)[threadIdx.x % kT] = gs;
      __syncthreads();
      if (s0 + kT < t.e)
        load(h, s0 + kT);
      else if (h + 1 < (hk + 1) * rep)
        load(h + 1, t.start);
      float x[kT / 8] = {}, y[kT / 8] = {};
      dots<D>(x, sk, r, sq, c);
      dots<D>(y, sv, r, sdo, c);
#pragma unroll
      for (int j = 0; j < kT / 8; ++j) {
        const int s = c + 8 * j;
        const float p = expf(x[j] * scale - sl[s]);
        sp.x[r][s] = p;
        sd.x[r][s] = p * (y[j] - sdl[s]);
      }
      // (a row's weights are written and read by the same 8 lanes of a wave)
      asm volatile("" ::: "memory");
      const int first = row > s0 ? int(row - s0) : 0, end = t.e - s0 < kT ? int(t.e - s0) : kT;
      combine<D>(av, sp, r, sdo, c, first, end);
      combine<D>(ak, sd, r, sq, c, first, end);
    }
  }
  if (row >= t.e) return;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) {
    const int64_t i = (row * Hkv + hk) * D + 4 * (c + 8 * j);
    store4(dk + i, ak[j] * scale);
    store4(dv + i, av[j]);
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
  const int64_t slots = tile_slots(a.N, a.max_segs, kT);
  attn_simple_dq<T, D><<<dim3(uint32_t(slots * a.H + kTail)), dim3(kThreads), 0, stream>>>(
      q, k, v, static_cast<const T*>(a.o), dout, a.lse, g.stats, a.cu, a.max_segs, a.N, a.H, a.Hkv, a.scale,
      static_cast<T*>(g.dq), a.flags, slots);
  attn_simple_dkv<T, D><<<dim3(uint32_t(slots * a.Hkv + kTail)), dim3(kThreads), 0, stream>>>(
      q, k, v, dout, a.lse, g.stats, a.cu, a.max_segs, a.N, a.H, a.Hkv, a.scale, static_cast<T*>(g.dk),
      static_cast<T*>(g.dv), slots);
  return hipGetLastError();
}

}  // namespace

int64_t attn_simple_grid(int64_t N, int32_t max_segs, int32_t H) {
  return tile_slots(N, max_segs, kT) * H + kTail;
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
