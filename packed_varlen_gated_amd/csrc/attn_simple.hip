// Packed causal softmax attention with grouped heads, and its reverse pass, in
// fp32 on the matrix cores: fp32 tensors, and bf16 tensors at D = 32.
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
// A work-group takes 32 rows (queries, or keys in the dk/dv pass) of one head. Its
// four waves take the tiles of 32 of the other side in turn, each in LDS of its
// own (no barrier inside a walk), and their sums are joined at the end, the
// softmax's by their maxima: these shapes serve the small fp32 batches that models
// are debugged on, where the length of a chain counts and not the rate.
//
// v_mfma_f32_32x32x2_f32: lane l holds row (or column) l % 32 and contraction slot
// l / 32 of an operand, and the result's column l % 32, rows
// 8 (i / 4) + 4 (l / 32) + i % 4. Over channels, step (p, e) pairs channels 8 p + e
// and 8 p + 4 + e: a lane reads its operand 16 bytes at a time. Over rows of a
// tile, step i pairs the rows of result register i of the two half-waves: a
// product's result is the next one's operand as it stands.
//
// 512 tokens in documents of about 56, H 4, Hkv 2, D 32, fp32, forward and reverse:
// 30 us, three dependent launches of 6.5, 7.6 and 14.2 us (one wave per 32 rows with
// scalar products: 73 us). One segment of 4096 tokens, forward / reverse: H 4, Hkv 2,
// D 64, fp32 165 / 639 us; H 16, Hkv 4, D 128, fp32 1.02 / 2.83 ms (67 and 61 TFLOP/s
// of causal products); D 32, bf16 0.31 / 1.16 ms.

#include "segments.h"

namespace pkv {
namespace {

constexpr int kT = 32;        // tokens per tile, both sides
constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr float kFinite = 3.4028234663852886e38f;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int D>
struct alignas(16) Tile {  // of one wave
  float x[kT][D + 4];      // (rows 4 banks apart)
  __device__ __forceinline__ f32x4 at(int r, int d) const { return *reinterpret_cast<const f32x4*>(&x[r][d]); }
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

// The wave's LDS accesses are in order; nothing is moved across.
__device__ __forceinline__ void wave_fence() { asm volatile("" ::: "memory"); }

__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32, 64); }
__device__ __forceinline__ int row_of(int i, int half) { return 8 * (i / 4) + 4 * half + i % 4; }

// 32 rows of a [N, H, D] tensor from `row` on into a wave's tile, zero past `end`;
// whether the lane's values are all finite.
template <typename T, int D>
__device__ __forceinline__ bool fill(Tile<D>& t, const T* __restrict__ src, int64_t row, int64_t end, int32_t H, int32_t h,
                                     int lane) {
  f32x4 v[D / 8];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    const int at = (i * 64 + lane) * 4, r = at / D, d = at % D;
    v[i] = row + r < end ? load4(src + ((row + r) * H + h) * D + d) : f32x4{0.f, 0.f, 0.f, 0.f};
  }
  bool ok = true;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    const int at = (i * 64 + lane) * 4;
    *reinterpret_cast<f32x4*>(&t.x[at / D][at % D]) = v[i];
#pragma unroll
    for (int e = 0; e < 4; ++e) ok &= fabsf(v[i][e]) <= kFinite;
  }
  return ok;
}

// The lane's part of row `row` (zero if not real) as an operand.
template <typename T, int D>
__device__ __forceinline__ void load_row(f32x4 (&f)[D / 8], const T* __restrict__ src, int64_t row, bool real, int32_t H,
                                         int32_t h, int half) {
#pragma unroll
  for (int p = 0; p < D / 8; ++p)
    f[p] = real ? load4(src + (row * H + h) * D + 8 * p + 4 * half) : f32x4{0.f, 0.f, 0.f, 0.f};
}

// Products of the tile's rows with the operand f.
template <int D>
__device__ __forceinline__ f32x16 over_channels(const Tile<D>& t, const f32x4 (&f)[D / 8], int col, int half) {
  f32x16 x = {};
#pragma unroll
  for (int p = 0; p < D / 8; ++p) {
    const f32x4 a = t.at(col, 8 * p + 4 * half);
#pragma unroll
    for (int e = 0; e < 4; ++e) x = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], f[p][e], x, 0, 0, 0);
  }
  return x;
}

// acc[channel][column of w] += sum over the tile's rows of t[row][channel] w[row].
template <int D>
__device__ __forceinline__ void over_rows(f32x16 (&acc)[D / 32], const Tile<D>& t, const f32x16& w, int col, int half) {
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
      acc[j] = __builtin_amdgcn_mfma_f32_32x32x2f32(t.x[row_of(i, half)][32 * j + col], w[i], acc[j], 0, 0, 0);
}

// A wave's sums into its tile, a row per column of the sums.
template <int D>
__device__ __forceinline__ void put_sums(Tile<D>& t, const f32x16 (&acc)[D / 32], int col, int half) {
#pragma unroll
  for (int j = 0; j < D / 32; ++j)
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *reinterpret_cast<f32x4*>(&t.x[col][32 * j + row_of(i, half)]) =
          f32x4{acc[j][i], acc[j][i + 1], acc[j][i + 2], acc[j][i + 3]};
}

// The sum of the waves' tiles (tile 2 w of wave w) times f, rows [0, rows), to out.
template <typename T, int D>
__device__ __forceinline__ void store_sums(const Tile<D>* t, float f, T* out, int64_t stride, int32_t rows) {
  for (int i = threadIdx.x; i < kT * D / 4; i += kThreads) {
    const int r = i / (D / 4), d = i % (D / 4) * 4;
    if (r >= rows) continue;
    f32x4 x = t[0].at(r, d);
#pragma unroll
    for (int w = 1; w < kWaves; ++w) x += t[2 * w].at(r, d);
    store4(out + r * stride + d, x * f);
  }
}

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_simple_fwd(
    const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
    const int32_t* __restrict__ cu, int32_t max_segs, int64_t N, int32_t H, int32_t Hkv, float scale,
    T* __restrict__ o, float* __restrict__ lse, int32_t* __restrict__ flags, int64_t slots) {
  __shared__ Tile<D> tiles[2 * kWaves];
  __shared__ float sm[kWaves][kT], sl[kWaves][kT];
  const int64_t b = blockIdx.x;
  if (b >= slots * H) {
    const int64_t j = b - slots * H, groups = gridDim.x - slots * H, c = covered_tokens(cu, max_segs, N);
    zero_tail(o, c, N, int64_t(H) * D * sizeof(T), j, groups);
    if (lse != nullptr)
      for (int64_t i = j * kThreads + threadIdx.x; i < (N - c) * H; i += groups * kThreads)
        lse[(i / (N - c)) * N + c + i % (N - c)] = -INFINITY;
    if (j == 0) check_cu(cu, max_segs, N, flags);
    return;
  }
  const int32_t h = int32_t(b % H);
  SegTile t;
  if (!find_tile(cu, max_segs, N, kT, int32_t(b / H), t)) return;
  const int32_t hk = h / (H / Hkv);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 31, half = lane >> 5;
  const int64_t row = int64_t(t.start) + col;
  Tile<D>&tk = tiles[2 * wave], &tv = tiles[2 * wave + 1];

  f32x4 qf[D / 8];
  load_row<T, D>(qf, q, row, row < t.e, H, h, half);
  float m = -INFINITY, l = 0.f;
  f32x16 acc[D / 32] = {};
  for (int64_t s0 = t.a + wave * kT; s0 <= t.start; s0 += kWaves * kT) {
    wave_fence();
    fill<T, D>(tk, k, s0, t.e, Hkv, hk, lane);
    const bool ok = fill<T, D>(tv, v, s0, t.e, Hkv, hk, lane);
    wave_fence();
    f32x16 x = over_channels<D>(tk, qf, col, half);
    float mt = m;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i] = s0 + row_of(i, half) <= row ? x[i] * scale : -INFINITY;
      mt = fmaxf(mt, x[i]);
    }
    mt = fmaxf(mt, other_half(mt));
    // a row whose scores so far are all -inf has no maximum to subtract
    const float ms = mt == -INFINITY ? 0.f : mt;
    const float f = expf(m - ms);
    m = mt;
    l *= f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x[i] = expf(x[i] - ms);
      l += x[i];
    }
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[j][i] *= f;
    if (s0 < t.start || __all(ok)) {
      over_rows<D>(acc, tv, x, col, half);
    } else {
      // The tile on the diagonal holds a value that is not finite: a weight of 0
      // times it is NaN, so such values are 0 in the product and are added for the
      // rows that attend to them alone. The other rows keep their bits.
      wave_fence();
      for (int i = lane; i < kT * D; i += 64) {
        const float y = tv.x[i / D][i % D];
        tk.x[i / D][i % D] = fabsf(y) <= kFinite ? y : 0.f;
      }
      wave_fence();
      over_rows<D>(acc, tk, x, col, half);
      wave_fence();
#pragma unroll
      for (int i = 0; i < 16; ++i) tk.x[row_of(i, half)][col] = x[i];
      wave_fence();
      for (int s = 0; s < kT && s0 + s <= row && s0 + s < t.e; ++s) {
        const float p = tk.x[s][col];
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float y = tv.x[s][32 * j + row_of(i, half)];
            if (!(fabsf(y) <= kFinite)) acc[j][i] += p * y;
          }
      }
    }
  }
  l += other_half(l);
  wave_fence();
  put_sums<D>(tk, acc, col, half);
  if (half == 0) {
    sm[wave][col] = m;
    sl[wave][col] = l;
  }
  __syncthreads();
  const int32_t rows = t.e - t.start;
  for (int i = threadIdx.x; i < kT * D / 4; i += kThreads) {
    const int r = i / (D / 4), d = i % (D / 4) * 4;
    if (r >= rows) continue;
    float top = sm[0][r];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) top = fmaxf(top, sm[w][r]);
    const float ms = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (t.a + w * kT > t.start) continue;  // (had no tile)
      const float f = expf(sm[w][r] - ms);
      sum += f * sl[w][r];
      x += f * tiles[2 * w].at(r, d);
    }
    store4(o + ((int64_t(t.start) + r) * H + h) * D + d, x * (1.f / sum));
    if (lse != nullptr && d == 0) lse[int64_t(h) * N + t.start + r] = top + logf(sum);
  }
}

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_simple_dq(
    const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, const T* __restrict__ o,
    const T* __restrict__ dout, const float* __restrict__ lse, float* __restrict__ delta,
    const int32_t* __restrict__ cu, int32_t max_segs, int64_t N, int32_t H, int32_t Hkv, float scale,
    T* __restrict__ dq, int32_t* __restrict__ flags, int64_t slots) {
  __shared__ Tile<D> tiles[2 * kWaves];
  const int64_t b = blockIdx.x;
  if (b >= slots * H) {
    zero_tail(dq, covered_tokens(cu, max_segs, N), N, int64_t(H) * D * sizeof(T), b - slots * H, gridDim.x - slots * H);
    if (b == slots * H) check_cu(cu, max_segs, N, flags);
    return;
  }
  const int32_t h = int32_t(b % H);
  SegTile t;
  if (!find_tile(cu, max_segs, N, kT, int32_t(b / H), t)) return;
  const int32_t hk = h / (H / Hkv);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 31, half = lane >> 5;
  const int64_t row = int64_t(t.start) + col;
  const bool real = row < t.e;
  Tile<D>&tk = tiles[2 * wave], &tv = tiles[2 * wave + 1];

  f32x4 qf[D / 8], df[D / 8];
  load_row<T, D>(qf, o, row, real, H, h, half);
  load_row<T, D>(df, dout, row, real, H, h, half);
  float dl = 0.f;
#pragma unroll
  for (int p = 0; p < D / 8; ++p)
#pragma unroll
    for (int e = 0; e < 4; ++e) dl += qf[p][e] * df[p][e];
  dl += other_half(dl);
  load_row<T, D>(qf, q, row, real, H, h, half);
  const float ls = real ? lse[int64_t(h) * N + row] : INFINITY;
  if (real && wave == 0 && half == 0) delta[int64_t(h) * N + row] = dl;  // for the keys pass
  f32x16 acc[D / 32] = {};
  for (int64_t s0 = t.a + wave * kT; s0 <= t.start; s0 += kWaves * kT) {
    wave_fence();
    fill<T, D>(tk, k, s0, t.e, Hkv, hk, lane);
    fill<T, D>(tv, v, s0, t.e, Hkv, hk, lane);
    wave_fence();
    f32x16 x = over_channels<D>(tk, qf, col, half);
    const f32x16 y = over_channels<D>(tv, df, col, half);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      x[i] = s0 + row_of(i, half) <= row ? expf(x[i] * scale - ls) * (y[i] - dl) : 0.f;
    over_rows<D>(acc, tk, x, col, half);
  }
  wave_fence();
  put_sums<D>(tk, acc, col, half);
  __syncthreads();
  store_sums<T, D>(tiles, scale, dq + (int64_t(t.start) * H + h) * D, int64_t(H) * D, t.e - t.start);
}

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_simple_dkv(
    const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, const T* __restrict__ dout,
    const float* __restrict__ lse, const float* __restrict__ delta, const int32_t* __restrict__ cu,
    int32_t max_segs, int64_t N, int32_t H, int32_t Hkv, float scale, T* __restrict__ dk,
    T* __restrict__ dv, int64_t slots) {
  __shared__ Tile<D> tiles[2 * kWaves];
  const int64_t b = blockIdx.x;
  if (b >= slots * Hkv) {
    const int64_t j = b - slots * Hkv, groups = gridDim.x - slots * Hkv, cov = covered_tokens(cu, max_segs, N);
    zero_tail(dk, cov, N, int64_t(Hkv) * D * sizeof(T), j, groups);
    zero_tail(dv, cov, N, int64_t(Hkv) * D * sizeof(T), j, groups);
    return;
  }
  const int32_t hk = int32_t(b % Hkv);
  SegTile t;
  if (!find_tile(cu, max_segs, N, kT, int32_t(b / Hkv), t)) return;
  const int32_t rep = H / Hkv;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 31, half = lane >> 5;
  const int64_t row = int64_t(t.start) + col;  // the lane's key
  Tile<D>&tq = tiles[2 * wave], &to = tiles[2 * wave + 1];

  f32x4 kf[D / 8], vf[D / 8];
  load_row<T, D>(kf, k, row, row < t.e, Hkv, hk, half);
  load_row<T, D>(vf, v, row, row < t.e, Hkv, hk, half);
  f32x16 ak[D / 32] = {}, av[D / 32] = {};
  // (query head, query tile) pairs, dealt to the waves in turn
  const int64_t per = (int64_t(t.e) - t.start + kT - 1) / kT;
  for (int64_t it = wave; it < per * rep; it += kWaves) {
    const int32_t h = hk * rep + int32_t(it / per);
    const int64_t s0 = t.start + it % per * kT;
    wave_fence();
    fill<T, D>(tq, q, s0, t.e, H, h, lane);
    fill<T, D>(to, dout, s0, t.e, H, h, lane);
    float ls[16], dl[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int64_t s = s0 + row_of(i, half);
      ls[i] = s < t.e ? lse[int64_t(h) * N + s] : INFINITY;
      dl[i] = s < t.e ? delta[int64_t(h) * N + s] : 0.f;
    }
    wave_fence();
    f32x16 x = over_channels<D>(tq, kf, col, half);
    f32x16 y = over_channels<D>(to, vf, col, half);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int64_t s = s0 + row_of(i, half);
      x[i] = s >= row && s < t.e ? expf(x[i] * scale - ls[i]) : 0.f;
      y[i] = x[i] * (y[i] - dl[i]);
    }
    over_rows<D>(av, to, x, col, half);
    over_rows<D>(ak, tq, y, col, half);
  }
  const int64_t to_ = (int64_t(t.start) * Hkv + hk) * D;
  wave_fence();
  put_sums<D>(tq, ak, col, half);
  __syncthreads();
  store_sums<T, D>(tiles, scale, dk + to_, int64_t(Hkv) * D, t.e - t.start);
  __syncthreads();
  put_sums<D>(tq, av, col, half);
  __syncthreads();
  store_sums<T, D>(tiles, 1.f, dv + to_, int64_t(Hkv) * D, t.e - t.start);
}

template <typename T, int D>
hipError_t fwd(const AttnArgs& a, hipStream_t stream) {
  const int64_t slots = tile_slots(a.N, a.max_segs, kT), grid = slots * a.H + tail_groups(a.N * a.H * D * sizeof(T));
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
  attn_simple_dq<T, D><<<dim3(uint32_t(slots * a.H + tail_groups(a.N * a.H * D * sizeof(T)))), dim3(kThreads), 0, stream>>>(
      q, k, v, static_cast<const T*>(a.o), dout, a.lse, g.stats, a.cu, a.max_segs, a.N, a.H, a.Hkv, a.scale,
      static_cast<T*>(g.dq), a.flags, slots);
  attn_simple_dkv<T, D><<<dim3(uint32_t(slots * a.Hkv + tail_groups(a.N * a.Hkv * D * sizeof(T)))), dim3(kThreads), 0, stream>>>(
      q, k, v, dout, a.lse, g.stats, a.cu, a.max_segs, a.N, a.H, a.Hkv, a.scale, static_cast<T*>(g.dk),
      static_cast<T*>(g.dv), slots);
  return hipGetLastError();
}

}  // namespace

// bf16: D = 32 alone (64 and 128 are attn_fwd.hip's and attn_bwd.hip's).
hipError_t launch_attn_simple(const AttnArgs& a, int32_t dtype, hipStream_t stream) {
  if (dtype == 0) return a.D == 32 ? fwd<bf16, 32>(a, stream) : hipErrorInvalidValue;
  if (a.D == 32) return fwd<float, 32>(a, stream);
  if (a.D == 64) return fwd<float, 64>(a, stream);
  return fwd<float, 128>(a, stream);
}

hipError_t launch_attn_simple_backward(const AttnArgs& a, const AttnGradArgs& g, int32_t dtype,
                                       hipStream_t stream) {
  if (dtype == 0) return a.D == 32 ? bwd<bf16, 32>(a, g, stream) : hipErrorInvalidValue;
  if (a.D == 32) return bwd<float, 32>(a, g, stream);
  if (a.D == 64) return bwd<float, 64>(a, g, stream);
  return bwd<float, 128>(a, g, stream);
}

}  // namespace pkv
