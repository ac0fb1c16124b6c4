// Attention of new tokens over the paged cache in fp32 on the matrix cores: fp32
// tensors, and bf16 tensors at D = 32.
//
//   o_t = sum_s softmax_s(scale q_t.k_s) v_s over the places s <= t of t's request,
//   with a window those with t - s < window or s < sinks.
//
// A work-group takes rows of one request and kv head, 32 at a time: row i is new token
// i / rep, query head i % rep of the group, so that a group's heads share the keys.
// Its four waves take the tiles of 32 places in turn, each in LDS of its own, and
// their sums are joined at the end. The products' layouts are those of the packed
// kernels in attn_simple.hip. Where the call has fewer row tiles than the chip holds
// work-groups, a walk is split over several, and a second launch joins their sums.
//
// These shapes serve the small fp32 batches that models are debugged on. Bound by the
// latency of a tile's loads: a wave has one tile at a time, and its fp32 products take 32
// rows where a decoding request has H / Hkv. fp32, one token each: one request of 131072
// tokens, H 32, Hkv 8, D 128: 0.81 ms (unsplit 25), 1.33 TB/s; 8 of 8000, H 8, Hkv 4, D 64:
// 62 us, 2.1 TB/s; 4 of 300, D 32: 18 us.

#include "attn_f32.h"
#include "paged.h"

namespace pkv {
namespace {

// What a tile's rows see, by the 16 places of a granule (pages are multiples of them): some
// row sees a granule whose first place is at most `hi` and past `oldest` or one of the sinks.
struct Seen {
  int32_t hi, sinks;
  int64_t oldest;
  // rows at places lo .. hi; window 0: none
  __device__ __forceinline__ Seen(int32_t lo, int32_t hi, int32_t window, int32_t sinks)
      : hi(hi), sinks(sinks), oldest(window > 0 ? int64_t(lo) - window - 15 : -16) {}
  __device__ __forceinline__ bool granule(int32_t p) const {
    const int32_t first = p & ~15;
    return first <= hi && (first > oldest || first < sinks);
  }
};

// 32 places of a request from p0 on, zero past its end, in a missing page and where no row
// sees the granule: its page may be gone, so the table is not asked for it.
template <typename T, int D>
__device__ __forceinline__ void fill(Tile<D>& tk, Tile<D>& tv, const PagedArgs& c, const T* __restrict__ kp,
                                     const T* __restrict__ vp, int32_t r, int32_t len, int32_t p0, const Seen& seen,
                                     int32_t hk, int lane) {
  // lane l looks up the row of place l % 32
  const int32_t p = p0 + (lane & 31);
  const int32_t page = p < len && seen.granule(p) ? page_of(c, r, p) : -1;
  const int64_t row = page < 0 ? -1 : page_row(c, page, p) * c.Hkv + hk;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    const int at = (i * 64 + lane) * 4, x = at / D, d = at % D;
    const int64_t src = __shfl(row, x, 64);
    const f32x4 z = {0.f, 0.f, 0.f, 0.f};
    *reinterpret_cast<f32x4*>(&tk.x[x][d]) = src < 0 ? z : load4(kp + src * D + d);
    *reinterpret_cast<f32x4*>(&tv.x[x][d]) = src < 0 ? z : load4(vp + src * D + d);
  }
}

// The parts' sums in the workspace, a record of [32, D] and [32, 2] (m, l) for each row
// tile, kv head and split. Tile i of request r has slot floor(cu[r] rep / 32) + r + i: those
// of different requests do not meet.
int64_t tile_slots(int64_t N, int64_t R, int32_t rep) { return N * rep / kT + R; }
template <int D>
__device__ __forceinline__ float* record(const AttnPagedArgs& x, const PagedArgs& c, const Request& rq, int32_t r,
                                         int64_t row0, int32_t hk, int splits, int split) {
  const int64_t slot = int64_t(rq.a) * (x.Hq / c.Hkv) / kT + r + row0 / kT;
  return static_cast<float*>(x.workspace) + ((slot * c.Hkv + hk) * splits + split) * (kT * (D + 2));
}

template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_paged_simple_kernel(const PagedArgs c, const AttnPagedArgs x, int parts,
                                                                     int splits, int64_t groups) {
  __shared__ Tile<D> tiles[2 * kWaves];
  __shared__ float sm[kWaves][kT], sl[kWaves][kT];
  const int64_t b = blockIdx.x;
  T* const o = static_cast<T*>(x.o);
  if (b >= groups) {
    const int64_t j = b - groups, n = gridDim.x - groups, end = covered_tokens(c.cu, c.R, c.N);
    zero_tail(o, end, c.N, int64_t(x.Hq) * D * sizeof(T), j, n);
    if (x.lse != nullptr)
      for (int64_t i = j * kThreads + threadIdx.x; i < (c.N - end) * x.Hq; i += n * kThreads)
        x.lse[(i / (c.N - end)) * c.N + end + i % (c.N - end)] = -INFINITY;
    if (j == 0) check_requests(c);
    return;
  }
  const int32_t split = int32_t(b % splits), part = int32_t(b / splits % parts);
  const int32_t hk = int32_t(b / splits / parts % c.Hkv), r = int32_t(b / splits / parts / c.Hkv);
  const Request rq = request(c, r);
  if (!rq.ok) return;
  const int32_t rep = x.Hq / c.Hkv, first = rq.len - rq.n;  // the first new token's place
  const int64_t rows = int64_t(rq.n) * rep;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 31, half = lane >> 5;
  const bool win = x.window > 0;
  const T *kp = static_cast<const T*>(x.k_pages), *vp = static_cast<const T*>(x.v_pages);
  Tile<D>&tk = tiles[2 * wave], &tv = tiles[2 * wave + 1];

  for (int64_t row0 = int64_t(part) * kT; row0 < rows; row0 += int64_t(parts) * kT) {
    const int64_t row = row0 + col, last_row = row0 + kT < rows ? row0 + kT - 1 : rows - 1;
    const int32_t place = first + int32_t(row / rep);  // of the lane's row
    const int64_t out = (rq.a + row / rep) * x.Hq + hk * rep + row % rep;
    const int32_t lo = first + int32_t(row0 / rep), hi = first + int32_t(last_row / rep);
    auto sees = [&](int32_t p) { return p <= place && (!win || place - p < x.window || p < x.sinks); };

    f32x4 qf[D / 8];
#pragma unroll
    for (int p = 0; p < D / 8; ++p)
      qf[p] = row < rows ? load4(static_cast<const T*>(x.q) + out * D + 8 * p + 4 * half) : f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;
    f32x16 acc[D / 32] = {};
    const WindowWalk ww(win ? x.window : 0x7fffffff, win ? x.sinks : 0, kT, lo > 0 ? lo : 0, 0);
    const int32_t n_tiles = hi < 0 ? 0 : ww.count(hi / kT + 1);
    const Seen seen(lo, hi, x.window, x.sinks);
    for (int32_t it = split * kWaves + wave; it < n_tiles; it += splits * kWaves) {
      const int32_t s0 = ww.tile(it) * kT;
      wave_fence();
      fill<T, D>(tk, tv, c, kp, vp, r, rq.len, s0, seen, hk, lane);
      wave_fence();
      f32x16 s = {};
#pragma unroll
      for (int p = 0; p < D / 8; ++p) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(&tk.x[col][8 * p + 4 * half]);
#pragma unroll
        for (int e = 0; e < 4; ++e) s = __builtin_amdgcn_mfma_f32_32x32x2f32(a[e], qf[p][e], s, 0, 0, 0);
      }
      float mt = m;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[i] = sees(s0 + row_of(i, half)) ? s[i] * x.scale : -INFINITY;
        mt = fmaxf(mt, s[i]);
      }
      mt = fmaxf(mt, other_half(mt));
      // a row whose scores so far are all -inf has no maximum to subtract
      const float ms = mt == -INFINITY ? 0.f : mt;
      // (more than 0, as it is without its rounding: an infinity in a sum stays one, however
      // much larger a later score)
      const float f = fmaxf(expf(m - ms), 0x1p-149f);
      m = mt;
      l *= f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[i] = expf(s[i] - ms);
        l += s[i];
      }
#pragma unroll
      for (int j = 0; j < D / 32; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[j][i] *= f;
      // A weight of 0 times a value that is not finite is NaN: such values are 0 in the
      // product and are added for the rows that see them alone.
      bool odd = false;
      for (int i = lane; i < kT * D; i += 64) {
        const float y = tv.x[i / D][i % D];
        tk.x[i / D][i % D] = fabsf(y) <= kFinite ? y : 0.f;
        odd |= !(fabsf(y) <= kFinite);
      }
      wave_fence();
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
          acc[j] = __builtin_amdgcn_mfma_f32_32x32x2f32(tk.x[row_of(i, half)][32 * j + col], s[i], acc[j], 0, 0, 0);
      if (__any(odd)) {
        for (int p = 0; p < kT; ++p) {
          if (!sees(s0 + p)) continue;
#pragma unroll
          for (int j = 0; j < D / 32; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float y = tv.x[p][32 * j + row_of(i, half)];
              if (!(fabsf(y) <= kFinite)) acc[j][i] += y;
            }
        }
      }
    }
    l += other_half(l);
    wave_fence();
#pragma unroll
    for (int j = 0; j < D / 32; ++j)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<f32x4*>(&tk.x[col][32 * j + row_of(i, half)]) =
            f32x4{acc[j][i], acc[j][i + 1], acc[j][i + 2], acc[j][i + 3]};
    if (half == 0) {
      sm[wave][col] = m;
      sl[wave][col] = l;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < kT * D / 4; i += kThreads) {
      const int q = i / (D / 4), d = i % (D / 4) * 4;
      if (row0 + q >= rows) continue;
      float top = sm[0][q];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) top = fmaxf(top, sm[w][q]);
      const float ms = top == -INFINITY ? 0.f : top;
      float sum = 0.f;
      f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = expf(sm[w][q] - ms);
        sum += f * sl[w][q];
        const f32x4 z = *reinterpret_cast<const f32x4*>(&tiles[2 * w].x[q][d]);
        // (an infinity stays one, however small its wave's share)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] += fabsf(z[e]) <= kFinite ? f * z[e] : z[e];
      }
      if (splits > 1) {
        float* rec = record<D>(x, c, rq, r, row0, hk, splits, split);
        store4(rec + q * D + d, y);
        if (d == 0) {
          rec[kT * D + 2 * q] = top;
          rec[kT * D + 2 * q + 1] = sum;
        }
        continue;
      }
      const int64_t to = (rq.a + (row0 + q) / rep) * x.Hq + hk * rep + (row0 + q) % rep;
      store4(o + to * D + d, sum == 0.f ? f32x4{0.f, 0.f, 0.f, 0.f} : y * (1.f / sum));
      if (x.lse != nullptr && d == 0)
        x.lse[(hk * rep + (row0 + q) % rep) * c.N + rq.a + (row0 + q) / rep] = sum == 0.f ? -INFINITY : top + logf(sum);
    }
    __syncthreads();
  }
}

// Joins the splits' sums in their order, a thread 4 channels of a row.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_paged_simple_join_kernel(const PagedArgs c, const AttnPagedArgs x,
                                                                          int parts, int splits) {
  const int64_t b = blockIdx.x;
  const int32_t part = int32_t(b % parts), hk = int32_t(b / parts % c.Hkv), r = int32_t(b / parts / c.Hkv);
  const Request rq = request(c, r);
  const int32_t rep = x.Hq / c.Hkv;
  const int64_t rows = int64_t(rq.n) * rep;
  for (int64_t row0 = int64_t(part) * kT; row0 < rows; row0 += int64_t(parts) * kT) {
    const float* rec = record<D>(x, c, rq, r, row0, hk, splits, 0);
    for (int i = threadIdx.x; i < kT * D / 4; i += kThreads) {
      const int q = i / (D / 4), d = i % (D / 4) * 4;
      if (row0 + q >= rows) continue;
      float top = -INFINITY, sum = 0.f;
      f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
      for (int u = 0; u < splits; ++u) top = fmaxf(top, rec[u * (kT * (D + 2)) + kT * D + 2 * q]);
      const float ms = top == -INFINITY ? 0.f : top;
#pragma unroll 4
      for (int u = 0; u < splits; ++u) {
        const float* __restrict__ at = rec + u * (kT * (D + 2));
        const float f = expf(at[kT * D + 2 * q] - ms);
        sum += f * at[kT * D + 2 * q + 1];
        const f32x4 z = load4(at + q * D + d);
        // (an infinity stays one, however small its split's share)
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] += fabsf(z[e]) <= kFinite ? f * z[e] : z[e];
      }
      const int64_t to = (rq.a + (row0 + q) / rep) * x.Hq + hk * rep + (row0 + q) % rep;
      store4(static_cast<T*>(x.o) + to * D + d, sum == 0.f ? f32x4{0.f, 0.f, 0.f, 0.f} : y * (1.f / sum));
      if (x.lse != nullptr && d == 0)
        x.lse[(hk * rep + (row0 + q) % rep) * c.N + rq.a + (row0 + q) / rep] = sum == 0.f ? -INFINITY : top + logf(sum);
    }
  }
}

// A walk is split where the call's row tiles are fewer than the work-groups that the chip
// holds (by LDS, two tiles for each wave), so that it does.
int64_t most_splits(int64_t N, int64_t R, int32_t Hq, int32_t Hkv, int32_t D) {
  const int64_t chip = 256 * (D == 128 ? 1 : D == 64 ? 2 : 4), n = chip / (tile_slots(N, R, Hq / Hkv) * Hkv);
  return n < 1 ? 1 : n < 64 ? n : 64;
}

template <typename T, int D>
hipError_t run(const PagedArgs& c, const AttnPagedArgs& x, hipStream_t stream) {
  // a request's tiles of rows are dealt to as many work-groups as the call's rows could fill
  const int64_t pairs = int64_t(c.R) * c.Hkv, most = (c.N * (x.Hq / c.Hkv) + kT - 1) / kT, room = (1 << 16) / pairs;
  const int64_t parts = c.cu == nullptr ? (x.Hq / c.Hkv + kT - 1) / kT : (room < 1 ? 1 : (room < most ? room : most));
  // (a split has two tiles for each wave of the longest walk that the table allows)
  const int64_t worth = int64_t(c.max_pages) * c.page_size / (2 * kWaves * kT);
  int64_t splits = most_splits(c.N, c.R, x.Hq, c.Hkv, D);
  splits = worth < splits ? (worth < 1 ? 1 : worth) : splits;
  const int64_t groups = pairs * parts * splits;
  attn_paged_simple_kernel<T, D><<<dim3(uint32_t(groups + tail_groups(c.N * x.Hq * D * sizeof(T)))), dim3(kThreads), 0,
                                   stream>>>(c, x, int(parts), int(splits), groups);
  if (splits > 1)
    attn_paged_simple_join_kernel<T, D><<<dim3(uint32_t(pairs * parts)), dim3(kThreads), 0, stream>>>(c, x, int(parts),
                                                                                                     int(splits));
  return hipGetLastError();
}

}  // namespace

size_t attn_paged_simple_workspace_bytes(int64_t N, int32_t R, int32_t Hq, int32_t Hkv, int32_t D) {
  const int64_t n = most_splits(N, R, Hq, Hkv, D);
  return n == 1 ? 0 : size_t(tile_slots(N, R, Hq / Hkv)) * Hkv * n * kT * (D + 2) * 4;
}

hipError_t launch_attn_paged_simple(const PagedArgs& c, const AttnPagedArgs& x, int32_t dtype, hipStream_t stream) {
  if (dtype == 0) return c.D == 32 ? run<bf16, 32>(c, x, stream) : hipErrorInvalidValue;
  if (c.D == 32) return run<float, 32>(c, x, stream);
  if (c.D == 64) return run<float, 64>(c, x, stream);
  return run<float, 128>(c, x, stream);
}

}  // namespace pkv
