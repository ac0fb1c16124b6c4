// Reverse pass of the packed causal softmax attention on the matrix cores
// (bf16, D in {64, 128}).
//
// With P_ts = exp(scale q_t.k_s - lse_t), delta_t = do_t.o_t and
// dS_ts = P_ts (do_t.v_s - delta_t):
//   dq_t = scale sum_s dS_ts k_s,  dk_s = scale sum_t dS_ts q_t,
//   dv_s = sum_t P_ts do_t, the last two also over the query heads of the kv head.
//
// Two passes, each owning its outputs, so nothing is added by atomics and equal
// calls give equal bits; S and dP are formed in both (7 products of the size of
// the forward pass's two instead of 5):
//   queries  a wave holds 32 queries (q and do as operands, dq^T as the sum) and
//            the work-group walks the keys in tiles of 64:
//            S^T = K Q^T, dP^T = V dO^T, dq^T += K^T dS^T. It also forms delta
//            and lse log2 e for the second pass.
//   keys     a wave holds 32 keys (k and v as operands, dk^T and dv^T as sums)
//            and the work-group walks the queries of every head of the group in
//            tiles of 64: S = Q K^T, dP = dO V^T, dv^T += dO^T P, dk^T += Q^T dS.
// As in the forward pass the result of the first products is, register for
// register, an operand of the second ones, and the other operand comes from the
// same LDS tile by transposing reads.
//
// Tiles go from memory into LDS without passing registers, the next while one
// is used. 16-byte chunk c of row r is kept at chunk c ^ f(r), with f such that
// 16 consecutive rows (row-wise reads) and the four 64-byte pieces of 4
// consecutive rows (transposing reads of 32 lanes) fall on distinct banks.

#include "mfma.h"
#include "segments.h"

namespace pkv {
namespace {

constexpr int kB = 128;   // queries, or keys, that a work-group owns
constexpr int kT = 64;    // tokens of a tile of the other side
constexpr int kThreads = 256;
constexpr int kTail = 256;

template <int D>
struct Lds {
  static constexpr int CH = D / 8, ROW = D * 2, BYTES = kT * ROW;
  static __device__ __forceinline__ int swz(int row) {
    return D == 128 ? ((row & 3) << 2) | ((row >> 2) & 3) : ((row & 2) << 1) | ((row >> 2) & 3);
  }
};

// The lane's part in loading a 64-row tile: byte offsets of its LD chunks.
template <int D>
struct Loader {
  static constexpr int LD = kT * Lds<D>::CH / kThreads;
  uint32_t off[LD];
  __device__ __forceinline__ Loader(int32_t stride) {
#pragma unroll
    for (int i = 0; i < LD; ++i) {
      const int ch = i * kThreads + threadIdx.x, row = ch / Lds<D>::CH, pos = ch % Lds<D>::CH;
      off[i] = uint32_t(row) * stride + (pos ^ Lds<D>::swz(row)) * 16;
    }
  }
  __device__ __forceinline__ void issue(__amdgpu_buffer_rsrc_t r, char* dst, int wave) const {
#pragma unroll
    for (int i = 0; i < LD; ++i) load_lds16(r, off[i], dst + wave * 1024 + i * kThreads * 16);
  }
};

// Operand reads from a tile: rows 32 j + lane % 32 (contraction over channels,
// step i of 16), and transposed: channels 32 i + lane % 32 (contraction over
// the rows of 16-row step j, in the order of a product's result registers).
template <int D>
struct Reader {
  int col, half, fx;
  int tr[2];   // row and half-chunk bytes of the two transposing reads
  int tc[2];   // swizzled chunk before the 32-channel group is added
  __device__ __forceinline__ Reader() {
    const int lane = threadIdx.x & 63;
    half = lane >> 5;
    col = lane & 31;
    fx = Lds<D>::swz(col);
    const int r = 4 * half + ((lane & 15) >> 2), c = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      tr[u] = (r + 8 * u) * Lds<D>::ROW + (lane & 1) * 8;
      tc[u] = c ^ Lds<D>::swz(r + 8 * u);
    }
  }
  __device__ __forceinline__ bf16x8 rows(const char* t, int j, int i) const {
    return *reinterpret_cast<const bf16x8*>(t + (32 * j + col) * Lds<D>::ROW + (((2 * i + half) ^ fx) * 16));
  }
  __device__ __forceinline__ bf16x8 channels(const char* t, int i, int j) const {
    const char* p = t + 16 * j * Lds<D>::ROW;
    return join(read_tr(p + tr[0] + ((4 * i) ^ tc[0]) * 16), read_tr(p + tr[1] + ((4 * i) ^ tc[1]) * 16));
  }
};

// `have` (<= 32) rows of one head as operand fragments: lane's row lane % 32.
template <int D>
__device__ __forceinline__ void load_rows(bf16x8 (&f)[D / 16], const bf16* base, int32_t have, int32_t stride,
                                          const Reader<D>& rd) {
  const auto r = buffer(base, have > 0 ? int64_t(have - 1) * stride + D * 2 : 0);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) f[i] = load8(r, uint32_t(rd.col) * stride + (2 * i + rd.half) * 16);
}

// 32 rows of a wave's transposed sums times f, through LDS, to `dst` (stride in
// elements); st: 32 rows of the wave's own.
template <int D>
__device__ __forceinline__ void store_rows(const f32x16 (&acc)[D / 32], float f, char* st, bf16* dst, int64_t stride,
                                           int32_t have, const Reader<D>& rd) {
  constexpr int CH = Lds<D>::CH, ROW = Lds<D>::ROW;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bf16x4 x;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = static_cast<bf16>(acc[i][4 * j + e] * f);
      *reinterpret_cast<bf16x4*>(st + rd.col * ROW + (((4 * i + j) ^ (rd.col & (CH - 1))) * 16) + rd.half * 8) = x;
    }
  asm volatile("" ::: "memory");  // the wave's own rows: its LDS accesses are in order
  for (int i = threadIdx.x & 63; i < 32 * CH; i += 64) {
    const int r = i / CH, ch = i % CH;
    if (r < have)
      *reinterpret_cast<i32x4*>(dst + r * stride + ch * 8) =
          *reinterpret_cast<const i32x4*>(st + r * ROW + ((ch ^ (r & (CH - 1))) * 16));
  }
}

template <int D>
__global__ __launch_bounds__(kThreads, 2) void attn_dq_kernel(
    const bf16* __restrict__ q, const bf16* __restrict__ k, const bf16* __restrict__ v, const bf16* __restrict__ o,
    const bf16* __restrict__ dout, const float* __restrict__ lse, const int32_t* __restrict__ cu, int32_t max_segs,
    int64_t N, int32_t H, int32_t Hkv, float scale, bf16* __restrict__ dq, float* __restrict__ stats,
    int32_t* __restrict__ flags, int32_t slots) {
  constexpr int KS = D / 16, DT = D / 32, TB = Lds<D>::BYTES;
  __shared__ __attribute__((aligned(1024))) char lds[4 * TB];  // K, V of the even tiles, K, V of the odd ones

  const int64_t b = blockIdx.x;
  if (b >= int64_t(slots) * H) {
    const int64_t j = b - int64_t(slots) * H;
    zero_tail(dq, covered_tokens(cu, max_segs, N), N, int64_t(H) * D * 2, j, kTail);
    if (j == 0) check_cu(cu, max_segs, N, flags);
    return;
  }
  const int32_t hi = int32_t(b % H), rep = H / Hkv, hk = hi % Hkv, h = hk * rep + hi / Hkv;
  SegTile t;
  if (!find_tile(cu, max_segs, N, kB, slots - 1 - int32_t(b / H), t)) return;

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Reader<D> rd;
  const int32_t kstride = Hkv * D * 2, qstride = H * D * 2;
  const int32_t q0 = t.start + wave * 32;
  const int32_t rows = t.e - q0, have = rows < 0 ? 0 : (rows > 32 ? 32 : rows);
  const int32_t qend = t.start + kB < t.e ? t.start + kB : t.e;
  const int n_tiles = (qend - t.a + kT - 1) / kT;
  const Loader<D> ld(kstride);
  auto issue = [&](int it) {
    const int32_t s0 = t.a + it * kT;
    const int32_t n = t.e - s0 < kT ? t.e - s0 : kT;
    const int64_t at = (int64_t(s0) * Hkv + hk) * D, bytes = int64_t(n - 1) * kstride + D * 2;
    char* dst = lds + (it & 1) * 2 * TB;
    ld.issue(buffer(k + at, bytes), dst, wave);
    ld.issue(buffer(v + at, bytes), dst + TB, wave);
  };
  issue(0);

  const int64_t at = (int64_t(have > 0 ? q0 : t.start) * H + h) * D;
  bf16x8 qf[KS], df[KS];
  load_rows<D>(df, dout + at, have, qstride, rd);
  float delta = 0.f;
  {
    load_rows<D>(qf, o + at, have, qstride, rd);
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) delta += to_f32(df[i][j]) * to_f32(qf[i][j]);
    delta += other_half(delta);
  }
  load_rows<D>(qf, q + at, have, qstride, rd);
  const int64_t row = int64_t(h) * N + q0 + rd.col;
  const float lse2 = rd.col < have ? lse[row] * kLog2e : 0.f;
  if (rd.half == 0 && rd.col < have) {
    stats[row] = lse2;
    stats[int64_t(H) * N + row] = delta;
  }

  const float c = scale * kLog2e;
  f32x16 acc[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) acc[i] = f32x16{};
  for (int it = 0; it < n_tiles; ++it) {
    wait_vm();
    bar();
    if (it + 1 < n_tiles) issue(it + 1);
    const char* kt = lds + (it & 1) * 2 * TB;
    const char* vt = kt + TB;
    const int32_t s0 = t.a + it * kT;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (have == 0 || s0 + 32 * j > q0 + 31) continue;
      f32x16 s = {}, dp = {};
#pragma unroll
      for (int i = 0; i < KS; ++i) s = mfma32(rd.rows(kt, j, i), qf[i], s);
#pragma unroll
      for (int i = 0; i < KS; ++i) dp = mfma32(rd.rows(vt, j, i), df[i], dp);
      bf16x8 ds[2];
      const int32_t last = s0 + 32 * j + 31 > q0 ? q0 + rd.col - s0 - 32 * j - 4 * rd.half : 32;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float p = ex2(fmaf(s[i], c, -lse2));
        const float x = p * (dp[i] - delta);
        ds[i / 8][i % 8] = static_cast<bf16>(8 * (i / 4) + i % 4 <= last ? x : 0.f);
      }
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) acc[i] = mfma32(rd.channels(kt, i, 2 * j + u), ds[u], acc[i]);
    }
  }
  __syncthreads();
  if (have > 0)
    store_rows<D>(acc, scale, lds + wave * (32 * D * 2), dq + (int64_t(q0) * H + h) * D, int64_t(H) * D, have, rd);
}

template <int D>
__global__ __launch_bounds__(kThreads, 2) void attn_dkv_kernel(
    const bf16* __restrict__ q, const bf16* __restrict__ k, const bf16* __restrict__ v,
    const bf16* __restrict__ dout, const float* __restrict__ stats, const int32_t* __restrict__ cu,
    int32_t max_segs, int64_t N, int32_t H, int32_t Hkv, float scale, bf16* __restrict__ dk,
    bf16* __restrict__ dv, int32_t slots) {
  constexpr int KS = D / 16, DT = D / 32, TB = Lds<D>::BYTES;
  // Q, dO of the even tiles, of the odd ones; then lse log2 e and delta of each
  __shared__ __attribute__((aligned(1024))) char lds[4 * TB + 4 * kT * 4];

  const int64_t b = blockIdx.x;
  if (b >= int64_t(slots) * Hkv) {
    const int64_t j = b - int64_t(slots) * Hkv, cov = covered_tokens(cu, max_segs, N);
    zero_tail(dk, cov, N, int64_t(Hkv) * D * 2, j, kTail);
    zero_tail(dv, cov, N, int64_t(Hkv) * D * 2, j, kTail);
    return;
  }
  const int32_t hk = int32_t(b % Hkv), rep = H / Hkv;
  SegTile t;
  if (!find_tile(cu, max_segs, N, kB, int32_t(b / Hkv), t)) return;

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Reader<D> rd;
  const int32_t kstride = Hkv * D * 2, qstride = H * D * 2;
  const int32_t k0 = t.start + wave * 32;  // the wave's first key
  const int32_t rows = t.e - k0, have = rows < 0 ? 0 : (rows > 32 ? 32 : rows);
  const int per_head = (t.e - t.start + kT - 1) / kT, n_tiles = per_head * rep;
  const Loader<D> ld(qstride);
  int ih = 0, iq = 0;  // head and query tile of the next load
  auto issue = [&](int it) {
    const int32_t s0 = t.start + iq * kT, h = hk * rep + ih;
    const int32_t n = t.e - s0 < kT ? t.e - s0 : kT;
    const int64_t at = (int64_t(s0) * H + h) * D, bytes = int64_t(n - 1) * qstride + D * 2;
    char* dst = lds + (it & 1) * 2 * TB;
    ld.issue(buffer(q + at, bytes), dst, wave);
    ld.issue(buffer(dout + at, bytes), dst + TB, wave);
    if (wave < 2)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          buffer(stats + (int64_t(wave) * H + h) * N + s0, int64_t(n) * 4),
          (__attribute__((address_space(3))) void*)(lds + 4 * TB + ((it & 1) * 2 + wave) * kT * 4), 4,
          uint32_t(lane) * 4, 0, 0, 0);
    if (++iq == per_head) {
      iq = 0;
      ++ih;
    }
  };
  issue(0);

  const int64_t at = (int64_t(have > 0 ? k0 : t.start) * Hkv + hk) * D;
  bf16x8 kf[KS], vf[KS];
  load_rows<D>(kf, k + at, have, kstride, rd);
  load_rows<D>(vf, v + at, have, kstride, rd);
  const float c = scale * kLog2e;
  f32x16 ak[DT], av[DT];
#pragma unroll
  for (int i = 0; i < DT; ++i) {
    ak[i] = f32x16{};
    av[i] = f32x16{};
  }
  int cq = 0;  // query tile in use
  for (int it = 0; it < n_tiles; ++it) {
    wait_vm();
    bar();
    if (it + 1 < n_tiles) issue(it + 1);
    const char* qt = lds + (it & 1) * 2 * TB;
    const char* ot = qt + TB;
    const f32x4* ls = reinterpret_cast<const f32x4*>(lds + 4 * TB + (it & 1) * 2 * kT * 4);
    const f32x4* dl = ls + kT / 4;
    const int32_t s0 = t.start + cq * kT;
    if (++cq == per_head) cq = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int32_t b0 = s0 + 32 * j;  // first query of the block
      if (have == 0 || b0 + 31 < k0 || b0 >= t.e) continue;
      f32x16 s = {}, dp = {};
#pragma unroll
      for (int i = 0; i < KS; ++i) s = mfma32(rd.rows(qt, j, i), kf[i], s);
#pragma unroll
      for (int i = 0; i < KS; ++i) dp = mfma32(rd.rows(ot, j, i), vf[i], dp);
      bf16x8 p[2], ds[2];
      // the lane's key takes part in the block's queries first .. end - 1
      const bool edge = b0 < k0 + 31 || b0 + 32 > t.e;
      const int32_t first = edge ? k0 + rd.col - b0 - 4 * rd.half : -64;
      const int32_t end = edge ? t.e - b0 - 4 * rd.half : 64;
#pragma unroll
      for (int i4 = 0; i4 < 4; ++i4) {
        const f32x4 l4 = ls[8 * j + 2 * i4 + rd.half], d4 = dl[8 * j + 2 * i4 + rd.half];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = 4 * i4 + e, r = 8 * i4 + e;
          float x = ex2(fmaf(s[i], c, -l4[e]));
          x = r >= first && r < end ? x : 0.f;
          p[i / 8][i % 8] = static_cast<bf16>(x);
          ds[i / 8][i % 8] = static_cast<bf16>(x * (dp[i] - d4[e]));
        }
      }
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          av[i] = mfma32(rd.channels(ot, i, 2 * j + u), p[u], av[i]);
          ak[i] = mfma32(rd.channels(qt, i, 2 * j + u), ds[u], ak[i]);
        }
    }
  }
  __syncthreads();
  if (have > 0) {
    char* st = lds + wave * (32 * D * 2);
    const int64_t to = (int64_t(k0) * Hkv + hk) * D;
    store_rows<D>(ak, scale, st, dk + to, int64_t(Hkv) * D, have, rd);
    asm volatile("" ::: "memory");
    store_rows<D>(av, 1.f, st, dv + to, int64_t(Hkv) * D, have, rd);
  }
}

template <int D>
hipError_t run(const AttnArgs& a, const AttnGradArgs& g, hipStream_t stream) {
  const auto *q = static_cast<const bf16*>(a.q), *k = static_cast<const bf16*>(a.k), *v = static_cast<const bf16*>(a.v);
  const bf16* dout = static_cast<const bf16*>(g.dout);
  const int64_t slots = tile_slots(a.N, a.max_segs, kB);
  attn_dq_kernel<D><<<dim3(uint32_t(slots * a.H + kTail)), dim3(kThreads), 0, stream>>>(
      q, k, v, static_cast<const bf16*>(a.o), dout, a.lse, a.cu, a.max_segs, a.N, a.H, a.Hkv, a.scale,
      static_cast<bf16*>(g.dq), g.stats, a.flags, int32_t(slots));
  attn_dkv_kernel<D><<<dim3(uint32_t(slots * a.Hkv + kTail)), dim3(kThreads), 0, stream>>>(
      q, k, v, dout, g.stats, a.cu, a.max_segs, a.N, a.H, a.Hkv, a.scale, static_cast<bf16*>(g.dk),
      static_cast<bf16*>(g.dv), int32_t(slots));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_bwd(const AttnArgs& a, const AttnGradArgs& g, hipStream_t stream) {
  return a.D == 64 ? run<64>(a, g, stream) : run<128>(a, g, stream);
}

}  // namespace pkv
