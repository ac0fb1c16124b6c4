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
//
// 8192 tokens (documents of about 800, the longest 3409), H 16, Hkv 4, D 128:
// forward 120, queries 171, keys 308 us, the longest document's walk; matrix
// instructions in 41 % and 30 % of the cycles. The keys pass holds k, v, dk and dv, 192
// registers at D 128, so two waves a SIMD and no step starts before the last is done
// with its registers. 32768 tokens in documents of about 104, H 32, D 64: 210 and
// 220 us for 0.55 and 0.69 GB, latency of one or two tiles a work-group.

#include "attn_grad.h"

#include <cmath>

namespace pkv {
namespace {

// A work-group of the keys pass is a serial walk over the queries of the group's
// heads. If the walk of the longest segment outlasts what all walks come to when
// dealt to the chip (512 work-groups of 128 keys at a time), it sets the time, and
// the form with kQ = 4 halves it; else the other form's steps are cheaper, and so
// is what its walks cost beside them. In queries: rep Lmax > 768 + 2 (rep Hkv sum L^2 / 2^17).
// Forward and reverse pass, kQ = 4 / 1 (rep Lmax, rep Hkv sum L^2 / 2^17):
//   one of 512 tokens, H 16, Hkv 4, D 128 (2048, 32)             89 / 147 us
//   one of 1024, H 8, Hkv 8, D 64 (1024, 64)                     63 / 84 us
//   one of 4096, H 16, Hkv 16, D 128 (4096, 2048)               480 / 496 us
//   8192, median 800, H 16, Hkv 4, D 128 (13636, 2579)          611 / 963 us
//   16384, median 800, H 32, Hkv 8, D 128 (13636, 7089)        1458 / 1461 us
//   16384 in docs of about 200, H 16, Hkv 4, D 128 (1580, 542)  335 / 271 us
//   32768, median 800, H 16, Hkv 16, D 128 (8192, 13547)       2775 / 2272 us
//   one of 32768, H 32, Hkv 8, D 128 (131072, 262144)          42.9 / 38.3 ms
__host__ __device__ inline bool shared_form(uint64_t longest, uint64_t squares, int32_t H, int32_t Hkv) {
  const double rep = H / Hkv;
  return rep * double(longest) > 768. + rep * Hkv * double(squares) * (1. / 65536);
}

// By one work-group, for the next launches.
__device__ __forceinline__ void choose_form(const int32_t* __restrict__ cu, int32_t max_segs, int64_t N, int32_t H,
                                            int32_t Hkv, int32_t* __restrict__ form, char* lds) {
  unsigned long long* sums = reinterpret_cast<unsigned long long*>(lds);  // the longest, the squares' sum
  if (threadIdx.x < 2) sums[threadIdx.x] = 0;
  __syncthreads();
  unsigned long long longest = 0, squares = 0;
  for (int64_t i = threadIdx.x; i < max_segs; i += kThreads) {
    const int64_t a = cu[i], e = cu[i + 1];
    if (!segment_ok(int32_t(i), a, e, N)) continue;
    const unsigned long long n = e - a;
    longest = n > longest ? n : longest;
    squares += n * n;
  }
  atomicMax(&sums[0], longest);
  atomicAdd(&sums[1], squares);
  __syncthreads();
  if (threadIdx.x == 0) *form = shared_form(sums[0], sums[1], H, Hkv) ? 4 : 1;
}

template <int D>
__global__ __launch_bounds__(kThreads, D == 64 ? 4 : 2) void attn_dq_kernel(
    const bf16* __restrict__ q, const bf16* __restrict__ k, const bf16* __restrict__ v, const bf16* __restrict__ o,
    const bf16* __restrict__ dout, const float* __restrict__ lse, const int32_t* __restrict__ cu, int32_t max_segs,
    int64_t N, int32_t H, int32_t Hkv, float scale, bf16* __restrict__ dq, float* __restrict__ stats,
    int32_t* __restrict__ flags, int32_t* __restrict__ form, SlotGrid grid) {
  constexpr int KS = D / 16, DT = D / 32, TB = Lds<D>::BYTES;
  __shared__ __attribute__((aligned(1024))) char lds[4 * TB];  // K, V of the even tiles, K, V of the odd ones

  const int64_t b = blockIdx.x;
  const int64_t blocks = slot_blocks(grid, H);
  if (b >= blocks) {
    const int64_t j = b - blocks, groups = gridDim.x - blocks;
    zero_tail(dq, covered_tokens(cu, max_segs, N), N, int64_t(H) * D * 2, j, groups);
    if (j == 0) check_cu(cu, max_segs, N, flags);
    if (j == 0 && form != nullptr) choose_form(cu, max_segs, N, H, Hkv, form, lds);
    return;
  }
  int32_t slot, h0, h1;
  slot_of(grid, b, H, slot, h0, h1);
  SegTile t;
  // late tiles have the most keys: they start first
  if (slot < grid.near) slot = grid.near - 1 - slot;
  if (!find_tile(cu, max_segs, N, kB, slot, t)) return;

  for (int32_t hi = h0; hi < h1; ++hi) {
    const int32_t hk = hi % Hkv, h = hk * (H / Hkv) + hi / Hkv;  // (as in the forward pass)
    // (nothing that goes by the lane is kept from one head to the next)
    const int tid = fresh(threadIdx.x), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Reader<D> rd(tid);
    const int32_t kstride = Hkv * D * 2, qstride = H * D * 2;
    const int32_t q0 = t.start + wave * 32;
    const int32_t rows = t.e - q0, have = rows < 0 ? 0 : (rows > 32 ? 32 : rows);
    const int32_t qend = t.start + kB < t.e ? t.start + kB : t.e;
    const int n_tiles = (qend - t.a + kT - 1) / kT;
    const Loader<D, kT, kThreads> ld(kstride, tid);
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

    const float c = scale * kLog2e;
    if (t.start == t.a) {
      // A segment's first 32 queries have all their keys in the first block: delta is
      // the sum of P dP there, without the rounding of o, which is as large as what
      // is left of dq where a row has few keys.
      wait_vm();
      bar();
      if (wave == 0) {
        const uint32_t kt = lds_addr(lds), vt = kt + TB;
        f32x16 s = {}, dp = {};
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          s = mfma32(rd.rows(kt, 0, i), qf[i], s);
          dp = mfma32(rd.rows(vt, 0, i), df[i], dp);
        }
        delta = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i)
          delta += 8 * (i / 4) + i % 4 <= rd.col - 4 * rd.half ? ex2(fmaf(s[i], c, -lse2)) * dp[i] : 0.f;
        delta += other_half(delta);
      }
    }
    float rest = 0.f;  // sum_s dS_ts
    f32x16 acc[DT];
#pragma unroll
    for (int i = 0; i < DT; ++i) acc[i] = f32x16{};
    for (int it = 0; it < n_tiles; ++it) {
      wait_vm();
      bar();
      if (it + 1 < n_tiles) issue(it + 1);
      const uint32_t kt = lds_addr(lds) + (it & 1) * 2 * TB, vt = kt + TB;
      const int32_t s0 = t.a + it * kT;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (have == 0 || s0 + 32 * j > q0 + 31) continue;
        f32x16 s = {}, dp = {};
#pragma unroll
        for (int i = 0; i < KS; ++i) {  // independent products take turns
          s = mfma32(rd.rows(kt, j, i), qf[i], s);
          dp = mfma32(rd.rows(vt, j, i), df[i], dp);
        }
        bf16x8 ds[2];
        const int32_t last = s0 + 32 * j + 31 > q0 ? q0 + rd.col - s0 - 32 * j - 4 * rd.half : 32;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float p = ex2(fmaf(s[i], c, -lse2));
          const float x = 8 * (i / 4) + i % 4 <= last ? p * (dp[i] - delta) : 0.f;
          rest += x;
          ds[i / 8][i % 8] = static_cast<bf16>(x);
        }
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int u = 0; u < 2; ++u) acc[i] = mfma32(rd.channels(kt, i, 2 * j + u), ds[u], acc[i]);
      }
    }
    // The sum of a row's dS is 0; what it is short of that is delta's error, which
    // stems from the rounding of o. The keys pass gets delta without it.
    rest += other_half(rest);
    if (rd.half == 0 && rd.col < have) {
      stats[row] = lse2;
      stats[int64_t(H) * N + row] = delta + rest;
    }
    __syncthreads();
    if (have > 0)
      store_rows<D>(acc, scale, lds + wave * (32 * D * 2), dq + (int64_t(q0) * H + h) * D, int64_t(H) * D, have, rd);
    if (hi + 1 < h1) __syncthreads();  // the outputs have left LDS
  }
}

// kQ waves share 32 keys and take the 32-query blocks of a tile in turn, their
// sums added at the end: kQ = 1, four waves hold 128 keys; kQ = 4, eight waves
// hold 64.
template <int kQ>
struct DkvShape {
  static constexpr int NT = kQ == 4 ? 512 : 256;  // threads
  static constexpr int KEYS = NT / 64 / kQ * 32;  // keys of a work-group
  static constexpr int T = kQ == 4 ? 128 : 64;    // queries per tile
};

template <int D, int kQ>
__global__ __launch_bounds__(DkvShape<kQ>::NT, D == 64 && kQ == 1 ? 3 : 2) void attn_dkv_kernel(
    const bf16* __restrict__ q, const bf16* __restrict__ k, const bf16* __restrict__ v,
    const bf16* __restrict__ dout, const float* __restrict__ stats, const int32_t* __restrict__ cu,
    int32_t max_segs, int64_t N, int32_t H, int32_t Hkv, float scale, bf16* __restrict__ dk,
    bf16* __restrict__ dv, const int32_t* __restrict__ form, SlotGrid grid) {
  if (form != nullptr && *form != kQ) return;
  constexpr int KS = D / 16, DT = D / 32;
  constexpr int NT = DkvShape<kQ>::NT, T = DkvShape<kQ>::T, TB = T * D * 2;
  // Q, dO of the even tiles, of the odd ones; then lse log2 e and delta of each
  __shared__ __attribute__((aligned(1024))) char lds[4 * TB + 4 * T * 4];

  const int64_t b = blockIdx.x;
  const int64_t blocks = slot_blocks(grid, Hkv);
  if (b >= blocks) {
    const int64_t j = b - blocks, groups = gridDim.x - blocks, cov = covered_tokens(cu, max_segs, N);
    zero_tail(dk, cov, N, int64_t(Hkv) * D * 2, j, groups);
    zero_tail(dv, cov, N, int64_t(Hkv) * D * 2, j, groups);
    return;
  }
  const int32_t rep = H / Hkv;
  int32_t slot, h0, h1;
  slot_of(grid, b, Hkv, slot, h0, h1);
  SegTile t;
  if (!find_tile(cu, max_segs, N, DkvShape<kQ>::KEYS, slot, t)) return;

  for (int32_t hk = h0; hk < h1; ++hk) {
    // (nothing that goes by the lane is kept from one head to the next)
    const int tid = fresh(threadIdx.x), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Reader<D> rd(tid);
    const int32_t kstride = Hkv * D * 2, qstride = H * D * 2;
    const int32_t k0 = t.start + wave / kQ * 32;  // the wave's first key
    const int32_t rows = t.e - k0, have = rows < 0 ? 0 : (rows > 32 ? 32 : rows);
    const int per_head = (t.e - t.start + T - 1) / T, n_tiles = per_head * rep;
    const Loader<D, T, NT> ld(qstride, tid);
    int ih = hk * rep, iq = 0;  // query head and tile of the next load
    // Q, dO and the statistics of the next tile
    auto issue = [&](int it) {
      const int32_t s0 = t.start + iq * T, h = ih;
      const int32_t n = t.e - s0 < T ? t.e - s0 : T;
      const int64_t at = (int64_t(s0) * H + h) * D, bytes = int64_t(n - 1) * qstride + D * 2;
      char* dst = lds + (it & 1) * 2 * TB;
      ld.issue(buffer(q + at, bytes), dst, wave);
      ld.issue(buffer(dout + at, bytes), dst + TB, wave);
      if (wave < T / 32) {  // lse log2 e and delta, 64 queries a wave
        const int w = wave / (T / 64), part = wave % (T / 64) * 64;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            buffer(stats + (int64_t(w) * H + h) * N + s0, int64_t(n) * 4),
            (__attribute__((address_space(3))) void*)(lds + 4 * TB + (((it & 1) * 2 + w) * T + part) * 4), 4,
            uint32_t(part + lane) * 4, 0, 0, 0);
      }
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
      const uint32_t qt0 = lds_addr(lds) + (it & 1) * 2 * TB;
      const f32x4* ls = reinterpret_cast<const f32x4*>(lds + 4 * TB + (it & 1) * 2 * T * 4);
      const f32x4* dl = ls + T / 4;
      const int32_t s0 = t.start + cq * T;
      if (++cq == per_head) cq = 0;
#pragma unroll 1
      for (int j = wave % kQ; j < T / 32; j += kQ) {
        const int32_t b0 = s0 + 32 * j;  // first query of the block
        // (addresses are formed per block: one register each instead of one per read)
        const uint32_t qt = fresh_uniform(qt0 + 32 * j * Lds<D>::ROW), ot = qt + TB;
        if (have == 0 || b0 + 31 < k0 || b0 >= t.e) continue;
        // Registers are full at D = 128 (k, v, dk and dv take 192): the weights are
        // done with before dP is begun, and nothing of a phase starts early. The
        // other wave of the SIMD fills the gaps.
        bf16x8 p[2], ds[2];
        f32x16 x = {};
#pragma unroll
        for (int i = 0; i < KS; ++i) x = mfma32(rd.rows(qt, 0, i), kf[i], x);
        if (D == 128) __builtin_amdgcn_sched_barrier(0);
        // the lane's key takes part in the block's queries first .. end - 1
        const bool edge = b0 < k0 + 31 || b0 + 32 > t.e;
        const int32_t first = edge ? k0 + rd.col - b0 - 4 * rd.half : -64;
        const int32_t end = edge ? t.e - b0 - 4 * rd.half : 64;
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) {
          const f32x4 l4 = ls[8 * j + 2 * i4 + rd.half];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 4 * i4 + e, r = 8 * i4 + e;
            const float y = ex2(fmaf(x[i], c, -l4[e]));
            x[i] = r >= first && r < end ? y : 0.f;
            p[i / 8][i % 8] = static_cast<bf16>(x[i]);
          }
        }
        if (D == 128) __builtin_amdgcn_sched_barrier(0);
        f32x16 dp = {};
#pragma unroll
        for (int i = 0; i < KS; ++i) dp = mfma32(rd.rows(ot, 0, i), vf[i], dp);
        if (D == 128) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) {
          const f32x4 d4 = dl[8 * j + 2 * i4 + rd.half];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 4 * i4 + e;
            ds[i / 8][i % 8] = static_cast<bf16>(x[i] * (dp[i] - d4[e]));
          }
        }
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            av[i] = mfma32(rd.channels(ot, i, u), p[u], av[i]);
            ak[i] = mfma32(rd.channels(qt, i, u), ds[u], ak[i]);
          }
      }
    }
    __syncthreads();
    if constexpr (kQ > 1) {
      // The sums of the waves that share keys: each in turn hands dk, then dv,
      // to the first of them.
      static_assert(NT / 64 / kQ * DT * 4096 <= 4 * TB, "sums in flight");
      f32x4* mine = reinterpret_cast<f32x4*>(lds) + (wave / kQ) * (DT * 4 * 64) + lane;
      auto join_sums = [&](f32x16 (&x)[DT], int from) {
        if (wave % kQ == from) {
#pragma unroll
          for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mine[(4 * i + j) * 64] = f32x4{x[i][4 * j], x[i][4 * j + 1], x[i][4 * j + 2], x[i][4 * j + 3]};
        }
        __syncthreads();
        if (wave % kQ == 0) {
#pragma unroll
          for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const f32x4 y = mine[(4 * i + j) * 64];
#pragma unroll
              for (int e = 0; e < 4; ++e) x[i][4 * j + e] += y[e];
            }
        }
        __syncthreads();
      };
#pragma unroll 1
      for (int from = 1; from < kQ; ++from) {
        join_sums(ak, from);
        join_sums(av, from);
      }
    }
    if (have > 0 && wave % kQ == 0) {
      char* st = lds + wave / kQ * (32 * D * 2);
      const int64_t to = (int64_t(k0) * Hkv + hk) * D;
      store_rows<D>(ak, scale, st, dk + to, int64_t(Hkv) * D, have, rd);
      asm volatile("" ::: "memory");
      store_rows<D>(av, 1.f, st, dv + to, int64_t(Hkv) * D, have, rd);
    }
    if (hk + 1 < h1) __syncthreads();  // the outputs have left LDS
  }
}

template <int D, int kQ>
void keys_pass(const AttnArgs& a, const AttnGradArgs& g, const int32_t* form, hipStream_t stream) {
  const SlotGrid grid = slot_grid(a.N, a.max_segs, DkvShape<kQ>::KEYS);
  const dim3 blocks(uint32_t(slot_blocks(grid, a.Hkv) + tail_groups(a.N * a.Hkv * D * 2)));
  attn_dkv_kernel<D, kQ><<<blocks, dim3(DkvShape<kQ>::NT), 0, stream>>>(
      static_cast<const bf16*>(a.q), static_cast<const bf16*>(a.k), static_cast<const bf16*>(a.v),
      static_cast<const bf16*>(g.dout), g.stats, a.cu, a.max_segs, a.N, a.H, a.Hkv, a.scale,
      static_cast<bf16*>(g.dk), static_cast<bf16*>(g.dv), form, grid);
}

template <int D>
hipError_t run(const AttnArgs& a, const AttnGradArgs& g, hipStream_t stream) {
  const SlotGrid grid = slot_grid(a.N, a.max_segs, kB);
  // Whether any lengths make the shared form the better one: of one segment of L
  // tokens, 1 > Hkv L / 2^16 + 768 / (rep L), the least at the L of equal terms.
  const double rep = a.H / a.Hkv, equal = sqrt(768. * 65536. / (rep * a.Hkv));
  const double L = equal < double(a.N) ? equal : double(a.N);
  const bool may = shared_form(uint64_t(L), uint64_t(L * L), a.H, a.Hkv);
  int32_t* form = may && a.cu != nullptr ? reinterpret_cast<int32_t*>(g.stats + 2 * a.N * a.H) : nullptr;
  const dim3 blocks(uint32_t(slot_blocks(grid, a.H) + tail_groups(a.N * a.H * D * 2)));
  attn_dq_kernel<D><<<blocks, dim3(kThreads), 0, stream>>>(
      static_cast<const bf16*>(a.q), static_cast<const bf16*>(a.k), static_cast<const bf16*>(a.v),
      static_cast<const bf16*>(a.o), static_cast<const bf16*>(g.dout), a.lse, a.cu, a.max_segs, a.N, a.H, a.Hkv,
      a.scale, static_cast<bf16*>(g.dq), g.stats, a.flags, form, grid);
  // With cu the lengths are on the device: both forms are launched, and the one
  // that was not chosen ends at once.
  const bool share = a.cu == nullptr && shared_form(a.N, uint64_t(a.N) * a.N, a.H, a.Hkv);
  if (form != nullptr || share) keys_pass<D, 4>(a, g, form, stream);
  if (!share) keys_pass<D, 1>(a, g, form, stream);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_bwd(const AttnArgs& a, const AttnGradArgs& g, hipStream_t stream) {
  if (a.window > 0 && a.window < a.N) return launch_attn_window_bwd(a, g, stream);
  return a.D == 64 ? run<64>(a, g, stream) : run<128>(a, g, stream);
}

}  // namespace pkv
