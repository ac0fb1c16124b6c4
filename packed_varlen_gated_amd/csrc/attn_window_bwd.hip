// Reverse pass of the packed causal softmax attention through a sliding window with sinks,
// on the matrix cores (bf16, D in {64, 128}).
//
// Query t of segment [a, e) sees key s <= t if t - s < window or s - a < sinks. The formulas
// and the two passes are those of attn_bwd.hip: the queries pass walks the tiles of WindowWalk
// (segments.h), the keys pass the queries up to `window` behind its keys, and a launch of its
// own between them takes the queries further behind that see the sinks (at FarGrid).
// Blocks that every row sees whole, most of a window's, have no comparisons, and dP begins
// from -delta in the keys pass. The loads' waits are written here (load_lds16_async).
//
// 8192 tokens (documents of about 800, the longest 3409), H 16, Hkv 4, D 128, window 512:
// queries 75, keys 86 us, of which 24 and 18 are the rows' own loads and stores (work-groups
// start and end together); matrix instructions in 28 and 33 % of the cycles, vector ones in
// as many, LDS reads in 15 and 22 %: a block's phases (products, weights, products) wait for
// one another, and registers allow two waves a SIMD. Left out in turn, the tiles' loads took
// 6 and 14 us, row-wise LDS reads 7 and 4, transposing ones 2 and 4, 2^x 3 and 4. 16384 tokens
// in one document, H 16, Hkv 16, D 64, window 256, 4 sinks: queries 64, far queries 29, keys
// 70 us, where 0.2, 0.07 and 0.2 GB take 39, 13 and 39 at a copy's rate.

#include "attn_grad.h"

namespace pkv {
namespace {

// (At D 64 the edges' comparisons do not fit the 128 registers of four waves a SIMD: 220 us
// the call with 13 of them in memory, 212 with three waves.)
template <int D>
__global__ __launch_bounds__(kThreads, D == 64 ? 3 : 2) void attn_window_dq_kernel(
    const bf16* __restrict__ q, const bf16* __restrict__ k, const bf16* __restrict__ v, const bf16* __restrict__ o,
    const bf16* __restrict__ dout, const float* __restrict__ lse, const int32_t* __restrict__ cu, int32_t max_segs,
    int64_t N, int32_t H, int32_t Hkv, float scale, bf16* __restrict__ dq, float* __restrict__ stats,
    int32_t* __restrict__ flags, SlotGrid grid, int32_t window, int32_t sinks) {
  constexpr int KS = D / 16, DT = D / 32, TB = Lds<D>::BYTES;
  __shared__ __attribute__((aligned(1024))) char lds[4 * TB];  // K, V of the even tiles, K, V of the odd ones

  const int64_t b = blockIdx.x;
  const int64_t blocks = slot_blocks(grid, H);
  if (b >= blocks) {
    const int64_t j = b - blocks, groups = gridDim.x - blocks;
    zero_tail(dq, covered_tokens(cu, max_segs, N), N, int64_t(H) * D * 2, j, groups);
    if (j == 0) check_cu(cu, max_segs, N, flags);
    return;
  }
  int32_t slot, h0, h1;
  slot_of(grid, b, H, slot, h0, h1);
  SegTile t;
  // late tiles have the most keys, up to a window of them: they start first
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
    const WindowWalk ww(window, sinks, kT, t.start, t.a);
    const int n_tiles = ww.count((qend - t.a + kT - 1) / kT);
    const Loader<D, kT, kThreads> ld(kstride, tid);
    auto issue = [&](int it) {
      const int32_t s0 = t.a + ww.tile(it) * kT;
      const int32_t n = t.e - s0 < kT ? t.e - s0 : kT;
      const int64_t at = (int64_t(s0) * Hkv + hk) * D, bytes = int64_t(n - 1) * kstride + D * 2;
      char* dst = lds + (it & 1) * 2 * TB;
      ld.issue_async(descriptor(k + at, bytes), dst, wave);
      ld.issue_async(descriptor(v + at, bytes), dst + TB, wave);
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
        for (int i = 0; i < 16; ++i) {
          const int32_t key = 8 * (i / 4) + i % 4, at = rd.col - 4 * rd.half;
          const bool sees = (key <= at) & ((key > at - window) | (key < sinks - 4 * rd.half));
          delta += sees ? ex2(fmaf(s[i], c, -lse2)) * dp[i] : 0.f;
        }
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
      const int32_t s0 = t.a + ww.tile(it) * kT;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (have == 0 || s0 + 32 * j > q0 + 31) continue;
        if (s0 + 32 * j + 31 <= q0 - window && s0 + 32 * j >= t.a + sinks) continue;
        f32x16 s = {}, dp = {};
#pragma unroll
        for (int i = 0; i < KS; ++i) {  // independent products take turns
          s = mfma32(rd.rows(kt, j, i), qf[i], s);
          dp = mfma32(rd.rows(vt, j, i), df[i], dp);
        }
        bf16x8 ds[2];
        // (blocks that every row sees whole, most of a window's, have no comparisons)
        auto weights = [&](auto sees) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float p = ex2(fmaf(s[i], c, -lse2));
            const float x = sees(8 * (i / 4) + i % 4) ? p * (dp[i] - delta) : 0.f;
            rest += x;
            ds[i / 8][i % 8] = static_cast<bf16>(x);
          }
        };
        const int32_t b0 = s0 + 32 * j;
        if (b0 + 31 <= q0 && b0 > q0 + 31 - window) {
          weights([](int32_t) { return true; });
        } else {
          // keys last + 1 .. are ahead, keys 0 .. old are behind the window, the first ones may be sinks
          const int32_t last = q0 + rd.col - b0 - 4 * rd.half, old = last - window;
          const int32_t sink = t.a + sinks - b0 - 4 * rd.half;
          weights([&](int32_t key) { return (key <= last) & ((key > old) | (key < sink)); });
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
    // (With its sign turned: that pass begins dP from it.)
    if (rd.half == 0 && rd.col < have) {
      stats[row] = lse2;
      stats[int64_t(H) * N + row] = -delta - rest;
    }
    __syncthreads();
    if (have > 0)
      store_rows<D>(acc, scale, lds + wave * (32 * D * 2), dq + (int64_t(q0) * H + h) * D, int64_t(H) * D, have, rd);
    if (hi + 1 < h1) __syncthreads();  // the outputs have left LDS
  }
}

// kQ waves share 32 keys and take the 32-query blocks of a tile in turn, their
// sums added at the end: kQ = 1, four waves hold 128 keys; kQ = 2, four hold 64;
// kQ = 4, eight waves hold 64.
template <int kQ>
struct DkvShape {
  static constexpr int NT = kQ == 4 ? 512 : 256;  // threads
  static constexpr int KEYS = NT / 64 / kQ * 32;  // keys of a work-group
  static constexpr int T = kQ == 4 ? 128 : 64;    // queries per tile
};

// The keys pass under a window. A key's queries end `window` tokens behind it, except
// a sink's, which go on to the segment's end: one work-group's walk over those would
// outlast all others, so the queries behind the window ("far") have a launch of their
// own before the keys pass. There a work-group takes the segment's sinks and a chunk of
// them and leaves its sums in the workspace; the keys pass adds a segment's in order.
// Far queries of segment i start at cu[i] + window; chunk c of them has slot
// floor(cu[i] / chunk) + inc i + c. With chunk <= window and inc = 0 the slots of
// different segments do not meet, since a segment of n tokens has at most
// floor((cu[i] + n) / chunk) - floor(cu[i] / chunk) of them; a window below 64 would make
// the chunks small and takes inc = 1 (one more slot per segment) instead. The chunks are
// 128 to 512 tokens, so that there are 512 work-groups if the call has that many: 8192
// tokens, H 16, Hkv 4, D 128, window 512, 4 sinks: 221 us the reverse pass in chunks of
// 512, 196 in chunks of 128; 16384 tokens: 388 and 371.
constexpr int kMaxSinks = 64;
struct FarGrid {
  int32_t chunk, inc;
  __host__ __device__ FarGrid(int64_t N, int32_t Hkv, int32_t window) {
    const int64_t want = N * Hkv / 512 / 128 * 128 + 128;
    chunk = want > 512 ? 512 : int32_t(want);
    inc = window < 64 ? 1 : 0;
    if (inc == 0 && chunk > window) chunk = window;
  }
  __host__ __device__ int64_t slots(int64_t N, int64_t max_segs) const { return N / chunk + inc * max_segs; }
};

// kFar: the sinks' far queries; else those of the window.
template <int D, int kQ, bool kFar>
__global__ __launch_bounds__(DkvShape<kQ>::NT, D == 64 && kQ == 1 ? 3 : 2) void attn_window_dkv_kernel(
    const bf16* __restrict__ q, const bf16* __restrict__ k, const bf16* __restrict__ v,
    const bf16* __restrict__ dout, const float* __restrict__ stats, const int32_t* __restrict__ cu,
    int32_t max_segs, int64_t N, int32_t H, int32_t Hkv, float scale, bf16* __restrict__ dk,
    bf16* __restrict__ dv, SlotGrid grid, int32_t window, int32_t sinks,
    float* __restrict__ far) {
  static_assert(!kFar || DkvShape<kQ>::KEYS >= kMaxSinks, "a work-group has a segment's sinks");
  constexpr int KS = D / 16, DT = D / 32;
  constexpr int NT = DkvShape<kQ>::NT, T = DkvShape<kQ>::T, TB = T * D * 2;
  // Q, dO of the even tiles, of the odd ones; then lse log2 e and -delta of each
  __shared__ __attribute__((aligned(1024))) char lds[4 * TB + 4 * T * 4];

  const int64_t b = blockIdx.x;
  const FarGrid fg(N, Hkv, window);
  int32_t slot, h0, h1;
  SegTile t;
  int32_t from, to;  // the queries [from, to)
  if constexpr (kFar) {
    slot = int32_t(b / Hkv);
    h0 = int32_t(b % Hkv);
    h1 = h0 + 1;
    t = {0, 0, 0, int32_t(N)};
    if (cu != nullptr && (!find_segment(cu, max_segs, fg.chunk, fg.inc, slot, t.seg, t.a, t.e) ||
                          !segment_ok(t.seg, t.a, t.e, N)))
      return;
    const int64_t c0 = int64_t(t.a) + window + (int64_t(slot) - t.a / fg.chunk - int64_t(fg.inc) * t.seg) * fg.chunk;
    if (c0 >= t.e) return;
    t.start = t.a;
    from = int32_t(c0);
    to = t.e - from < fg.chunk ? t.e : from + fg.chunk;
  } else {
    const int64_t blocks = slot_blocks(grid, Hkv);
    if (b >= blocks) {
      const int64_t j = b - blocks, groups = gridDim.x - blocks, cov = covered_tokens(cu, max_segs, N);
      zero_tail(dk, cov, N, int64_t(Hkv) * D * 2, j, groups);
      zero_tail(dv, cov, N, int64_t(Hkv) * D * 2, j, groups);
      return;
    }
    slot_of(grid, b, Hkv, slot, h0, h1);
    if (!find_tile(cu, max_segs, N, DkvShape<kQ>::KEYS, slot, t)) return;
    from = t.start;
    to = t.e - t.start > DkvShape<kQ>::KEYS - 1 + window ? t.start + DkvShape<kQ>::KEYS - 1 + window : t.e;
  }
  const int32_t rep = H / Hkv;

  for (int32_t hk = h0; hk < h1; ++hk) {
    // (nothing that goes by the lane is kept from one head to the next)
    const int tid = fresh(threadIdx.x), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const Reader<D> rd(tid);
    const int32_t kstride = Hkv * D * 2, qstride = H * D * 2;
    const int32_t k0 = t.start + wave / kQ * 32;  // the wave's first key
    const int32_t kend = kFar && t.e - t.a > sinks ? t.a + sinks : t.e;
    const int32_t rows = kend - k0, have = rows < 0 ? 0 : (rows > 32 ? 32 : rows);
    const int per_head = (to - from + T - 1) / T, n_tiles = per_head * rep;
    const Loader<D, T, NT> ld(qstride, tid);
    int ih = hk * rep, iq = 0;  // query head and tile of the next load
    // Q, dO and the statistics of the next tile
    auto issue = [&](int it) {
      const int32_t s0 = from + iq * T, h = ih;
      const int32_t n = to - s0 < T ? to - s0 : T;
      const int64_t at = (int64_t(s0) * H + h) * D, bytes = int64_t(n - 1) * qstride + D * 2;
      char* dst = lds + (it & 1) * 2 * TB;
      ld.issue_async(descriptor(q + at, bytes), dst, wave);
      ld.issue_async(descriptor(dout + at, bytes), dst + TB, wave);
      if (wave < T / 32) {  // lse log2 e and -delta, 64 queries a wave
        const int w = wave / (T / 64), part = wave % (T / 64) * 64;
        load_lds4_async(descriptor(stats + (int64_t(w) * H + h) * N + s0, n * 4), uint32_t(part + lane) * 4,
                        lds_addr(lds) + 4 * TB + (((it & 1) * 2 + w) * T + part) * 4);
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
      const int32_t s0 = from + cq * T;
      if (++cq == per_head) cq = 0;
#pragma unroll 1
      for (int j = wave % kQ; j < T / 32; j += kQ) {
        const int32_t b0 = s0 + 32 * j;  // first query of the block
        // (addresses are formed per block: one register each instead of one per read)
        const uint32_t qt = fresh_uniform(qt0 + 32 * j * Lds<D>::ROW), ot = qt + TB;
        const int32_t kq = kFar ? k0 + window : k0;  // the first key's first query
        if (have == 0 || b0 + 31 < kq || b0 >= to) continue;
        if (!kFar && b0 >= k0 + 31 + window) continue;
        // Registers are full at D = 128 (k, v, dk and dv take 192; 5 to 8 of the others
        // are in memory): the weights are done with before dP is begun, and nothing of a
        // phase starts early. The other wave of the SIMD fills the gaps.
        bf16x8 p[2], ds[2];
        f32x16 x = {};
#pragma unroll
        for (int i = 0; i < KS; ++i) x = mfma32(rd.rows(qt, 0, i), kf[i], x);
        if (D == 128) __builtin_amdgcn_sched_barrier(0);
        // the lane's key takes part in the block's queries first .. end - 1
        const bool edge = b0 < kq + 31 || b0 + 32 > to || (!kFar && b0 + 32 > k0 + window);
        const int32_t first = edge ? kq + rd.col - b0 - 4 * rd.half : -64;
        const int32_t qend = !kFar && to - k0 > rd.col + window ? k0 + rd.col + window : to;
        const int32_t end = edge ? qend - b0 - 4 * rd.half : 64;
        auto weights = [&](auto sees) {
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            const f32x4 l4 = ls[8 * j + 2 * i4 + rd.half];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int i = 4 * i4 + e;
              const float y = ex2(fmaf(x[i], c, -l4[e]));
              x[i] = sees(8 * i4 + e) ? y : 0.f;
              p[i / 8][i % 8] = static_cast<bf16>(x[i]);
            }
          }
        };
        if (!edge)
          weights([](int32_t) { return true; });
        else
          weights([&](int32_t r) { return (r >= first) & (r < end); });
        if (D == 128) __builtin_amdgcn_sched_barrier(0);
        f32x16 dp;  // from -delta on
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) {
          const f32x4 d4 = dl[8 * j + 2 * i4 + rd.half];
#pragma unroll
          for (int e = 0; e < 4; ++e) dp[4 * i4 + e] = d4[e];
        }
#pragma unroll
        for (int i = 0; i < KS; ++i) dp = mfma32(rd.rows(ot, 0, i), vf[i], dp);
        if (D == 128) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < 16; ++i) ds[i / 8][i % 8] = static_cast<bf16>(x[i] * dp[i]);
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
    if constexpr (kFar) {
      if (rd.col < have && wave % kQ == 0) {
        float* out = far + ((int64_t(slot) * Hkv + hk) * 2 * sinks + (k0 - t.a) + rd.col) * D + 4 * rd.half;
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float* x = out + 32 * i + 8 * j;
            *reinterpret_cast<f32x4*>(x) = f32x4{ak[i][4 * j], ak[i][4 * j + 1], ak[i][4 * j + 2], ak[i][4 * j + 3]};
            *reinterpret_cast<f32x4*>(x + int64_t(sinks) * D) =
                f32x4{av[i][4 * j], av[i][4 * j + 1], av[i][4 * j + 2], av[i][4 * j + 3]};
          }
      }
      return;
    }
    if (!kFar && far != nullptr && t.start == t.a && t.e - t.a > window) {
      // The sinks' sums over the far queries: every thread sums 4 channels of a sink over
      // the chunks, the loads of 8 going out together.
      static_assert(4 * TB >= 2 * kMaxSinks * D * 4 || kFar, "the far sums fit the tiles' buffers");
      f32x4* fs = reinterpret_cast<f32x4*>(lds);  // dk, dv of [sink][D / 4]
      const int64_t first = int64_t(t.a) / fg.chunk + int64_t(fg.inc) * t.seg;
      const int32_t chunks = (t.e - t.a - window + fg.chunk - 1) / fg.chunk;
      const int64_t step = int64_t(Hkv) * 2 * sinks * (D / 4);
      if (kQ == 1) __syncthreads();  // every wave is done with the tiles
      for (int i = tid; i < 2 * sinks * (D / 4); i += NT) {
        const f32x4* part = reinterpret_cast<const f32x4*>(far) + (first * Hkv + hk) * 2 * sinks * (D / 4) + i;
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
        for (int32_t c0 = 0; c0 < chunks; c0 += 8) {
          f32x4 y[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) y[u] = part[(c0 + u < chunks ? c0 + u : c0) * step];
#pragma unroll
          for (int u = 0; u < 8; ++u) x += c0 + u < chunks ? y[u] : f32x4{0.f, 0.f, 0.f, 0.f};
        }
        fs[i] = x;
      }
      __syncthreads();
      const int key = k0 - t.a + rd.col;
      if (key < sinks && wave % kQ == 0) {
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x4 y = fs[key * (D / 4) + 8 * i + 2 * j + rd.half];
            const f32x4 z = fs[(sinks + key) * (D / 4) + 8 * i + 2 * j + rd.half];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              ak[i][4 * j + e] += y[e];
              av[i][4 * j + e] += z[e];
            }
          }
      }
      __syncthreads();
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
void keys_pass(const AttnArgs& a, const AttnGradArgs& g, hipStream_t stream) {
  const SlotGrid grid = slot_grid(a.N, a.max_segs, DkvShape<kQ>::KEYS);
  const dim3 blocks(uint32_t(slot_blocks(grid, a.Hkv) + tail_groups(a.N * a.Hkv * D * 2)));
  attn_window_dkv_kernel<D, kQ, false><<<blocks, dim3(DkvShape<kQ>::NT), 0, stream>>>(
      static_cast<const bf16*>(a.q), static_cast<const bf16*>(a.k), static_cast<const bf16*>(a.v),
      static_cast<const bf16*>(g.dout), g.stats, a.cu, a.max_segs, a.N, a.H, a.Hkv, a.scale,
      static_cast<bf16*>(g.dk), static_cast<bf16*>(g.dv), grid, a.window, a.sinks, g.far);
}

// The queries pass, the sinks' far queries, the keys pass.
template <int D>
hipError_t run(const AttnArgs& a, const AttnGradArgs& g, hipStream_t stream) {
  const SlotGrid grid = slot_grid(a.N, a.max_segs, kB);
  const dim3 blocks(uint32_t(slot_blocks(grid, a.H) + tail_groups(a.N * a.H * D * 2)));
  attn_window_dq_kernel<D><<<blocks, dim3(kThreads), 0, stream>>>(
      static_cast<const bf16*>(a.q), static_cast<const bf16*>(a.k), static_cast<const bf16*>(a.v),
      static_cast<const bf16*>(a.o), static_cast<const bf16*>(g.dout), a.lse, a.cu, a.max_segs, a.N, a.H, a.Hkv,
      a.scale, static_cast<bf16*>(g.dq), g.stats, a.flags, grid, a.window, a.sinks);
  const int64_t far = a.sinks > 0 ? FarGrid(a.N, a.Hkv, a.window).slots(a.N, a.max_segs) * a.Hkv : 0;
  if (far > 0)
    attn_window_dkv_kernel<D, 4, true><<<dim3(uint32_t(far)), dim3(DkvShape<4>::NT), 0, stream>>>(
        static_cast<const bf16*>(a.q), static_cast<const bf16*>(a.k), static_cast<const bf16*>(a.v),
        static_cast<const bf16*>(g.dout), g.stats, a.cu, a.max_segs, a.N, a.H, a.Hkv, a.scale, nullptr, nullptr,
        grid, a.window, a.sinks, g.far);
  // Few keys leave most of the chip without work unless waves share them. kQ = 1 / 2 / 4,
  // the whole reverse pass, window 512, H 16, Hkv 4 but where said:
  //   65536 tokens, H 32, Hkv 8, D 128, window 1024 (4096 work-groups of 128 keys)  3686 / 3713 / 4127 us
  //   16384, Hkv 16, D 64, window 256 (2048)                                         181 / 187 / 294
  //   16384, D 128, window 1024 (512)                                                638 / 610 / 675
  //   16384, D 64 (512)                                                              208 / 208 / 246
  //   8192, D 128 (256)                                                              217 / 172 / 191
  //   2048, H 8, Hkv 8, D 64, window 256 (128)                                        36 / 29 / 30
  //   4096, H 8, Hkv 1, D 128, window 2048 (32)                                      952 / 563 / 384
  const int64_t keys = (a.N + 127) / 128 * a.Hkv;
  if (keys > 512)
    keys_pass<D, 1>(a, g, stream);
  else if (keys > 64)
    keys_pass<D, 2>(a, g, stream);
  else
    keys_pass<D, 4>(a, g, stream);
  return hipGetLastError();
}

}  // namespace

size_t attn_far_bytes(int64_t N, int64_t max_segs, int32_t Hkv, int32_t D, int32_t window, int32_t sinks) {
  if (sinks == 0 || window >= N) return 0;
  return size_t(FarGrid(N, Hkv, window).slots(N, max_segs)) * Hkv * 2 * sinks * D * 4;
}

hipError_t launch_attn_window_bwd(const AttnArgs& a, const AttnGradArgs& g, hipStream_t stream) {
  return a.D == 64 ? run<64>(a, g, stream) : run<128>(a, g, stream);
}

}  // namespace pkv
