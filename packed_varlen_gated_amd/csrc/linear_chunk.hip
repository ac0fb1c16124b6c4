// Packed linear attention with one decay per head in chunks of 32 tokens on the
// matrix cores (bf16, head dimensions 64 and 128).
//
//   S_t = lam S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t,  lam = e^{g_h}
//
// One walk serves the forward pass and the three gradients (roles (a, b, c) and
// directions as in linear_serial.hip). Over a chunk of n tokens, forward
// (backward: the two powers change places and the mask is s >= t):
//   out_t = sum_{s <= t} lam^(t - s) (a_t.b_s) c_s + lam^(t + 1) X^T a_t
//   X <- lam^n X + sum_s lam^(n - 1 - s) b_s c_s^T
// A team of DB / 32 waves takes one run (up to `run` tokens of a segment) of one
// head; a wave owns 32 columns of X, in fp32 registers, and of the output. The
// in-chunk weights are formed in 16-token blocks, a block of columns per wave,
// and shared through LDS as bf16. X is rounded to bf16 once, as the operand of
// the readout; the update's decayed c is split into three bf16 parts (24 bits) so
// that X itself, an fp32 result, sees no bf16 rounding.
//
// Rows and columns of X are dealt to the registers so that 8 consecutive ones
// are 8 consecutive registers of a lane (the transposing LDS reads take their
// 8-byte pieces in the order 0, 2, 1, 3): a is read in 16-byte pieces, outputs
// are stored in 16-byte pieces.
//
// Tiles go from memory into LDS without passing registers, the next chunk's while
// this one is used. A chunk is a chain of dependent steps (LDS reads, products,
// a barrier, products, the update), so what counts is how many work-groups take
// turns: two stages of 24 KiB at 128 channels and at most 168 registers, three
// work-groups per compute unit. Backward, dk and dv walk together where Dk = Dv:
// two teams in a work-group, q and do (b of one, c of the other) loaded once.
//
// Segments longer than a run: a first launch walks every run but the segment's
// last (in the walk's direction) without outputs and saves its own end state, a
// second one turns these into the states before each run, and the walk starts
// from those; the reverse pass does both directions in one launch each. A run's
// length depends on the call's sizes only.
//
// Bound by the chain of dependent steps of a chunk: the walk of 65536 tokens, H 32,
// D 128 takes 585 us for 2.15 GB (413 us at a copy's rate), waiting 51 % of its
// cycles, behind 159 us of run states and 20 us of their scan, over 8 calls under the
// profiler; in a timed loop the call takes 0.680-0.688 ms (0.660 with two parts in the
// update, 2^-17). With 64-token
// chunks the walk of two parts took 682 us, with three stages and two work-groups per
// compute unit 622, with the update before the middle barrier 578 instead of 562.
// 32768 tokens in one segment, H 16, with states: 75 + 23 + 130 us. 8192 tokens,
// H 16, forward and reverse: 0.264 ms in seven launches. 32768 tokens in documents
// of about 104, H 32, D 64: walks of 164, 164 and 217 us.

#include "mfma.h"
#include "segments.h"

namespace pkv {
namespace {

constexpr int kC = 32;       // tokens per chunk of a walk
constexpr int kCState = 64;  // ... of a state walk
constexpr int kParts = 3;    // bf16 parts of the update's c

template <int D>
struct Rows {  // an LDS tile of a chunk's rows of D channels
  static constexpr int CH = D / 8, ROW = D * 2;
  static __device__ __forceinline__ int swz(int row) {
    return D == 128 ? ((row & 3) << 2) | ((row >> 2) & 3) : ((row & 2) << 1) | ((row >> 2) & 3);
  }
};

template <int D, int C, int NT>
__device__ __forceinline__ void issue_tile(__amdgpu_buffer_rsrc_t r, int32_t stride, char* dst, int wave) {
  constexpr int STEP = NT / Rows<D>::CH;
  const int row = fresh(threadIdx.x) / Rows<D>::CH, pos = threadIdx.x % Rows<D>::CH;
#pragma unroll
  for (int i = 0; i < C / STEP; ++i) {
    const int s = STEP % 16 == 0 ? Rows<D>::swz(row) : Rows<D>::swz(row + i * STEP);
    load_lds16(r, uint32_t(row + i * STEP) * stride + (pos ^ s) * 16, dst + wave * 1024 + i * NT * 16);
  }
}

// 32 rows of 16-row step j, channels 32 i + (lane's) in the register order above.
template <int D>
struct Transposed {
  int at[2], ch[2];
  __device__ __forceinline__ Transposed(int lane) {
    const int r = 4 * (lane >> 5) + ((lane & 15) >> 2);
    const int c = ((lane >> 4) & 1) * 2 + (lane & 1);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      at[u] = (r + 8 * u) * Rows<D>::ROW + ((lane >> 1) & 1) * 8;
      ch[u] = c ^ Rows<D>::swz(r + 8 * u);
    }
  }
  __device__ __forceinline__ bf16x8 read(const char* t, int i, int j) const {
    const char* p = t + 16 * j * Rows<D>::ROW;
    return join(read_tr(p + at[0] + ((4 * i) ^ ch[0]) * 16), read_tr(p + at[1] + ((4 * i) ^ ch[1]) * 16));
  }
};

struct Role {
  const bf16 *a, *b, *c;
  bf16* out;
  const float* init;  // [max_segs, H, ..] or null
  float* saved;       // [N / run, H, ..]: states between runs
  float* fin;         // [max_segs, H, ..] or null
  float in_scale, out_scale;
  bool transposed;  // states are [DB][DA] in memory
};
struct WalkArgs {
  Role r[2];
  const float* g;
  const int32_t* cu;
  int32_t max_segs;
  int64_t N;
  int32_t H, run;
  SlotGrid grid;
  int32_t* flags;
};

// The log decay in base 2; one of -inf (nothing is kept) stays finite, since it is
// multiplied by distances of 0.
__device__ __forceinline__ float log2_decay(float g) {
  const float x = g * kLog2e;
  return x < -1e30f ? -1e30f : x;
}

// X of one (state, head) <-> registers: register 8 v + j of tile i is row
// 32 i + 16 v + 8 (lane / 32) + j of the lane's column. One address register;
// the rest of an offset is an immediate or a scalar.
template <int DA, int DB>
struct StateAddr {
  __amdgpu_buffer_rsrc_t r;
  uint32_t off;
  bool transposed;
  __device__ __forceinline__ StateAddr(const float* p, bool transposed, int tid) : transposed(transposed) {
    const int l = tid & 31, half = (tid >> 5) & 1;
    const int e = 32 * (tid >> 6) + (l & 16) + ((l & 4) << 1) + ((l & 8) >> 1) + (l & 3);
    r = buffer(p, int64_t(DA) * DB * 4);
    off = 4 * (transposed ? e * DA + 8 * half : 8 * half * DB + e);
  }
  __device__ __forceinline__ void load(f32x16 (&X)[DA / 32]) const {
    if (transposed) {
#pragma unroll
      for (int i = 0; i < DA / 32; ++i)
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const auto x = __builtin_bit_cast(
              f32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off + 4 * (32 * i + 2 * (j & 8) + (j & 7)), 0, 0));
#pragma unroll
          for (int e = 0; e < 4; ++e) X[i][j + e] = x[e];
        }
    } else {
#pragma unroll
      for (int i = 0; i < DA / 32; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j)
          X[i][j] = __builtin_bit_cast(
              float, __builtin_amdgcn_raw_buffer_load_b32(r, off, 4 * DB * (32 * i + 2 * (j & 8) + (j & 7)), 0));
    }
  }
  __device__ __forceinline__ void store(const f32x16 (&X)[DA / 32]) const {
    if (transposed) {
#pragma unroll
      for (int i = 0; i < DA / 32; ++i)
#pragma unroll
        for (int j = 0; j < 16; j += 4)
          store16(r, off + 4 * (32 * i + 2 * (j & 8) + (j & 7)),
                  __builtin_bit_cast(i32x4, f32x4{X[i][j], X[i][j + 1], X[i][j + 2], X[i][j + 3]}));
    } else {
#pragma unroll
      for (int i = 0; i < DA / 32; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j)
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_int(X[i][j]), r, off,
                                                4 * DB * (32 * i + 2 * (j & 8) + (j & 7)), 0);
    }
  }
};

// Saved state j of a segment whose first token is a has index a / run + j: a
// segment of m runs has m - 1, and no two share an index. Forward it is the
// state after run j, backward after run j + 1. The segment is the last one with
// cu[i] / run <= index: those before it with the same quotient are shorter than
// a run.
template <bool kRev>
__device__ __forceinline__ bool find_saved(const int32_t* __restrict__ cu, int32_t max_segs, int64_t N, int32_t run,
                                           int32_t idx, SegTile& t) {
  t.seg = 0;
  t.a = 0;
  t.e = int32_t(N);
  if (cu != nullptr && !find_segment(cu, max_segs, run, 0, idx, t.seg, t.a, t.e)) return false;
  if (!segment_ok(t.seg, t.a, t.e, N)) return false;
  const int64_t j = idx - t.a / run, m = (int64_t(t.e) - t.a + run - 1) / run;
  if (j < 0 || j >= m - 1) return false;
  t.start = int32_t(t.a + (kRev ? j + 1 : j) * run);
  return true;
}

// The update: X <- carry X + sum_s w_s b_s c_s^T from a chunk's tiles.
template <int DA, int C>
__device__ __forceinline__ void update(f32x16 (&X)[DA / 32], float carry, const bf16x8 (&cf)[C / 16], const float* w, int half,
                                       const Transposed<DA>& tb, const char* bt) {
  constexpr int TA = DA / 32;
#pragma unroll
  for (int i = 0; i < TA; ++i)
#pragma unroll
    for (int j = 0; j < 16; ++j) X[i][j] *= carry;
#pragma unroll
  for (int j = 0; j < C / 16; ++j) {
    bf16x8 part[kParts];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const f32x4 ws = *reinterpret_cast<const f32x4*>(w + 16 * j + 8 * u + 4 * half);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float y = to_f32(cf[j][4 * u + e]) * ws[e];
#pragma unroll
        for (int s = 0; s < kParts; ++s) {
          const bf16 r = static_cast<bf16>(y);
          part[s][4 * u + e] = r;
          y -= to_f32(r);
        }
      }
    }
    bf16x8 bT[TA];
#pragma unroll
    for (int i = 0; i < TA; ++i) bT[i] = tb.read(bt, i, j);
#pragma unroll
    for (int s = 0; s < kParts; ++s)
#pragma unroll
      for (int i = 0; i < TA; ++i) X[i] = mfma32(bT[i], part[s], X[i]);
  }
}

// What a team knows of its run.
template <int C, bool kRev>
struct Run {
  int32_t start, end;
  int n_chunks;
  __device__ __forceinline__ int32_t chunk(int i) const { return start + (kRev ? n_chunks - 1 - i : i) * C; }
  __device__ __forceinline__ int32_t len(int32_t s0) const { return end - s0 < C ? end - s0 : C; }
};

// A tile of a chunk's rows [s0, s0 + n) of head h, into dst.
template <int D, int C, int NT>
__device__ __forceinline__ void issue_rows(const bf16* p, int32_t s0, int32_t n, int32_t H, int32_t h, char* dst,
                                           int wave) {
  const int32_t stride = H * D * 2;
  issue_tile<D, C, NT>(buffer(p + (int64_t(s0) * H + h) * D, int64_t(n - 1) * stride + D * 2), stride, dst, wave);
}

template <bool kRev>
__device__ __forceinline__ float update_weight(float scale, float g2, int s, int32_t n) {
  return s < n ? scale * ex2(g2 * (kRev ? s + 1 : n - 1 - s)) : 0.f;
}

// The state walk of one run: block blk of saved states x heads.
template <int DA, int DB, bool kRev>
__device__ __forceinline__ void state_walk(const WalkArgs& x, const Role& R, int64_t blk, char* lds, float* upd) {
  constexpr int C = kCState, NT = 2 * DB, TA = DA / 32, SB = C * DA * 2, SC = C * DB * 2;
  const int32_t h = int32_t(blk % x.H), idx = int32_t(blk / x.H);
  SegTile t;
  if (!find_saved<kRev>(x.cu, x.max_segs, x.N, x.run, idx, t)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  Run<C, kRev> run;
  run.start = t.start;
  run.end = t.e - t.start > x.run ? t.start + x.run : t.e;
  run.n_chunks = (run.end - run.start + C - 1) / C;
  const float g2 = log2_decay(x.g[h]);
  auto issue = [&](int i) {
    const int32_t s0 = run.chunk(i), n = run.len(s0), stage = i & 1;
    char* dst = lds + stage * (SB + SC);
    issue_rows<DA, C, NT>(R.b, s0, n, x.H, h, dst, wave);
    issue_rows<DB, C, NT>(R.c, s0, n, x.H, h, dst + SB, wave);
    if (tid < C) upd[stage * C + tid] = update_weight<kRev>(R.in_scale, g2, tid, n);
  };
  // chunks whose tokens decay to a weight that fp32 has only 0 for (2^-150) by
  // the run's end are left out
  const float far = g2 < 0.f ? fminf(150.f / (-C * g2), 1e6f) : 1e6f;
  int it = run.n_chunks - 1 - int(far);
  it = it < 0 ? 0 : it;
  issue(it);
  f32x16 X[TA];
#pragma unroll
  for (int i = 0; i < TA; ++i) X[i] = f32x16{};
  const Transposed<DA> tb(lane);
  const Transposed<DB> tc(lane);
  for (; it < run.n_chunks; ++it) {
    wait_all();
    bar();
    if (it + 1 < run.n_chunks) issue(it + 1);
    const char* bt = lds + (it & 1) * (SB + SC);
    bf16x8 cf[C / 16];
#pragma unroll
    for (int j = 0; j < C / 16; ++j) cf[j] = tc.read(bt + SB, wave, j);
    update<DA, C>(X, ex2(g2 * run.len(run.chunk(it))), cf, upd + (it & 1) * C, lane >> 5, tb, bt);
  }
  StateAddr<DA, DB>(R.saved + (int64_t(idx) * x.H + h) * DA * DB, R.transposed, tid).store(X);
}

// Role 0 forward and, with kBoth, role 1 backward.
template <int DA, int DB, bool kBoth>
__global__ __launch_bounds__(2 * DB, 3) void linear_state_kernel(const WalkArgs x) {
  __shared__ __attribute__((aligned(1024))) char lds[2 * kCState * (DA + DB) * 2];
  __shared__ __attribute__((aligned(16))) float upd[2 * kCState];
  const int64_t n = x.N / x.run * x.H, blk = blockIdx.x;
  if (!kBoth || blk < n)
    state_walk<DA, DB, false>(x, x.r[0], blk, lds, upd);
  else
    state_walk<DA, DB, true>(x, x.r[1], blk - n, lds, upd);
}

template <int DA, int DB, bool kRev, bool kPair>
__global__ __launch_bounds__((kPair ? 4 : 2) * DB, kPair ? 2 : 3) void linear_walk_kernel(const WalkArgs x) {
  constexpr int NW = DB / 32, NT = (kPair ? 2 : 1) * 64 * NW, KA = DA / 16, TA = DA / 32;
  constexpr int SB = kC * DA * 2, SC = kC * DB * 2;
  static_assert(!kPair || DA == DB, "a team's b is the other one's c");
  // a stage: a, b and c of a team; of two, a and b of each (a team's c is the
  // other one's b)
  constexpr int kStage = kPair ? 4 * SB : 2 * SB + SC;
  constexpr int kStores = 2;  // of a chunk's outputs, per lane
  __shared__ __attribute__((aligned(1024))) char lds[2 * kStage];
  constexpr int WP = kC + 8;  // row of the in-chunk weights [t][s]
  __shared__ __attribute__((aligned(16))) bf16 wts[kPair ? 2 : 1][kC][WP];
  __shared__ __attribute__((aligned(16))) float upd[2][kC];

  const int64_t blk = blockIdx.x;
  if (blk >= slot_blocks(x.grid, x.H)) {
    const int64_t j = blk - slot_blocks(x.grid, x.H), groups = gridDim.x - slot_blocks(x.grid, x.H);
    const int64_t cov = covered_tokens(x.cu, x.max_segs, x.N);
#pragma unroll
    for (int i = 0; i < (kPair ? 2 : 1); ++i) zero_tail(x.r[i].out, cov, x.N, int64_t(x.H) * DB * 2, j, groups);
    if (j == 0) check_cu(x.cu, x.max_segs, x.N, x.flags);
    if (x.r[0].fin != nullptr && x.cu != nullptr) {
      // empty slots keep their initial state (or 0)
      const int64_t n = int64_t(x.H) * DA * DB / 4;
      for (int64_t s = j; s < x.max_segs; s += groups) {
        if (x.cu[s] != x.cu[s + 1]) continue;
        f32x4* to = reinterpret_cast<f32x4*>(x.r[0].fin) + s * n;
        const f32x4* from = x.r[0].init ? reinterpret_cast<const f32x4*>(x.r[0].init) + s * n : nullptr;
        for (int64_t i = threadIdx.x; i < n; i += NT) to[i] = from ? from[i] : f32x4{0.f, 0.f, 0.f, 0.f};
      }
    }
    return;
  }
  int32_t slot, h0, h1;
  SegTile t;
  slot_of(x.grid, blk, x.H, slot, h0, h1);
  if (!find_tile(x.cu, x.max_segs, x.N, x.run, slot, t)) return;
  Run<kC, kRev> run;
  run.start = t.start;
  run.end = t.e - t.start > x.run ? t.start + x.run : t.e;
  run.n_chunks = (run.end - run.start + kC - 1) / kC;
  const bool first = kRev ? run.end == t.e : t.start == t.a;  // in the walk's direction
  const bool last = kRev ? t.start == t.a : run.end == t.e;
  // the saved state that this run starts from
  const int64_t at = int64_t(t.a / x.run) + (t.start - t.a) / x.run - (kRev ? 0 : 1);

  for (int32_t h = h0; h < h1; ++h) {
    // (nothing that goes by the lane is kept from one head to the next)
    const int tid = fresh(threadIdx.x), lane = tid & 63, wave_ = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int team = kPair ? wave_ / NW : 0, wave = kPair ? wave_ % NW : wave_;
    const Role& R = x.r[team];
    if (h != h0) __syncthreads();  // the last head is done with LDS
    const float g2 = log2_decay(x.g[h]);
    const int half = lane >> 5, col = lane & 31;
    const int32_t cs = x.H * DB * 2;
    auto issue = [&](int i) {
      const int32_t s0 = run.chunk(i), n = run.len(s0), stage = i & 1;
      char* dst = lds + stage * kStage;
      issue_rows<DA, kC, NT>(x.r[0].a, s0, n, x.H, h, dst, wave_);
      issue_rows<DA, kC, NT>(x.r[0].b, s0, n, x.H, h, dst + SB, wave_);
      if constexpr (kPair) {
        issue_rows<DA, kC, NT>(x.r[1].a, s0, n, x.H, h, dst + 2 * SB, wave_);
        issue_rows<DA, kC, NT>(x.r[1].b, s0, n, x.H, h, dst + 3 * SB, wave_);
      } else {
        issue_rows<DB, kC, NT>(x.r[0].c, s0, n, x.H, h, dst + 2 * SB, wave_);
      }
      if (tid < kC) upd[stage][tid] = update_weight<kRev>(x.r[0].in_scale, g2, tid, n);
    };
    issue(0);

    f32x16 X[TA];
    const float* from = first ? (R.init ? R.init + (int64_t(t.seg) * x.H + h) * DA * DB : nullptr)
                              : R.saved + (at * x.H + h) * DA * DB;
    if (from != nullptr) {
      StateAddr<DA, DB>(from, R.transposed, tid - team * 64 * NW).load(X);
    } else {
#pragma unroll
      for (int i = 0; i < TA; ++i) X[i] = f32x16{};
    }

    // In-chunk weights of the lane: column t = lane % 16 of a 16-token block,
    // rows s = 4 (lane / 16) + e; near: of a block on the diagonal, next: of the
    // block beside it.
    const int c16 = lane & 15, r16 = lane >> 4;
    f32x4 near, next;
    const float both = R.in_scale * R.out_scale;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int d = kRev ? 4 * r16 + e - c16 : c16 - 4 * r16 - e;
      near[e] = d >= 0 ? both * ex2(g2 * d) : 0.f;
      next[e] = both * ex2(g2 * (d + 16));
    }
    bf16* wt = &wts[team][0][0];
    // the block that never has any
    if (wave == NW - 1)
      *reinterpret_cast<uint64_t*>(wt + (16 * (kRev ? 1 : 0) + c16) * WP + 16 * (kRev ? 0 : 1) + 4 * r16) = 0;
    const Transposed<DA> tb(lane);
    const Transposed<DB> tc(lane);

    for (int it = 0; it < run.n_chunks; ++it) {
      // This chunk has come; the last chunk's outputs, stored after it was asked
      // for, may be on their way (the counter is in order).
      if (it == 0)
        wait_all();
      else
        wait_loads<kStores>();
      bar();
      if (it + 1 < run.n_chunks) issue(it + 1);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      const char* st = lds + (it & 1) * kStage;
      const char* at_ = st + (kPair ? 2 * team * SB : 0);
      const char* bt = at_ + SB;
      const char* ct = st + (kPair ? (3 - 2 * team) * SB : 2 * SB);
      const int32_t s0 = run.chunk(it), n = run.len(s0);

      // in-chunk weights: three blocks of 16 x 16, one or two a wave
#pragma unroll
      for (int v = 0; v < (3 + NW - 1) / NW; ++v) {
        const int blk16 = wave + v * NW;  // 0, 1: on the diagonal, 2: beside it
        if (blk16 > 2) continue;
        const int cb = blk16 < 2 ? blk16 : (kRev ? 0 : 1), sb = blk16 < 2 ? blk16 : (kRev ? 1 : 0);
        f32x4 w = {};
#pragma unroll
        for (int i = 0; i < DA / 32; ++i) {
          auto row = [&](const char* tile, int b16) {
            return *reinterpret_cast<const bf16x8*>(tile + (16 * b16 + c16) * Rows<DA>::ROW +
                                                    (((4 * i + r16) ^ Rows<DA>::swz(c16)) * 16));
          };
          w = mfma16(row(bt, sb), row(at_, cb), w);
        }
        bf16x4 y;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = static_cast<bf16>(w[e] * (blk16 < 2 ? near[e] : next[e]));
        *reinterpret_cast<bf16x4*>(wt + (16 * cb + c16) * WP + 16 * sb + 4 * r16) = y;
      }
      // readout of X, in two chains
      f32x16 o = {}, o2 = {};
#pragma unroll
      for (int i = 0; i < KA; ++i) {
        bf16x8 xs;
#pragma unroll
        for (int j = 0; j < 8; ++j) xs[j] = static_cast<bf16>(X[i / 2][8 * (i % 2) + j]);
        const bf16x8 a = *reinterpret_cast<const bf16x8*>(at_ + col * Rows<DA>::ROW +
                                                          (((2 * i + half) ^ Rows<DA>::swz(col)) * 16));
        if (i % 2 == 0)
          o = mfma32(xs, a, o);
        else
          o2 = mfma32(xs, a, o2);
      }
      __builtin_amdgcn_s_waitcnt(0xC07F);  // LDS stores
      bar();                               // the weights are in LDS
      bf16x8 cf[kC / 16];
#pragma unroll
      for (int j = 0; j < kC / 16; ++j) cf[j] = tc.read(ct, wave, j);
      const int d = kRev ? n - 1 - col : col + 1;
      const float ow = R.out_scale * ex2(g2 * (d < 0 ? 0 : d));
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] = (o[i] + o2[i]) * ow;
#pragma unroll
      for (int j = 0; j < kC / 16; ++j) {
        const bf16* p = wt + col * WP + 16 * j + 4 * half;
        o = mfma32(cf[j], join(*reinterpret_cast<const s16x4*>(p), *reinterpret_cast<const s16x4*>(p + 8)), o);
      }
      // (rows past the chunk's end are out of the buffer's range)
      const auto ro = buffer(R.out + (int64_t(s0) * x.H + h) * DB, int64_t(n - 1) * cs + DB * 2);
#pragma unroll
      for (int v = 0; v < kStores; ++v) {
        bf16x8 y;
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = static_cast<bf16>(o[8 * v + j]);
        store16(ro, uint32_t(col) * cs + 64 * wave + 16 * half + 32 * v, __builtin_bit_cast(i32x4, y));
      }
      __builtin_amdgcn_sched_barrier(0);
      update<DA, kC>(X, ex2(g2 * n), cf, upd[(it & 1)], half, tb, bt);
    }

    if (last && R.fin != nullptr)
      StateAddr<DA, DB>(R.fin + (int64_t(t.seg) * x.H + h) * DA * DB, R.transposed, tid - team * 64 * NW).store(X);
  }
}

// The saved states, each its run's own end state, become the states that the
// walk has there: X <- own + lam^(run's tokens) X, X = init before a segment's
// first run. A work-group takes 256 x 4 elements of one head through all indices
// in order.
constexpr int kScan = 256;
constexpr int kAhead = 8;  // states whose loads are in flight at once

template <bool kRev>
__device__ __forceinline__ void scan(const WalkArgs& x, const Role& R, int32_t blk, int32_t size, int32_t count,
                                     int32_t* seg_of, float* decay) {
  // seg_of: segment of the index if it starts the walk there, -1 if it goes on, -2 if unused
  const int tid = threadIdx.x;
  const int32_t parts = size / (4 * kScan), h = blk / parts;
  const int64_t elem = (int64_t(blk % parts) * kScan + tid) * 4;
  const float g2 = log2_decay(x.g[h]);
  f32x4 X = {0.f, 0.f, 0.f, 0.f};
  for (int32_t base = 0; base < count; base += kScan) {
    const int32_t n = count - base < kScan ? count - base : kScan;
    __syncthreads();
    if (tid < n) {
      const int32_t idx = kRev ? count - 1 - (base + tid) : base + tid;
      // the last segment i with cu[i] / run <= idx: those before it with the same
      // quotient are shorter than a run
      int32_t lo = 0, hi = x.max_segs;
      if (x.cu != nullptr)
        while (hi - lo > 1) {
          const int32_t mid = lo + (hi - lo) / 2, c = x.cu[mid];
          if ((c < 0 ? 0 : c / x.run) <= idx) lo = mid; else hi = mid;
        }
      const int64_t a = x.cu ? x.cu[lo] : 0, e = x.cu ? x.cu[lo + 1] : x.N;
      int32_t s = -2;
      float d = 0.f;
      if (segment_ok(lo, a, e, x.N)) {
        const int64_t j = idx - a / x.run, m = (e - a + x.run - 1) / x.run;
        if (j >= 0 && j < m - 1) {
          const bool starts = kRev ? j == m - 2 : j == 0;
          s = starts ? lo : -1;
          d = ex2(g2 * float(kRev && starts ? e - a - (m - 1) * x.run : x.run));
        }
      }
      seg_of[tid] = s;
      decay[tid] = d;
    }
    __syncthreads();
    for (int32_t i0 = 0; i0 < n; i0 += kAhead) {
      f32x4 own[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int32_t i = i0 + u;
        if (i < n && seg_of[i] != -2) {
          const int64_t idx = kRev ? count - 1 - (base + i) : base + i;
          own[u] = *reinterpret_cast<const f32x4*>(R.saved + (idx * x.H + h) * size + elem);
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int32_t i = i0 + u;
        if (i >= n || seg_of[i] == -2) continue;
        if (seg_of[i] >= 0)
          X = R.init ? *reinterpret_cast<const f32x4*>(R.init + (int64_t(seg_of[i]) * x.H + h) * size + elem)
                     : f32x4{0.f, 0.f, 0.f, 0.f};
        const int64_t idx = kRev ? count - 1 - (base + i) : base + i;
#pragma unroll
        for (int e = 0; e < 4; ++e) X[e] = own[u][e] + decay[i] * X[e];
        *reinterpret_cast<f32x4*>(R.saved + (idx * x.H + h) * size + elem) = X;
      }
    }
  }
}

// Role 0 forward and, behind its work-groups, role 1 backward.
__global__ __launch_bounds__(kScan) void linear_scan_kernel(const WalkArgs x, int32_t size, int32_t count) {
  __shared__ int32_t seg_of[kScan];
  __shared__ float decay[kScan];
  const int32_t n = x.H * (size / (4 * kScan)), blk = blockIdx.x;
  if (blk < n)
    scan<false>(x, x.r[0], blk, size, count, seg_of, decay);
  else
    scan<true>(x, x.r[1], blk - n, size, count, seg_of, decay);
}

// Tokens of a run: the smallest power of two from sqrt(1.5 N H) on, in
// [256, 4096]. Shorter runs keep more work-groups busy but save, scan and read
// back more states (their number times their length is N H). Measured, us at
// runs of 512 / 1024 / 2048: N H = 2^21 (65536 tokens, 39 segments, 32 heads of
// 128): 883 / 742 / 680; 2^19 (one segment of 32768, 16 heads): 246 / 207 / 281;
// 2^17 (8192 tokens, forward and reverse): 265 / 353 / 641 (256: 277).
int32_t run_tokens(int64_t N, int32_t H) {
  int32_t r = 256;
  while (r < 4096 && int64_t(r) * r < N * H * 3 / 2) r *= 2;
  return r;
}

Role role(const void* a, const void* b, const void* c, void* out, const float* init, float* saved, float* fin,
          float in_scale, float out_scale, bool transposed) {
  return {static_cast<const bf16*>(a), static_cast<const bf16*>(b), static_cast<const bf16*>(c),
          static_cast<bf16*>(out), init, saved, fin, in_scale, out_scale, transposed};
}

// Own end states of the runs, then the states before them, of one or both roles.
template <int DA, int DB, bool kBoth>
void states(const WalkArgs& x, hipStream_t stream) {
  const int32_t count = int32_t(x.N / x.run), size = DA * DB;
  linear_state_kernel<DA, DB, kBoth><<<dim3(uint32_t(int64_t(count) * x.H * (kBoth ? 2 : 1))), dim3(2 * DB), 0,
                                               stream>>>(x);
  linear_scan_kernel<<<dim3(uint32_t(x.H * (size / (4 * kScan)) * (kBoth ? 2 : 1))), dim3(kScan), 0, stream>>>(x, size,
                                                                                                               count);
}

template <int DA, int DB, bool kRev, bool kPair>
void walk(const WalkArgs& x, hipStream_t stream) {
  const int64_t tail = x.N * x.H * DB * 2 + (x.r[0].fin ? int64_t(x.max_segs) * x.H * DA * DB * 4 : 0);
  linear_walk_kernel<DA, DB, kRev, kPair>
      <<<dim3(uint32_t(slot_blocks(x.grid, x.H) + tail_groups(tail))), dim3((kPair ? 4 : 2) * DB), 0, stream>>>(x);
}

WalkArgs common(const LinearArgs& y) {
  WalkArgs x{};
  x.g = y.g;
  x.cu = y.cu;
  x.max_segs = y.max_segs;
  x.N = y.N;
  x.H = y.H;
  x.run = run_tokens(y.N, y.H);
  x.grid = slot_grid(y.N, y.max_segs, x.run);
  x.flags = y.flags;
  return x;
}

template <int DK, int DV>
hipError_t fwd(const LinearArgs& y, hipStream_t s) {
  WalkArgs x = common(y);
  x.r[0] = role(y.q, y.k, y.v, y.o, y.initial_state, static_cast<float*>(y.workspace), y.final_state, 1.f, y.scale, false);
  if (y.N > x.run) states<DK, DV, false>(x, s);
  walk<DK, DV, false, false>(x, s);
  return hipGetLastError();
}

template <int DK, int DV>
hipError_t bwd(const LinearArgs& y, const LinearGradArgs& z, hipStream_t s) {
  WalkArgs x = common(y);
  float* saved = static_cast<float*>(y.workspace);
  float* adjoint = saved + y.N / x.run * y.H * DK * DV;
  if (y.N > x.run) {
    x.r[0] = role(nullptr, y.k, y.v, nullptr, y.initial_state, saved, nullptr, 1.f, 1.f, false);
    x.r[1] = role(nullptr, y.q, z.dout, nullptr, z.dfinal_state, adjoint, nullptr, y.scale, 1.f, false);
    states<DK, DV, true>(x, s);
  }
  const Role dq = role(z.dout, y.v, y.k, z.dq, y.initial_state, saved, nullptr, 1.f, y.scale, true);
  const Role dv = role(y.k, y.q, z.dout, z.dv, z.dfinal_state, adjoint, z.d_initial_state, y.scale, 1.f, false);
  const Role dk = role(y.v, z.dout, y.q, z.dk, z.dfinal_state, adjoint, nullptr, y.scale, 1.f, true);
  x.r[0] = dq;
  walk<DV, DK, false, false>(x, s);
  x.r[0] = dv;
  if constexpr (DK == DV) {
    x.r[1] = dk;
    walk<DK, DV, true, true>(x, s);
  } else {
    walk<DK, DV, true, false>(x, s);
    x.r[0] = dk;
    walk<DV, DK, true, false>(x, s);
  }
  return hipGetLastError();
}

}  // namespace

bool linear_chunk_supported(int32_t Dk, int32_t Dv, int32_t dtype) {
  return dtype == 0 && (Dk == 64 || Dk == 128) && (Dv == 64 || Dv == 128);
}

size_t linear_chunk_workspace_bytes(int64_t N, int32_t H, int32_t Dk, int32_t Dv, bool reverse) {
  const int32_t run = run_tokens(N, H);
  return N > run ? size_t(N / run) * H * Dk * Dv * 4 * (reverse ? 2 : 1) : 0;
}

int64_t linear_chunk_grid(int64_t N, int32_t max_segs, int32_t H) {
  return tile_slots(N, max_segs, run_tokens(N, H)) * H + 256;
}

hipError_t launch_linear_chunk(const LinearArgs& x, hipStream_t s) {
  if (x.Dk == 64) return x.Dv == 64 ? fwd<64, 64>(x, s) : fwd<64, 128>(x, s);
  return x.Dv == 64 ? fwd<128, 64>(x, s) : fwd<128, 128>(x, s);
}

hipError_t launch_linear_chunk_backward(const LinearArgs& x, const LinearGradArgs& y, hipStream_t s) {
  if (x.Dk == 64) return x.Dv == 64 ? bwd<64, 64>(x, y, s) : bwd<64, 128>(x, y, s);
  return x.Dv == 64 ? bwd<128, 64>(x, y, s) : bwd<128, 128>(x, y, s);
}

}  // namespace pkv
