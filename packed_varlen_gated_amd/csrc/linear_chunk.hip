// Packed linear attention with one decay per head in chunks of 64 tokens on the
// matrix cores (bf16, head dimensions 64 and 128).
//
//   S_t = lam S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t,  lam = e^{g_h}
//
// One walk serves the forward pass and the three gradients (roles (a, b, c) and
// directions as in linear_serial.hip). Over a chunk of n tokens, forward
// (backward: the two powers change places and the mask is s >= t):
//   out_t = sum_{s <= t} lam^(t - s) (a_t.b_s) c_s + lam^(t + 1) X^T a_t
//   X <- lam^n X + sum_s lam^(n - 1 - s) b_s c_s^T
// A work-group takes one run (up to `run` tokens of a segment) of one head; a
// wave owns 32 columns of X, in fp32 registers, and of the output. The in-chunk
// weights are formed by every wave: b rows from LDS against a in registers, and
// their result is, register for register, an operand of the product with c.
// X is rounded to bf16 once, as the operand of the readout; the update's decayed
// c is split into three bf16 parts (24 bits), so X itself sees no bf16 rounding:
// its products would cost less with one part, but final states are fp32 results.
//
// Rows and columns of X are dealt to the registers so that 8 consecutive ones
// are 8 consecutive registers of a lane (the transposing LDS reads take their
// 8-byte pieces in the order 0, 2, 1, 3): a is read in 16-byte pieces, outputs
// are stored in 16-byte pieces.
//
// Tiles go from memory into LDS without passing registers. b has two buffers; a
// and c have one each, since a is done with after the products that c is not yet
// needed for: the next a is loaded over a's second half of a chunk, c over the
// first. 73 KiB at 128 channels: two work-groups per compute unit.
//
// Segments longer than a run: a first launch walks every run but the segment's
// last (in the walk's direction) without outputs and saves its own end state, a
// second one turns these into the states before each run, and the walk starts
// from those. A run's length depends on the call's sizes only.

#include "mfma.h"
#include "segments.h"

namespace pkv {
namespace {

constexpr int kC = 64;      // tokens per chunk
constexpr int kTail = 256;  // work-groups for the rows no segment has and empty slots

template <int D>
struct Rows {  // an LDS tile of 64 rows of D channels
  static constexpr int CH = D / 8, ROW = D * 2, BYTES = kC * ROW;
  static __device__ __forceinline__ int swz(int row) {
    return D == 128 ? ((row & 3) << 2) | ((row >> 2) & 3) : ((row & 2) << 1) | ((row >> 2) & 3);
  }
};

template <int D, int NT>
__device__ __forceinline__ void issue_tile(__amdgpu_buffer_rsrc_t r, int32_t stride, char* dst, int wave) {
  constexpr int STEP = NT / Rows<D>::CH;
  const int row = fresh(threadIdx.x) / Rows<D>::CH, pos = threadIdx.x % Rows<D>::CH;
#pragma unroll
  for (int i = 0; i < kC / STEP; ++i) {
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

struct WalkArgs {
  const bf16 *a, *b, *c;
  const float* g;
  const int32_t* cu;
  int32_t max_segs;
  int64_t N;
  int32_t H, run;
  SlotGrid grid;
  float in_scale, out_scale;
  bool transposed;    // states are [DB][DA] in memory
  const float* init;  // [max_segs, H, ..] or null
  float* saved;       // [N / run, H, ..]: states between runs
  bf16* out;
  float* fin;  // [max_segs, H, ..] or null
  int32_t* flags;
};

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

template <int DA, int DB, bool kRev, bool kState>
__global__ __launch_bounds__(2 * DB, 2) void linear_walk_kernel(const WalkArgs x) {
  constexpr int NW = DB / 32, NT = 64 * NW, KA = DA / 16, TA = DA / 32;
  constexpr int SB = Rows<DA>::BYTES, SC = Rows<DB>::BYTES;
  // b of the even chunks, of the odd ones, then c and a (the state walk: c of the
  // even chunks, of the odd ones); the update's weights of each parity; the
  // in-chunk weights of the lane
  constexpr int kPieces = kC * Rows<DA>::CH / NT;  // loads of a b tile per lane
  __shared__ __attribute__((aligned(1024))) char lds[2 * SB + (kState ? 2 * SC : SC + SB)];
  __shared__ float upd[2][kC];
  __shared__ f32x4 rel[kState ? 1 : 2][kState ? 1 : 4][kState ? 1 : 64];

  const int64_t blk = blockIdx.x;
  if (!kState && blk >= slot_blocks(x.grid, x.H)) {
    const int tid = threadIdx.x;
    const int64_t j = blk - slot_blocks(x.grid, x.H);
    zero_tail(x.out, covered_tokens(x.cu, x.max_segs, x.N), x.N, int64_t(x.H) * DB * 2, j, kTail);
    if (j == 0) check_cu(x.cu, x.max_segs, x.N, x.flags);
    if (x.fin != nullptr && x.cu != nullptr) {
      // empty slots keep their initial state (or 0)
      const int64_t n = int64_t(x.H) * DA * DB / 4;
      for (int64_t s = j; s < x.max_segs; s += kTail) {
        if (x.cu[s] != x.cu[s + 1]) continue;
        f32x4* to = reinterpret_cast<f32x4*>(x.fin) + s * n;
        const f32x4* from = x.init ? reinterpret_cast<const f32x4*>(x.init) + s * n : nullptr;
        for (int64_t i = tid; i < n; i += NT) to[i] = from ? from[i] : f32x4{0.f, 0.f, 0.f, 0.f};
      }
    }
    return;
  }
  int32_t slot, h0, h1;
  SegTile t;
  if constexpr (kState) {
    // the run that ends in saved state blk / H
    h0 = int32_t(blk % x.H);
    h1 = h0 + 1;
    if (!find_saved<kRev>(x.cu, x.max_segs, x.N, x.run, int32_t(blk / x.H), t)) return;
  } else {
    slot_of(x.grid, blk, x.H, slot, h0, h1);
    if (!find_tile(x.cu, x.max_segs, x.N, x.run, slot, t)) return;
  }
  const int32_t end = t.e - t.start > x.run ? t.start + x.run : t.e;
  const bool first = kRev ? end == t.e : t.start == t.a;  // in the walk's direction
  const bool last = kRev ? t.start == t.a : end == t.e;
  // the saved state that this run starts from is at - 1 (backward: at), and the
  // one it ends in is at (backward: at - 1)
  const int64_t at = int64_t(t.a / x.run) + (t.start - t.a) / x.run;
  constexpr int64_t kState_ = int64_t(DA) * DB;

  for (int32_t h = h0; h < (kState ? h0 + 1 : h1); ++h) {
  // (nothing that goes by the lane is kept from one head to the next)
  const int tid = fresh(threadIdx.x), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  if (!kState && h != h0) __syncthreads();  // the last head is done with LDS
  const float g2 = x.g[h] * kLog2e;
  const int half = lane >> 5, col = lane & 31;
  const int32_t as = x.H * DA * 2, cs = x.H * DB * 2;
  const int n_chunks = (end - t.start + kC - 1) / kC;
  auto chunk_start = [&](int i) { return t.start + (kRev ? n_chunks - 1 - i : i) * kC; };
  auto chunk_len = [&](int32_t s0) { return end - s0 < kC ? end - s0 : kC; };
  auto issue_b = [&](int i) {
    const int32_t s0 = chunk_start(i), n = chunk_len(s0);
    issue_tile<DA, NT>(buffer(x.b + (int64_t(s0) * x.H + h) * DA, int64_t(n - 1) * as + DA * 2), as,
                       lds + (i & 1) * SB, wave);
    if (tid < kC) upd[i & 1][tid] = tid < n ? x.in_scale * ex2(g2 * (kRev ? tid + 1 : n - 1 - tid)) : 0.f;
  };
  auto issue_c = [&](int i) {
    const int32_t s0 = chunk_start(i), n = chunk_len(s0);
    issue_tile<DB, NT>(buffer(x.c + (int64_t(s0) * x.H + h) * DB, int64_t(n - 1) * cs + DB * 2), cs,
                       lds + 2 * SB + (kState ? (i & 1) * SC : 0), wave);
  };
  auto issue_a = [&](int i) {
    const int32_t s0 = chunk_start(i), n = chunk_len(s0);
    issue_tile<DA, NT>(buffer(x.a + (int64_t(s0) * x.H + h) * DA, int64_t(n - 1) * as + DA * 2), as,
                       lds + 2 * SB + SC, wave);
  };
  // The state walk leaves out the chunks whose tokens decay to a weight that
  // fp32 has only 0 for (2^-150) by the run's end.
  int it0 = 0;
  if constexpr (kState) {
    const float far = g2 < 0.f ? fminf(150.f / (-kC * g2), 1e6f) : 1e6f;
    it0 = n_chunks - 1 - int(far);
    it0 = it0 < 0 ? 0 : it0;
  }
  issue_b(it0);
  if constexpr (kState) issue_c(it0);
  else issue_a(0);

  f32x16 X[TA];
  const float* from = kState ? nullptr
                             : first ? (x.init ? x.init + (int64_t(t.seg) * x.H + h) * kState_ : nullptr)
                                     : x.saved + ((kRev ? at : at - 1) * x.H + h) * kState_;
  if (from != nullptr) {
    StateAddr<DA, DB>(from, x.transposed, tid).load(X);
  } else {
#pragma unroll
    for (int i = 0; i < TA; ++i) X[i] = f32x16{};
  }

  if constexpr (!kState) {
    // rel[0]: weights inside a 32 x 32 block on the diagonal, rel[1]: of the
    // block below it (s 32 .. 1 tokens further from t)
    if (wave == 0) {
      const float f = x.in_scale * x.out_scale;
#pragma unroll
      for (int i4 = 0; i4 < 4; ++i4) {
        f32x4 w0, w1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int s = 8 * i4 + 4 * half + e, d = kRev ? s - col : col - s;
          w0[e] = d >= 0 ? f * ex2(g2 * d) : 0.f;
          w1[e] = f * ex2(g2 * (d + 32));
        }
        rel[0][i4][lane] = w0;
        rel[1][i4][lane] = w1;
      }
    }
  }
  const Transposed<DA> tb(lane);
  const Transposed<DB> tc(lane);
  const int fx = Rows<DA>::swz(col);

  for (int it = it0; it < n_chunks; ++it) {
    __builtin_amdgcn_s_waitcnt(0x0070);  // loads into LDS and LDS stores done
    bar();
    if constexpr (!kState) {
      issue_c(it);
      // c's loads stay before the next b's: the wait for c below counts those
      asm volatile("" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    }
    if (it + 1 < n_chunks) {
      issue_b(it + 1);
      if constexpr (kState) issue_c(it + 1);
    }
    __builtin_amdgcn_sched_barrier(0);
    const char* bt = lds + (it & 1) * SB;
    const char* ct = lds + 2 * SB + (kState ? (it & 1) * SC : 0);
    const char* at_ = lds + 2 * SB + SC;
    const int32_t s0 = chunk_start(it), n = chunk_len(s0);

    bf16x8 cf[4];
    if constexpr (!kState) {
      // In-chunk weights of a 32 x 32 block (rows s of block sb, columns t of
      // block u) as operands; three of the four blocks have any.
      bf16x8 wf[2][4];
      auto weigh = [&](const f32x16& w, int u, int sb) {
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) {
          const f32x4 f = rel[sb == u ? 0 : 1][i4][lane];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            wf[u][2 * sb + i4 / 2][4 * (i4 % 2) + e] = static_cast<bf16>(w[4 * i4 + e] * f[e]);
        }
      };
      auto row = [&](const char* t, int sb, int i) {
        return *reinterpret_cast<const bf16x8*>(t + (32 * sb + col) * Rows<DA>::ROW + (((2 * i + half) ^ fx) * 16));
      };
      // Five independent products take turns: the three blocks and the readout
      // of X for both column blocks.
      constexpr int sFar = kRev ? 1 : 0, sOne = kRev ? 0 : 1;  // row blocks of both, of one
      f32x16 o[2] = {};
      {
        f32x16 w0 = {}, w1 = {}, w2 = {};
#pragma unroll
        for (int i = 0; i < KA; ++i) {
          const bf16x8 br = row(bt, sFar, i), a0 = row(at_, 0, i), a1 = row(at_, 1, i);
          bf16x8 xs;
#pragma unroll
          for (int j = 0; j < 8; ++j) xs[j] = static_cast<bf16>(X[i / 2][8 * (i % 2) + j]);
          w0 = mfma32(br, a0, w0);
          w1 = mfma32(br, a1, w1);
          w2 = mfma32(row(bt, sOne, i), kRev ? a0 : a1, w2);
          o[0] = mfma32(xs, a0, o[0]);
          o[1] = mfma32(xs, a1, o[1]);
        }
        __builtin_amdgcn_sched_barrier(0);
        weigh(w0, 0, sFar);
        weigh(w1, 1, sFar);
        weigh(w2, sOne, sOne);
      }
      // c has come (the next b may still be on its way), a is free
      if (it + 1 < n_chunks)
        __builtin_amdgcn_s_waitcnt(0x0070 | kPieces);
      else
        __builtin_amdgcn_s_waitcnt(0x0070);
      bar();
      if (it + 1 < n_chunks) issue_a(it + 1);
#pragma unroll
      for (int j = 0; j < 4; ++j) cf[j] = tc.read(ct, wave, j);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int d = kRev ? n - 1 - 32 * u - col : 32 * u + col + 1;
        const float ow = x.out_scale * ex2(g2 * (d < 0 ? 0 : d));
#pragma unroll
        for (int i = 0; i < 16; ++i) o[u][i] *= ow;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (kRev ? j / 2 < u : j / 2 > u) continue;
          o[u] = mfma32(cf[j], wf[u][j], o[u]);
        }
      // (rows past the chunk's end are out of the buffer's range)
      const auto ro = buffer(x.out + (int64_t(s0) * x.H + h) * DB, int64_t(n - 1) * cs + DB * 2);
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          bf16x8 y;
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = static_cast<bf16>(o[u][8 * v + j]);
          store16(ro, uint32_t(32 * u + col) * cs + 64 * wave + 16 * half + 32 * v, __builtin_bit_cast(i32x4, y));
        }
      __builtin_amdgcn_sched_barrier(0);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) cf[j] = tc.read(ct, wave, j);
    }

    const float carry = ex2(g2 * n);
#pragma unroll
    for (int i = 0; i < TA; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) X[i][j] *= carry;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bf16x8 part[3];  // exact to 24 bits
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const f32x4 w = *reinterpret_cast<const f32x4*>(&upd[it & 1][16 * j + 8 * u + 4 * half]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float y = to_f32(cf[j][4 * u + e]) * w[e];
#pragma unroll
          for (int s = 0; s < 3; ++s) {
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
      for (int s = 0; s < 3; ++s)
#pragma unroll
        for (int i = 0; i < TA; ++i) X[i] = mfma32(bT[i], part[s], X[i]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  float* to = kState ? x.saved + ((kRev ? at - 1 : at) * x.H + h) * kState_
                     : (last && x.fin ? x.fin + (int64_t(t.seg) * x.H + h) * kState_ : nullptr);
  if (to != nullptr) StateAddr<DA, DB>(to, x.transposed, tid).store(X);
  }
}

// The saved states, each its run's own end state, become the states that the
// walk has there: X <- own + lam^(run's tokens) X, X = init before a segment's
// first run. A work-group takes 256 x 4 elements of one head through all indices
// in order.
constexpr int kScan = 256;
constexpr int kAhead = 8;  // states whose loads are in flight at once

template <bool kRev>
__global__ __launch_bounds__(kScan) void linear_scan_kernel(const WalkArgs x, int32_t size, int32_t count) {
  __shared__ int32_t seg_of[kScan];  // segment of the index if it starts the walk there, -1 if it goes on, -2 if unused
  __shared__ float decay[kScan];
  const int tid = threadIdx.x;
  const int32_t parts = size / (4 * kScan), h = blockIdx.x / parts;
  const int64_t elem = (int64_t(blockIdx.x % parts) * kScan + tid) * 4;
  const float g2 = x.g[h] * kLog2e;
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
          own[u] = *reinterpret_cast<const f32x4*>(x.saved + (idx * x.H + h) * size + elem);
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int32_t i = i0 + u;
        if (i >= n || seg_of[i] == -2) continue;
        if (seg_of[i] >= 0)
          X = x.init ? *reinterpret_cast<const f32x4*>(x.init + (int64_t(seg_of[i]) * x.H + h) * size + elem)
                     : f32x4{0.f, 0.f, 0.f, 0.f};
        const int64_t idx = kRev ? count - 1 - (base + i) : base + i;
#pragma unroll
        for (int e = 0; e < 4; ++e) X[e] = own[u][e] + decay[i] * X[e];
        *reinterpret_cast<f32x4*>(x.saved + (idx * x.H + h) * size + elem) = X;
      }
    }
  }
}

// Tokens of a run: the smallest power of two from sqrt(1.5 N H) on, in
// [256, 4096]. Shorter runs keep more work-groups busy but save, scan and read
// back more states (their number times their length is N H). Measured, us at
// runs of 512 / 1024 / 2048 / 4096: N H = 2^21 (65536 tokens, 39 segments, 32
// heads of 128): 900 / 755 / 704 / 825; 2^19 (one segment of 32768, 16 heads):
// 249 / 213 / 253 / 448; 2^17 (8192 tokens, forward and reverse): 282 / 398 /
// 694 / 843 (256: 325).
int32_t run_tokens(int64_t N, int32_t H) {
  int32_t r = 256;
  while (r < 4096 && int64_t(r) * r < N * H * 3 / 2) r *= 2;
  return r;
}

template <int DA, int DB, bool kRev, bool kState>
void walk(WalkArgs x, const void* a, const void* b, const void* c, bool transposed, float in_scale, float out_scale,
          const float* init, void* out, float* fin, hipStream_t stream) {
  x.a = static_cast<const bf16*>(a);
  x.b = static_cast<const bf16*>(b);
  x.c = static_cast<const bf16*>(c);
  x.transposed = transposed;
  x.in_scale = in_scale;
  x.out_scale = out_scale;
  x.init = init;
  x.out = static_cast<bf16*>(out);
  x.fin = fin;
  const int64_t grid = kState ? x.N / x.run * x.H : slot_blocks(x.grid, x.H) + kTail;
  linear_walk_kernel<DA, DB, kRev, kState><<<dim3(uint32_t(grid)), dim3(2 * DB), 0, stream>>>(x);
}

template <bool kRev>
void scan(WalkArgs x, int32_t size, const float* init, hipStream_t stream) {
  x.init = init;
  linear_scan_kernel<kRev><<<dim3(uint32_t(x.H * (size / (4 * kScan)))), dim3(kScan), 0, stream>>>(
      x, size, int32_t(x.N / x.run));
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
  x.saved = static_cast<float*>(y.workspace);
  x.flags = y.flags;
  return x;
}

template <int DK, int DV>
hipError_t fwd(const LinearArgs& y, hipStream_t s) {
  const WalkArgs x = common(y);
  if (y.N > x.run) {
    walk<DK, DV, false, true>(x, nullptr, y.k, y.v, false, 1.f, 1.f, nullptr, nullptr, nullptr, s);
    scan<false>(x, DK * DV, y.initial_state, s);
  }
  walk<DK, DV, false, false>(x, y.q, y.k, y.v, false, 1.f, y.scale, y.initial_state, y.o, y.final_state, s);
  return hipGetLastError();
}

template <int DK, int DV>
hipError_t bwd(const LinearArgs& y, const LinearGradArgs& z, hipStream_t s) {
  const WalkArgs x = common(y);
  if (y.N > x.run) {
    walk<DK, DV, false, true>(x, nullptr, y.k, y.v, false, 1.f, 1.f, nullptr, nullptr, nullptr, s);
    scan<false>(x, DK * DV, y.initial_state, s);
  }
  walk<DV, DK, false, false>(x, z.dout, y.v, y.k, true, 1.f, y.scale, y.initial_state, z.dq, nullptr, s);
  if (y.N > x.run) {
    walk<DK, DV, true, true>(x, nullptr, y.q, z.dout, false, y.scale, 1.f, nullptr, nullptr, nullptr, s);
    scan<true>(x, DK * DV, z.dfinal_state, s);
  }
  walk<DV, DK, true, false>(x, y.v, z.dout, y.q, true, y.scale, 1.f, z.dfinal_state, z.dk, nullptr, s);
  walk<DK, DV, true, false>(x, y.k, y.q, z.dout, false, y.scale, 1.f, z.dfinal_state, z.dv, z.d_initial_state, s);
  return hipGetLastError();
}

}  // namespace

bool linear_chunk_supported(int32_t Dk, int32_t Dv, int32_t dtype) {
  return dtype == 0 && (Dk == 64 || Dk == 128) && (Dv == 64 || Dv == 128);
}

size_t linear_chunk_workspace_bytes(int64_t N, int32_t H, int32_t Dk, int32_t Dv) {
  const int32_t run = run_tokens(N, H);
  return N > run ? size_t(N / run) * H * Dk * Dv * 4 : 0;
}

int64_t linear_chunk_grid(int64_t N, int32_t max_segs, int32_t H) {
  return tile_slots(N, max_segs, run_tokens(N, H)) * H + kTail;
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
