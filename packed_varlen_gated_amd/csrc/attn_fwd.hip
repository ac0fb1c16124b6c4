// Packed causal softmax attention with grouped heads on the matrix cores (bf16,
// D in {64, 128}).
//
//   o_t = sum_{s <= t, same segment} softmax_s(scale q_t.k_s) v_s
//   lse_t = ln sum_s exp(scale q_t.k_s)
//
// A work-group of 4 waves takes 128 queries of one head (a tile aligned to its
// segment's start, segments.h) and walks the keys in tiles of 64; a wave holds
// 32 queries. Per tile, with the running maximum m and sum l of a row (base 2):
//   S^T = K Q^T, P = 2^(c S - m), l += sum P, O^T += V^T P^T    (c = scale log2 e)
// S^T has a query per lane, so the softmax needs one exchange between the
// lanes l and l + 32, and P^T in the registers of S^T is the B operand of the
// second product as it stands: its contraction slots are the keys
// {4 g .. 4 g + 3, 8 + 4 g .. 8 + 4 g + 3} of a 16-key step (g = lane / 32), and
// V^T is read through transposing LDS reads in that order.
//
// O and l are rescaled only when a row's maximum grew by more than 2^8 since
// the last rescaling: weights are then at most 2^8 instead of 1, which neither
// their bf16 rounding (relative) nor the fp32 sums see, and most tiles skip 2 D
// multiplications per query.
//
// K and V tiles go from memory into LDS without passing registers, the next
// tile while this one is used; two buffers, one barrier per tile. 16-byte chunk
// c of row r is kept at chunk c ^ f(r) (the loads' source addresses are
// permuted), so both the row-wise reads of K and the transposing reads of V
// touch every bank once.
//
// A weight of 0 times a value that is not finite is NaN, so a later token's
// value could reach an earlier one through a tile on the diagonal. When an
// output is not finite the work-group walks the keys once more with such
// values as 0, and adds to each row the infinity or NaN of its own past (the
// weight of a finite score is above 0): with every value finite nothing is spent
// but the check.
//
// Bound by the matrix and the vector units' turns: 46 % of the cycles have a
// matrix instruction, the softmax's vector work takes about as many, and two
// work-groups per compute unit (the sums and Q take 192 registers at D 128) do not
// hide all of one under the other. 65536 tokens in documents of up to 8192, H 32,
// Hkv 8, D 128: 2.06-2.16 ms, 888-932 TFLOP/s of causal products (a large matrix
// product reaches 1220 here, 1.57 ms); 77 tokens, H 16: 8.5-9.0 us. A raised wave
// priority around the products made the first 2.31 ms.
//
// Through a window (kWin) a tile's walk is that of WindowWalk (segments.h): the tiles that
// hold the segment's first `sinks` keys, then those from the first query's window on.
// 65536 tokens in documents of up to 8192, H 32, Hkv 8, D 128, window 1024, 4 sinks:
// 1.03 ms, 783 TFLOP/s of visible products (0.66 ms at the rate of a large product); a
// wave walks 1184 keys for the 1028 that a row sees, so its rate is the causal kernel's.
// The loads' waits are written here, not the compiler's (1.13 ms). Leaving out the hidden
// 32 keys of a tile's half: 1.13 ms, for registers that no longer fit. 8192 tokens, H 16,
// Hkv 4, D 128, window 512: 57 us; 16384, H 16, D 64, window 256, 4 sinks: 56 us.

#include "mfma.h"
#include "segments.h"

#include <float.h>

namespace pkv {
namespace {

constexpr int kThreads = 256;
// kS waves share 32 queries, each with 64 keys of a tile, their sums joined at the
// end: kS = 1, a work-group has 128 queries; kS = 2, 64 and tiles of 128 keys.
template <int kS>
struct Shape {
  static constexpr int BM = 128 / kS, BN = 64 * kS;  // queries of a work-group, keys of a tile
};
constexpr float kGrow = 8.f;      // log2 of what a row's maximum may grow by before O is rescaled

template <int D, int kBN>
struct Tile {
  static constexpr int CH = D / 8;          // 16-byte chunks per row
  static constexpr int BYTES = kBN * D * 2;
  // chunk swizzles: rows read by the 16 lanes of a pass (K), or the four rows
  // of 64 bytes that a transposing read of 32 lanes takes (V), on distinct banks
  static __device__ __forceinline__ int k_swz(int row) { return D == 128 ? row & 15 : (row >> 1) & 7; }
  static __device__ __forceinline__ int v_swz(int row) { return D == 128 ? (row & 3) << 2 : (row & 2) << 1; }
};

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= FLT_MAX; }

template <int D, int kS, bool kWin>
__global__ __launch_bounds__(kThreads, D == 64 && kS == 1 ? 3 : 2) void attn_fwd_kernel(
    const bf16* __restrict__ q, const bf16* __restrict__ k, const bf16* __restrict__ v,
    const int32_t* __restrict__ cu, int32_t max_segs, int64_t N, int32_t H, int32_t Hkv, float scale,
    bf16* __restrict__ o, float* __restrict__ lse, int32_t* __restrict__ flags, SlotGrid grid, int32_t window,
    int32_t sinks) {
  static_assert(!kWin || kS == 1, "windowed walks are short");
  constexpr int kBM = Shape<kS>::BM, kBN = Shape<kS>::BN;
  using TileD = Tile<D, kBN>;
  constexpr int CH = TileD::CH, KS = D / 16, DT = D / 32, LD = kBN * CH / kThreads;
  constexpr int TB = TileD::BYTES;
  __shared__ __attribute__((aligned(1024))) char lds[4 * TB];  // K, V of the even tiles, K, V of the odd ones
  static_assert(4 * TB >= kBM * D * 2, "the outputs are staged in the tiles' buffers");

  const int64_t b = blockIdx.x;
  const int64_t blocks = slot_blocks(grid, H);
  if (b >= blocks) {
    const int64_t j = b - blocks, groups = gridDim.x - blocks, c = covered_tokens(cu, max_segs, N);
    zero_tail(o, c, N, int64_t(H) * D * 2, j, groups);
    if (lse != nullptr)
      for (int64_t i = j * kThreads + threadIdx.x; i < (N - c) * H; i += groups * kThreads)
        lse[(i / (N - c)) * N + c + i % (N - c)] = -INFINITY;
    if (j == 0) check_cu(cu, max_segs, N, flags);
    return;
  }
  int32_t slot, h0, h1;
  slot_of(grid, b, H, slot, h0, h1);
  SegTile t;
  // late tiles have the most keys: they start first
  if (slot < grid.near) slot = grid.near - 1 - slot;
  if (!find_tile(cu, max_segs, N, kBM, slot, t)) return;

  for (int32_t hi = h0; hi < h1; ++hi) {
    // Consecutive work-groups run on different XCDs: the query heads of one kv
    // head are Hkv apart, so with Hkv a multiple of 8 they share an L2.
    const int32_t hk = hi % Hkv, h = hk * (H / Hkv) + hi / Hkv;
    // (nothing that goes by the lane is kept from one head to the next)
    const int tid = fresh(threadIdx.x), lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int half = lane >> 5, col = lane & 31;
    const int32_t kstride = Hkv * D * 2, qstride = H * D * 2;
    const int part = wave % kS;                    // of the keys
    const int32_t q0 = t.start + wave / kS * 32;  // the wave's first query
    const int32_t rows = t.e - q0;           // its real queries (may be <= 0 or > 32)
    const int32_t qend = t.start + kBM < t.e ? t.start + kBM : t.e;
    const WindowWalk ww(kWin ? window : 0x7fffffff, kWin ? sinks : 0, kBN, t.start, t.a);
    const int n_tiles = kWin ? ww.count((qend - t.a + kBN - 1) / kBN) : (qend - t.a + kBN - 1) / kBN;
    auto tile_start = [&](int it) { return t.a + (kWin ? ww.tile(it) : it) * kBN; };

    // the lane's first chunk of a tile; the others are whole multiples of 16 rows
    // further (the swizzles' period)
    constexpr int STEP = kThreads / CH;
    static_assert(STEP % 16 == 0, "the swizzles repeat");
    const int lrow = tid / CH, lpos = tid % CH;
    const uint32_t koff = uint32_t(lrow) * kstride + (lpos ^ TileD::k_swz(lrow)) * 16;
    const uint32_t voff = uint32_t(lrow) * kstride + (lpos ^ TileD::v_swz(lrow)) * 16;
    auto issue = [&](int it) {
      const int32_t s0 = tile_start(it);
      const int32_t have = t.e - s0 < kBN ? t.e - s0 : kBN;
      const int64_t at = (int64_t(s0) * Hkv + hk) * D, bytes = int64_t(have - 1) * kstride + D * 2;
      const uint32_t ko = fresh(koff), vo = fresh(voff);
      if constexpr (kWin) {
        const u32x4 rk = descriptor(k + at, bytes), rv = descriptor(v + at, bytes);
        const uint32_t dst = lds_addr(lds) + (it & 1) * 2 * TB + wave * 1024;
        uint32_t off[LD];
#pragma unroll
        for (int i = 0; i < LD; ++i) off[i] = ko + i * STEP * kstride;
        load_lds16_async<LD, kThreads * 16>(rk, off, dst);
#pragma unroll
        for (int i = 0; i < LD; ++i) off[i] = vo + i * STEP * kstride;
        load_lds16_async<LD, kThreads * 16>(rv, off, dst + TB);
        return;
      }
      const auto rk = buffer(k + at, bytes), rv = buffer(v + at, bytes);
      char* dst = lds + (it & 1) * 2 * TB + wave * 1024;
#pragma unroll
      for (int i = 0; i < LD; ++i) load_lds16(rk, ko + i * STEP * kstride, dst + i * kThreads * 16);
#pragma unroll
      for (int i = 0; i < LD; ++i) load_lds16(rv, vo + i * STEP * kstride, dst + TB + i * kThreads * 16);
    };

    // c > 0: a negative scale flips the queries' signs, a scale of 0 clears them
    // (a masked score is -inf, which a factor of 0 would turn into NaN)
    const float c = scale == 0.f ? 1.f : fabsf(scale) * kLog2e;
    bf16x8 qf[KS];
    {
      const int32_t have = rows < 0 ? 0 : (rows > 32 ? 32 : rows);
      const auto r = buffer(q + (int64_t(rows > 0 ? q0 : t.start) * H + h) * D,
                            have > 0 ? int64_t(have - 1) * qstride + D * 2 : 0);
      const uint32_t flip = scale < 0.f ? 0x80008000u : 0u, keep = scale == 0.f ? 0u : ~0u;
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        i32x4 x = __builtin_bit_cast(i32x4, load8(r, uint32_t(col) * qstride + (2 * i + half) * 16));
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = int((uint32_t(x[j]) ^ flip) & keep);
        qf[i] = __builtin_bit_cast(bf16x8, x);
      }
    }

    f32x16 acc[DT];
    float m = -FLT_MAX, l = 0.f;
#pragma unroll
    for (int i = 0; i < DT; ++i) acc[i] = f32x16{};

    // LDS addresses of this lane's operand chunks
    const int krow = col, kx = TileD::k_swz(col);
    const int vr = 4 * half + ((lane & 15) >> 2);              // key of the transposing read (mod 8)
    const int vc = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);  // its chunk in a 32-channel group
    const int vb = (lane & 1) * 8;                             // its half of the chunk
    const int vx = TileD::v_swz(vr);                         // (the swizzle has period 4)

    auto walk = [&](bool clean) {
      issue(0);
      for (int it = 0; it < n_tiles; ++it) {
        wait_vm();
        bar();
        if (it + 1 < n_tiles) issue(it + 1);
        char* kt = lds + (it & 1) * 2 * TB;
        char* vt = kt + TB;
        if (clean) {
          // values that are not finite become 0
          for (int i = tid; i < TB / 4; i += kThreads) {
            uint32_t x = reinterpret_cast<uint32_t*>(vt)[i];
            if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
            if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
            reinterpret_cast<uint32_t*>(vt)[i] = x;
          }
          __syncthreads();
        }
        const int32_t s0 = tile_start(it) + part * 64;  // the wave's first key
        if (rows <= 0 || s0 > q0 + 31) continue;
        if (kWin && s0 + 63 <= q0 - window && s0 >= t.a + sinks) continue;
        kt += part * (64 * D * 2);
        vt += part * (64 * D * 2);

        f32x16 s[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          s[j] = f32x16{};
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            const char* at = kt + (32 * j + krow) * (D * 2) + (((2 * i + half) ^ kx) * 16);
            const bf16x8 a = *reinterpret_cast<const bf16x8*>(at);
            s[j] = mfma32(a, qf[i], s[j]);
          }
        }
        if (s0 + 63 > q0) {
          const int32_t last = q0 + col - s0;  // the lane's query attends to keys 0 .. last of the tile
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              s[j][i] = 32 * j + 8 * (i / 4) + 4 * half + i % 4 <= last ? s[j][i] : -INFINITY;
        }
        if (kWin && s0 <= q0 + 31 - window) {
          // keys 0 .. old of the tile are behind the window, the first ones may be sinks
          const int32_t old = q0 + col - window - s0 - 4 * half, sink = t.a + sinks - s0 - 4 * half;
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int32_t key = 32 * j + 8 * (i / 4) + i % 4;
              s[j][i] = key > old || key < sink ? s[j][i] : -INFINITY;
            }
        }
        float mx = s[0][0];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[j][i]);
        mx = fmaxf(mx, other_half(mx)) * c;
        const bool grew = mx > m + kGrow;
        if (__builtin_amdgcn_ballot_w64(grew) != 0) {
          // (a row that did not grow keeps its bits, whatever the wave's other rows hold)
          const float f = grew ? ex2(m - mx) : 1.f;
          m = grew ? mx : m;
          l *= f;
#pragma unroll
          for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[i][j] *= f;
        }
        bf16x8 p[4];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float x = ex2(fmaf(s[j][i], c, -m));
            l += x;
            p[2 * j + i / 8][i % 8] = static_cast<bf16>(x);
          }
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const char* a = vt + (16 * j + vr) * (D * 2) + (((4 * i + vc) ^ vx) * 16) + vb;
            acc[i] = mfma32(join(read_tr(a), read_tr(a + 8 * (D * 2))), p[j], acc[i]);
          }
      }
    };
    // the shares' sums, by their maxima
    auto join_parts = [&] {
      if constexpr (kS > 1) {
        __syncthreads();  // every wave is done with the tiles
        f32x4* at = reinterpret_cast<f32x4*>(lds) + wave / kS * (DT * 4 * 64 + 64) + lane;
        if (part == 1) {
#pragma unroll
          for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              at[(4 * i + j) * 64] = f32x4{acc[i][4 * j], acc[i][4 * j + 1], acc[i][4 * j + 2], acc[i][4 * j + 3]};
          at[DT * 4 * 64] = f32x4{m, l, 0.f, 0.f};
        }
        __syncthreads();
        if (part == 0) {
          const f32x4 y = at[DT * 4 * 64];
          const float mn = fmaxf(m, y[0]), f0 = ex2(m - mn), f1 = ex2(y[0] - mn);
          m = mn;
          l = l * f0 + y[1] * f1;
#pragma unroll
          for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const f32x4 x = at[(4 * i + j) * 64];
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[i][4 * j + e] = acc[i][4 * j + e] * f0 + x[e] * f1;
            }
        }
      }
    };
    walk(false);

    join_parts();
    l += other_half(l);
    const float inv = 1.f / l;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        acc[i][j] *= inv;
        bad |= !finite(acc[i][j]);
      }
    bad = bad && col < rows && part == 0;
    if (lse != nullptr && half == 0 && col < rows && part == 0) lse[int64_t(h) * N + q0 + col] = m * kLn2 + logf(l);

    // outputs: rows of the wave through LDS, 16-byte stores
    const int have = part != 0 ? 0 : rows > 32 ? 32 : rows;
    auto put = [&](const int32_t* first) {
      char* st = lds + wave * (32 * D * 2);
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          bf16x4 x;
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = static_cast<bf16>(acc[i][4 * j + e]);
          const int ch = 4 * i + j;  // channels 32 i + 8 j + 4 half ..
          *reinterpret_cast<bf16x4*>(st + col * (D * 2) + ((ch ^ (col & (CH - 1))) * 16) + half * 8) = x;
        }
      // the wave's own rows: its LDS accesses are in order
      asm volatile("" ::: "memory");
      for (int i = lane; i < 32 * CH; i += 64) {
        const int r = i / CH, ch = i % CH;
        if (r >= have) continue;
        i32x4 x = *reinterpret_cast<const i32x4*>(st + r * (D * 2) + ((ch ^ (r & (CH - 1))) * 16));
        if (first != nullptr) {
          // the infinities and NaN of the row's own past
          bf16x8 y = __builtin_bit_cast(bf16x8, x);
          for (int e = 0; e < 8; ++e) {
            const int32_t* at = first + ch * 8 + e;
            float z = to_f32(y[e]);
            if (at[0] <= q0 + r) z += INFINITY;
            if (at[D] <= q0 + r) z -= INFINITY;
            if (at[2 * D] <= q0 + r) z = NAN;
            y[e] = static_cast<bf16>(z);
          }
          x = __builtin_bit_cast(i32x4, y);
        }
        *reinterpret_cast<i32x4*>(o + (int64_t(q0 + r) * H + h) * D + ch * 8) = x;
      }
    };
    const bool again = __syncthreads_or(bad);  // (also: every wave is done with the tiles)
    put(nullptr);
    if (!again) {
      if (hi + 1 < h1) __syncthreads();  // the outputs have left LDS
      continue;
    }

    if constexpr (kWin) {
      // Some output is not finite. What a row sees is no longer a prefix: after a walk
      // with such values as 0, another one adds them to the rows that see them.
      m = -FLT_MAX;
      l = 0.f;
#pragma unroll
      for (int i = 0; i < DT; ++i) acc[i] = f32x16{};
      __syncthreads();  // the outputs have left LDS
      walk(true);
      l += other_half(l);
      const float inv2 = 1.f / l;
#pragma unroll
      for (int i = 0; i < DT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[i][j] *= inv2;
      __shared__ uint32_t odd[kBN / 32];  // keys of the tile with such a value
      for (int it = 0; it < n_tiles; ++it) {
        __syncthreads();
        if (tid < kBN / 32) odd[tid] = 0;
        issue(it);
        wait_vm();
        __syncthreads();
        const char* vt = lds + (it & 1) * 2 * TB + TB;
        for (int i = tid; i < TB / 4; i += kThreads) {
          const uint32_t x = reinterpret_cast<const uint32_t*>(vt)[i];
          const int row = i / (D / 2);
          if ((x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u) atomicOr(&odd[row / 32], 1u << (row % 32));
        }
        __syncthreads();
        const int32_t s0 = tile_start(it);
        for (int s = 0; s < kBN; ++s) {
          if ((odd[s / 32] >> (s % 32) & 1) == 0) continue;
          const int32_t at = s0 + s, t_ = q0 + col;
          const bool sees = at <= t_ && (t_ - at < window || at - t.a < sinks);
          // (a fixed register per value: acc is indexed by constants alone)
#pragma unroll
          for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int ch = 32 * i + 8 * (j / 4) + 4 * half + j % 4;
              const float y = to_f32(*reinterpret_cast<const bf16*>(
                  vt + s * (D * 2) + (((ch / 8) ^ TileD::v_swz(s)) * 16) + ch % 8 * 2));
              if (sees && !finite(y)) acc[i][j] += y;
            }
        }
      }
      __syncthreads();
      put(nullptr);
      __syncthreads();
      continue;
    }

    // Some output is not finite. first[D x + d]: the first token of the segment
    // whose value d is inf (x = 0), -inf (1), NaN (2).
    __shared__ int32_t first[3 * D];
    for (int i = tid; i < 3 * D; i += kThreads) first[i] = 0x7fffffff;
    __syncthreads();
    const int c8 = tid % CH * 8;
    uint32_t seen = 0;  // by this thread: value e, kind x at bit 8 x + e
    for (int32_t s = t.a + tid / CH; s < qend && seen >> 16 != 0xff; s += 4 * STEP) {
      i32x4 y[4];  // (asked for together; a row past the end is the last one again)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int32_t su = s + u * STEP < qend ? s + u * STEP : qend - 1;
        y[u] = *reinterpret_cast<const i32x4*>(v + (int64_t(su) * Hkv + hk) * D + c8);
      }
      // (loops as they are: unrolled, they changed the order of the first walk's LDS
      // reads, which at D 128 then took 2.20 ms for 2.13 on attn_flat_microbatch)
#pragma unroll 1
      for (int u = 0; u < 4; ++u) {
#pragma unroll 1
        for (int e = 0; e < 8; ++e) {
          const uint32_t x = uint32_t(y[u][e / 2]) >> (e % 2 * 16) & 0xffff;
          if ((x & 0x7f80) != 0x7f80) continue;
          const int kind = (x & 0x7f) != 0 ? 2 : int(x >> 15), bit = 8 * kind + e;
          if (seen >> bit & 1) continue;
          seen |= 1u << bit;
          atomicMin(&first[kind * D + c8 + e], s + u * STEP < qend ? s + u * STEP : qend - 1);
        }
      }
    }
    m = -FLT_MAX;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < DT; ++i) acc[i] = f32x16{};
    __syncthreads();
    walk(true);
    join_parts();
    l += other_half(l);
    const float inv2 = 1.f / l;
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[i][j] *= inv2;
    __syncthreads();
    put(first);
    __syncthreads();
  }
}

}  // namespace

bool attn_mfma_supported(int32_t D, int32_t dtype) { return dtype == 0 && (D == 64 || D == 128); }

template <int D, int kS, bool kWin = false>
void run(const AttnArgs& a, hipStream_t stream) {
  const SlotGrid g = slot_grid(a.N, a.max_segs, Shape<kS>::BM);
  const dim3 blocks(uint32_t(slot_blocks(g, a.H) + tail_groups(a.N * a.H * D * 2)));
  attn_fwd_kernel<D, kS, kWin><<<blocks, dim3(kThreads), 0, stream>>>(
      static_cast<const bf16*>(a.q), static_cast<const bf16*>(a.k), static_cast<const bf16*>(a.v), a.cu, a.max_segs,
      a.N, a.H, a.Hkv, a.scale, static_cast<bf16*>(a.o), a.lse, a.flags, g, a.window, a.sinks);
}

hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t stream) {
  // (a window that no segment is longer than hides nothing)
  if (a.window > 0 && a.window < a.N) {
    a.D == 64 ? run<64, 1, true>(a, stream) : run<128, 1, true>(a, stream);
    return hipGetLastError();
  }
  // With few work-groups the longest walk over the keys sets the time, and waves that
  // share queries make it shorter; with many, or with many short walks, their joins
  // cost more than they save. Only the length of a call's one slot is known here, and
  // taken for N: a prompt with empty slots behind it takes kS = 1. kS = 2 / 1,
  // one segment, D 64: 1024 tokens, H 8 (64 tiles) 12.9 / 19.7 us; 4096, H 8 (256)
  // 40.0 / 65.1; 8192, H 8 (512) 98 / 129; 8192, H 16 (1024) 187 / 172; 512, H 8
  // 10.4 / 12.2 (8 to 10 of them the host's). D 128 (one work-group per compute unit):
  // 1024, H 8 (64) 19.8 / 25.0; 4096, H 4 (128) 58.5 / 82.5; 1024, H 32 (256)
  // 28.8 / 26.9; 77 tokens 10.0 / 10.0. 4096 tokens in 20 segments, H 8, D 128:
  // 27.6 / 14.3 us.
  const int64_t tiles = a.N / 128 * a.H;
  const bool share = a.max_segs == 1 && a.N >= 1024 && (a.D == 64 ? tiles <= 512 : tiles < 256);
  if (a.D == 64)
    share ? run<64, 2>(a, stream) : run<64, 1>(a, stream);
  else
    share ? run<128, 2>(a, stream) : run<128, 1>(a, stream);
  return hipGetLastError();
}

}  // namespace pkv
