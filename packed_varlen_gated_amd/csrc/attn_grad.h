// What the two reverse passes of packed softmax attention share (attn_bwd.hip, and
// attn_window_bwd.hip through a window): their tiles in LDS and the operands read from them.
#pragma once

#include "mfma.h"
#include "segments.h"

namespace pkv {
namespace {

constexpr int kB = 128;   // queries, or keys, that a work-group owns
constexpr int kT = 64;    // tokens of a tile of the other side
constexpr int kThreads = 256;

template <int D>
struct Lds {
  static constexpr int CH = D / 8, ROW = D * 2, BYTES = kT * ROW;
  static __device__ __forceinline__ int swz(int row) {
    return D == 128 ? ((row & 3) << 2) | ((row >> 2) & 3) : ((row & 2) << 1) | ((row >> 2) & 3);
  }
};

// The lane's part in loading a tile of T rows: its first chunk; the others are
// whole multiples of 16 rows further (the swizzle's period).
template <int D, int T, int NT>
struct Loader {
  static constexpr int LD = T * Lds<D>::CH / NT, STEP = NT / Lds<D>::CH;
  static_assert(STEP % 16 == 0, "the swizzle repeats");
  uint32_t off, step;
  __device__ __forceinline__ Loader(int32_t stride, int tid) {
    const int row = tid / Lds<D>::CH, pos = tid % Lds<D>::CH;
    off = uint32_t(row) * stride + (pos ^ Lds<D>::swz(row)) * 16;
    step = uint32_t(STEP) * stride;
  }
  __device__ __forceinline__ void issue_async(u32x4 r, char* dst, int wave) const {
    uint32_t o[LD];
    o[0] = fresh(off);
#pragma unroll
    for (int i = 1; i < LD; ++i) o[i] = o[0] + i * step;
    load_lds16_async<LD, NT * 16>(r, o, lds_addr(dst) + wave * 1024);
  }
  __device__ __forceinline__ void issue(__amdgpu_buffer_rsrc_t r, char* dst, int wave) const {
    const uint32_t o = fresh(off);
#pragma unroll
    for (int i = 0; i < LD; ++i) load_lds16(r, o + i * step, dst + wave * 1024 + i * NT * 16);
  }
};

// Operand reads from a tile (of 1024-byte alignment): rows 32 j + lane % 32
// (contraction over channels, step i of 16), and transposed: channels
// 32 i + lane % 32 (contraction over the rows of 16-row step j, in the order of
// a product's result registers). The swizzle is an XOR of address bits that the
// step only flips: an address register per read kind, not one per step.
template <int D>
struct Reader {
  int col, half;
  uint32_t row0, tr0, tr1;
  __device__ __forceinline__ Reader(int tid) {
    const int lane = tid & 63;
    half = lane >> 5;
    col = lane & 31;
    row0 = col * Lds<D>::ROW + (half ^ Lds<D>::swz(col)) * 16;
    const int r = 4 * half + ((lane & 15) >> 2), c = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
    tr0 = r * Lds<D>::ROW + (lane & 1) * 8 + (c ^ Lds<D>::swz(r)) * 16;
    tr1 = (r + 8) * Lds<D>::ROW + (lane & 1) * 8 + (c ^ Lds<D>::swz(r + 8)) * 16;
  }
  __device__ __forceinline__ bf16x8 rows(uint32_t t, int j, int i) const {
    return read_lds8(((t + row0) ^ (32 * i)) + 32 * j * Lds<D>::ROW);
  }
  __device__ __forceinline__ bf16x8 channels(uint32_t t, int i, int j) const {
    return join(read_tr(((t + tr0) ^ (64 * i)) + 16 * j * Lds<D>::ROW),
                read_tr(((t + tr1) ^ (64 * i)) + 16 * j * Lds<D>::ROW));
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
  for (int i = rd.half * 32 + rd.col; i < 32 * CH; i += 64) {
    const int r = i / CH, ch = i % CH;
    if (r < have)
      *reinterpret_cast<i32x4*>(dst + r * stride + ch * 8) =
          *reinterpret_cast<const i32x4*>(st + r * ROW + ((ch ^ (r & (CH - 1))) * 16));
  }
}

}  // namespace
}  // namespace pkv
