// Tiles of packed segments without a plan (shared by the attention and
// linear-attention kernels).
//
// Segment i covers tokens [cu[i], cu[i+1]) and is cut into tiles of BM tokens
// aligned to its start. Tile t of segment i has slot floor(cu[i] / BM) + i + t.
// ceil(n / BM) <= floor((c + n) / BM) - floor(c / BM) + 1 for every c and n,
// so the slots of different segments never meet, all slots lie in
// [0, floor(N / BM) + max_segs), and the first slot of segment i grows with i:
// a work-group finds its segment by a search over cu. There is no planning
// launch and no workspace; the slots that no tile has end at once.
#pragma once

#include "common.h"

namespace pkv {

// The work-groups of a call. A batch with many empty segment slots has many slots
// without a tile, and a work-group that only finds that out still costs its
// dispatch (30000 of them 40 us). The first `near` slots, enough for segments of
// a tile's length on average, get a work-group per head; the ones behind them,
// real only when most segments are shorter, one for kFarHeads heads.
constexpr int kFarHeads = 8;
struct SlotGrid {
  int32_t slots, near;
};
inline SlotGrid slot_grid(int64_t N, int64_t max_segs, int64_t bm) {
  const int64_t few = N / bm < 64 ? 64 : N / bm;
  return {int32_t(N / bm + max_segs), int32_t(N / bm + (max_segs < few ? max_segs : few))};
}
__host__ __device__ inline int64_t slot_blocks(const SlotGrid& g, int32_t heads) {
  return int64_t(g.near) * heads + int64_t(g.slots - g.near) * ((heads + kFarHeads - 1) / kFarHeads);
}
// The slot and heads [h0, h1) of work-group b.
__device__ __forceinline__ void slot_of(const SlotGrid& g, int64_t b, int32_t heads, int32_t& slot, int32_t& h0,
                                        int32_t& h1) {
  // (those of several heads start first)
  const int32_t per = (heads + kFarHeads - 1) / kFarHeads;
  const int64_t far = int64_t(g.slots - g.near) * per;
  if (b >= far) {
    slot = int32_t((b - far) / heads);
    h0 = int32_t((b - far) % heads);
    h1 = h0 + 1;
  } else {
    slot = g.near + int32_t(b / per);
    h0 = int32_t(b % per) * kFarHeads;
    h1 = h0 + kFarHeads < heads ? h0 + kFarHeads : heads;
  }
}

struct SegTile {
  int32_t seg;    // segment slot
  int32_t start;  // first token of the tile
  int32_t a, e;   // the segment's tokens [a, e)
};

inline int64_t tile_slots(int64_t N, int64_t max_segs, int64_t bm) { return N / bm + max_segs; }

// Whether cu[i], cu[i+1] bound a segment inside [0, N).
__device__ __forceinline__ bool segment_ok(int32_t i, int64_t a, int64_t e, int64_t N) {
  return a >= 0 && e >= a && e <= N && (i != 0 || a == 0);
}

// The last segment i < max_segs with floor(cu[i] / bm) + inc * i <= key, and its
// bounds; false when there is none. Every lane of the wave takes part (64 probes
// a round, so 2 rounds up to 4096 segments) and gets the same answer. A
// malformed cu gives some segment.
__device__ __forceinline__ bool find_segment(const int32_t* __restrict__ cu, int32_t max_segs, int32_t bm,
                                             int32_t inc, int32_t key, int32_t& seg, int32_t& a, int32_t& e) {
  const int lane = threadIdx.x & 63;
  int32_t lo = 0, hi = max_segs;  // the segment is in [lo, hi)
  for (;;) {
    const int32_t step = (hi - lo + 63) >> 6;
    const int64_t i = int64_t(lo) + int64_t(lane) * step;
    const int32_t c = cu[i < hi ? i : hi];  // (cu holds max_segs + 1)
    const bool le = i < hi && int64_t(c < 0 ? 0 : c / bm) + inc * i <= key;
    const uint64_t m = ~__builtin_amdgcn_ballot_w64(le);
    const int n = m == 0 ? 64 : __builtin_ctzll(m);
    if (n == 0) return false;
    lo = lo + (n - 1) * step;
    if (step == 1) {
      seg = __builtin_amdgcn_readfirstlane(lo);
      a = __builtin_amdgcn_readlane(c, n - 1);
      // the probe after it holds its end (or, past lane 63, memory does)
      e = n < 64 ? __builtin_amdgcn_readlane(c, n) : cu[seg + 1];
      e = __builtin_amdgcn_readfirstlane(e);
      return true;
    }
    if (hi - lo > step) hi = lo + step;
  }
}

// The tile of a slot; false when the slot has none. Every lane of the wave
// takes part (64 probes a round, so 2 rounds up to 4096 segments) and gets the
// same answer. A malformed cu gives some answer within [0, N) or none.
__device__ __forceinline__ bool find_tile(const int32_t* __restrict__ cu, int32_t max_segs,
                                          int64_t N, int32_t bm, int32_t slot, SegTile& t) {
  if (cu == nullptr) {
    const int64_t s = int64_t(slot) * bm;
    if (s >= N) return false;
    t.seg = 0;
    t.start = int32_t(s);
    t.a = 0;
    t.e = int32_t(N);
    return true;
  }
  int32_t lo, a, e;
  if (!find_segment(cu, max_segs, bm, 1, slot, lo, a, e)) return false;
  if (!segment_ok(lo, a, e, N)) return false;
  const int64_t s = a + (int64_t(slot) - (a / bm + lo)) * bm;
  if (s < a || s >= e) return false;
  t.seg = lo;
  t.start = int32_t(s);
  t.a = a;
  t.e = e;
  return true;
}

// The number of tokens that cu covers, clamped to [0, N].
__device__ __forceinline__ int64_t covered_tokens(const int32_t* __restrict__ cu, int32_t max_segs,
                                                  int64_t N) {
  if (cu == nullptr) return N;
  const int64_t c = cu[max_segs];
  return c < 0 ? 0 : (c > N ? N : c);
}

// Work-groups behind those of the slots, which zero the rows that no segment has
// (and copy the states of empty slots): one per 64 KiB that there may be to write,
// at most 256, so that a small call does not wait for them.
inline int64_t tail_groups(int64_t bytes) { return bytes >> 16 < 255 ? (bytes >> 16) + 1 : 256; }

// One work-group's check of the whole cu: sets kFlagBadCuSeqlens.
__device__ __forceinline__ void check_cu(const int32_t* __restrict__ cu, int32_t max_segs, int64_t N,
                                         int32_t* __restrict__ flags) {
  if (cu == nullptr || flags == nullptr) return;
  bool bad = false;
  for (int64_t i = threadIdx.x; i < max_segs; i += blockDim.x)
    bad |= !segment_ok(int32_t(i), cu[i], cu[i + 1], N);
  if (bad) atomicOr(flags, kFlagBadCuSeqlens);
}

// Zeroes rows [covered, N) of a [N, width]-byte tensor; part j of n of the
// work (16-byte stores; width is a multiple of 16).
__device__ __forceinline__ void zero_tail(void* base, int64_t covered, int64_t N, int64_t width,
                                          int64_t j, int64_t n) {
  typedef int v4 __attribute__((ext_vector_type(4)));
  v4* p = reinterpret_cast<v4*>(static_cast<char*>(base) + covered * width);
  const int64_t total = (N - covered) * (width / 16);
  for (int64_t i = j * blockDim.x + threadIdx.x; i < total; i += n * blockDim.x) p[i] = v4{0, 0, 0, 0};
}

}  // namespace pkv
