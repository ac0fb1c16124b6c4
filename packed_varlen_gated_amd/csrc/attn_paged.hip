// Attention of new tokens over the paged cache on the matrix cores (bf16, D in
// {64, 128}).
//
//   o_t = sum_s softmax_s(scale q_t.k_s) v_s over the places s <= t of t's request,
//   with a window those with t - s < window or s < sinks.
//
// Row i of a (request, kv head) is its new token i / rep under query head i % rep of
// the group: the heads that share keys share their loads. Two forms:
//   small  at most 32 rows (decoding): a work-group's four waves hold the same rows
//          and take 16 (D 64: 32) keys each of a block; every wave streams its keys through
//          LDS of its own (no barrier in the walk), and the sums are joined at the end.
//   big    tiles of 256 rows (chunks of prompts): a wave holds 32 rows, the eight
//          share blocks of 64 keys, four waves loading K and four V. A walk is that of the
//          packed kernel (attn_fwd.hip): S^T = K Q^T, P = 2^(c S - m), O^T += V^T P^T, O
//          rescaled only when a row's maximum grew by more than 2^8.
//
// The small form is bound by the bytes of the cache that are seen, read once. Every wave
// has two blocks in flight (the waits are written here: the compiler's own, before a read
// of LDS behind a load into LDS, would wait for both). One request of 131072 tokens, H 32,
// Hkv 8, D 128: 108 us for 0.54 GB, 5.0 TB/s of the 5.13 that a large copy reaches. 64 requests
// of about 2000 tokens, the longest 16384: 145 us for 0.69 GB, 4.8 TB/s. 128 requests with
// a window of 1024, H 16, Hkv 4, D 64: 38 us for 0.13 GB; a work-group has about 9 blocks
// there, and its start (the scan over the requests), the parts' sums and the join are the rest.
// The big form is bound by matrix instructions and what feeds them: 2048 new tokens behind
// 27953 others, H 32, Hkv 8, D 128: 984 us, 989 TFLOP/s, where a product of 8192^3 reaches
// 1233. With tiles of 128 rows and four waves, each key was loaded twice as often: 1080 us.
// Loads into LDS take about a fifth of it, reads of LDS a tenth, 2^x nothing (each left out
// in turn).
//
// Lengths are on the device and differ widely, so the work is dealt there: a tile's
// blocks of keys are units, all units of the call are in one order (kv head, request,
// tile, block), and work-group w takes units [w per, (w + 1) per) of it, the last
// part of one tile, whole tiles, the first part of another. A tile that is cut leaves
// its parts' sums in the workspace (two for each work-group at most) and a second
// launch joins them. Every work-group finds its place by one scan over the requests.
// In the big form a chunk's later tiles have more blocks than its earlier ones; tile i
// and tile J - 1 - i together have nearly the same number for all i, so such a pair is
// what a request has equal ones of.
//
// Pages are multiples of 16 places and a wave's loads go by 16 of them: one page and
// one buffer descriptor for each 16 keys, whose size ends at the request's last token,
// so that nothing else of a page is read.
//
// A weight of 0 times a value that is not finite is NaN. When a sum of a part is not
// finite the part is walked again with such values as 0, and then they are added to
// the rows that see them.

#include "mfma.h"
#include "paged.h"

#include <float.h>

namespace pkv {
namespace {

constexpr int kThreads = 256;  // of the join
constexpr int32_t kPlaces = 1 << 29;  // of a request
constexpr float kGrow = 8.f;  // log2 of what a row's maximum may grow by before O is rescaled

template <int D, bool kBig>
struct Form {
  static constexpr int NT = kBig ? 512 : 256;                 // threads
  static constexpr int BM = kBig ? 256 : 32;                  // rows of a tile
  static constexpr int KW = kBig ? 64 : D == 128 ? 16 : 32;   // keys of a wave in a block
  static constexpr int BK = kBig ? 64 : 4 * KW;               // keys of a block
  static constexpr int HALF = KW * D * 2;                     // bytes of a block's K (or V) in LDS, of a wave or of all
  static constexpr int STAGE = 2 * HALF * (kBig ? 1 : 4);     // of a block
  static constexpr int GROUPS = kBig ? 256 : 512;             // at most: what the chip holds at a time
  static constexpr int LEAST = 2;  // units of a work-group (4: a prompt of 128 tokens 38 us instead of 27)
  // the parts' sums in the workspace: two of a work-group, [BM, D] and [BM, 2] m, l
  static constexpr size_t STATS = size_t(2) * GROUPS * BM * D;
  static constexpr size_t PARTS = (STATS + size_t(2) * GROUPS * BM * 2) * 4;
};

// A cut tile, written by the work-group where its second part lies.
struct Cut {
  int32_t last;  // work-group of the last part; -1: there is no tile whose second part is here
  int32_t rows, hk, rep_first, a, rep_mod;  // its rows, from row rep_first * rep + rep_mod of the request on
};

template <int D>
struct Swz {
  static constexpr int CH = D / 8;  // 16-byte chunks of a row
  static __device__ __forceinline__ int k(int row) { return D == 128 ? row & 15 : (row >> 1) & 7; }
  static __device__ __forceinline__ int v(int row) { return D == 128 ? (row & 3) << 2 : (row & 2) << 1; }
};

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= FLT_MAX; }
__device__ __forceinline__ int32_t uni(int32_t x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uni(int64_t x) {
  return int64_t(uint64_t(uint32_t(uni(int32_t(x)))) | uint64_t(uint32_t(uni(int32_t(x >> 32)))) << 32);
}

// What a tile's rows see.
struct Span {
  int32_t lo, hi;  // places of its first and last row
  int32_t blocks;  // at least 1
  WindowWalk ww;
};
template <int BM, int BK>
__device__ __forceinline__ Span span_of(const Request& q, int32_t rep, int32_t window, int32_t sinks, int32_t j) {
  const int32_t first = q.len - q.n;
  const int64_t last = int64_t(BM) * (j + 1) - 1, rows = int64_t(q.n) * rep;
  const int32_t lo = first + int32_t(int64_t(BM) * j / rep);
  const int32_t hi = first + int32_t((last < rows ? last : rows - 1) / rep);
  const WindowWalk ww(window > 0 ? window : 0x7fffffff, window > 0 ? sinks : 0, BK, lo > 0 ? lo : 0, 0);
  return {lo, hi, hi < 0 ? 1 : ww.count(hi / BK + 1), ww};
}

// A request's part in the call: `pairs` (small form: its one tile) of `cost` units.
struct Share {
  Request q;
  int32_t tiles, pairs, cost;
  __device__ __forceinline__ int64_t units() const { return int64_t(pairs) * cost; }
};
template <int D, bool kBig>
__device__ __forceinline__ Share share_of(const PagedArgs& c, const AttnPagedArgs& x, int32_t r) {
  using F = Form<D, kBig>;
  const int32_t rep = x.Hq / c.Hkv;
  Share s{request(c, r), 0, 0, 0};
  const int64_t rows = int64_t(s.q.n) * rep;
  if (rows == 0 || (rows > 32) != kBig) return s;
  if constexpr (!kBig) {
    s.tiles = s.pairs = 1;
    s.cost = span_of<F::BM, F::BK>(s.q, rep, x.window, x.sinks, 0).blocks;
    return s;
  }
  s.tiles = int32_t((rows + F::BM - 1) / F::BM);
  s.pairs = (s.tiles + 1) / 2;
  // Without a window a tile's blocks are a rounded linear function of its number, at
  // least 1 (the last tile's are fewer, where it is not full, by BM / BK at most): the sum
  // over a pair is at most that of the outermost one, 2 and what the last tile lacks. With
  // one no tile has more than its window, its tokens and its sinks need.
  const int32_t a = span_of<F::BM, F::BK>(s.q, rep, 0, 0, 0).blocks +
                    span_of<F::BM, F::BK>(s.q, rep, 0, 0, s.tiles - 1).blocks;
  s.cost = s.tiles == 1 ? a / 2 : a + 3 + F::BM / F::BK;
  if (x.window > 0) {
    const int64_t most = (int64_t(x.window) + F::BM / rep + 1) / F::BK + 2 + (x.sinks + F::BK - 1) / F::BK;
    const int64_t b = (s.tiles == 1 ? 1 : 2) * most;
    s.cost = b < s.cost ? int32_t(b) : s.cost;
  }
  return s;
}

// The same in every lane: kept in scalar registers.
__device__ __forceinline__ Share uniform(const Share& s) {
  return {{uni(s.q.a), uni(s.q.n), uni(s.q.len), s.q.ok}, uni(s.tiles), uni(s.pairs), uni(s.cost)};
}

// The sum over the work-group's threads, and over those before this one.
template <int NT>
__device__ __forceinline__ int64_t scan(int64_t x, int64_t& before, int64_t* lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t s = x;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int64_t y = __shfl_up(s, d, 64);
    if (lane >= d) s += y;
  }
  __syncthreads();  // the last scan's readers are done
  if (lane == 63) lds[wave] = s;
  __syncthreads();
  int64_t base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) {
    base += w < wave ? lds[w] : 0;
    all += lds[w];
  }
  before = base + s - x;
  return uni(all);
}

// The order of the call's units, and a place in it.
template <int D, bool kBig>
struct Place {
  int64_t per_head;  // units of a kv head
  int64_t per;       // units of a work-group
  int32_t hk, r;     // the place's kv head and request
  int64_t at;        // the request's first unit (of all)
  Share s;           // the request

  // All threads of the work-group; units of the call and the place of unit `per` w.
  // False where there is none.
  __device__ __forceinline__ bool find(const PagedArgs& c, const AttnPagedArgs& x, int64_t w, int64_t groups,
                                       int64_t& unit) {
    constexpr int NT = Form<D, kBig>::NT;
    __shared__ int64_t lds[NT / 64 + 2];
    int64_t mine = 0, before, total = 0;
    if (threadIdx.x == 0) lds[NT / 64] = -1;
    for (int32_t r0 = 0; r0 < c.R; r0 += NT) {
      const int32_t i = r0 + int32_t(threadIdx.x);
      mine = i < c.R ? share_of<D, kBig>(c, x, i).units() : 0;
      total += scan<NT>(mine, before, lds);
    }
    per_head = total;
    const int64_t all = total * c.Hkv;
    per = (all + groups - 1) / groups;
    per = per < Form<D, kBig>::LEAST ? Form<D, kBig>::LEAST : per;
    unit = per * w;
    if (unit >= all) return false;
    hk = int32_t(unit / total);
    const int64_t y = unit - hk * total;
    int64_t base = 0;
    for (int32_t r0 = 0; r0 < c.R; r0 += NT) {
      if (c.R > NT) {  // (else the scan above is the one needed)
        const int32_t i = r0 + int32_t(threadIdx.x);
        mine = i < c.R ? share_of<D, kBig>(c, x, i).units() : 0;
        total = scan<NT>(mine, before, lds);
      }
      if (y >= base + before && y < base + before + mine) {
        lds[NT / 64] = r0 + int32_t(threadIdx.x);
        lds[NT / 64 + 1] = base + before;
      }
      base += total;
      if (y < base) break;
    }
    __syncthreads();
    r = uni(int32_t(lds[NT / 64]));
    if (r < 0) return false;  // (as in `next`)
    at = int64_t(hk) * per_head + uni(lds[NT / 64 + 1]);
    s = uniform(share_of<D, kBig>(c, x, r));
    return true;
  }

  // The next request with units, 64 at a time. False where there is none, which only a
  // caller sees that changes the lengths under a running call: it ends all the same.
  __device__ __forceinline__ bool next(const PagedArgs& c, const AttnPagedArgs& x) {
    at += s.units();
    ++r;
    for (;;) {
      if (r >= c.R) {
        r = 0;
        if (++hk >= c.Hkv) return false;
      }
      const int32_t i = r + int32_t(threadIdx.x & 63);
      const uint64_t m = __builtin_amdgcn_ballot_w64(i < c.R && share_of<D, kBig>(c, x, i).pairs > 0);
      if (m != 0) {
        r = uni(r + int32_t(__builtin_ctzll(m)));
        break;
      }
      r += 64;
    }
    s = uniform(share_of<D, kBig>(c, x, r));
    return s.pairs > 0;
  }
};

// A part of a tile that begins at unit `unit`: its tile, and blocks [b0, b1) of it as
// far as the tile goes; where the unit is one of the spare ones of a pair, b0 = b1.
// `skip`: units from `unit` to the next tile.
struct Part {
  int32_t j;
  Span sp;
  int32_t b0;
  int64_t skip;
};
template <int D, bool kBig>
__device__ __forceinline__ Part part_at(const Place<D, kBig>& pl, const AttnPagedArgs& x, int32_t rep, int64_t unit) {
  using F = Form<D, kBig>;
  const Share& s = pl.s;
  const int64_t off = unit - pl.at;
  if constexpr (!kBig) {
    const Span sp = span_of<F::BM, F::BK>(s.q, rep, x.window, x.sinks, 0);
    return {0, sp, int32_t(off), sp.blocks - off};
  }
  const int32_t i = int32_t(off / s.cost), in = int32_t(off - int64_t(i) * s.cost);
  const int32_t ja = s.tiles - 1 - i;
  Span sp = span_of<F::BM, F::BK>(s.q, rep, x.window, x.sinks, ja);
  if (in < sp.blocks) return {ja, sp, in, sp.blocks - in};
  const int32_t past = sp.blocks;
  if (ja != i) {
    sp = span_of<F::BM, F::BK>(s.q, rep, x.window, x.sinks, i);
    if (in < past + sp.blocks) return {i, sp, in - past, past + sp.blocks - in};
  }
  return {-1, sp, 0, s.cost - in};
}

// A launch's arguments. They are read again (scalar loads) for each part of the work: held in
// registers over a walk, they would push more of what the walk needs out of them. At D 128 its
// own are still too many: 106 (small form) and 117 (big) scalar registers are kept in vector
// lanes, some of them read back for every block (D 64: 11 and 4).
struct Launch {
  PagedArgs c;
  AttnPagedArgs x;
  float* sums;
  Cut* cuts;
  int64_t groups;
};
typedef __attribute__((address_space(4))) void* KernelArgs;
__device__ __forceinline__ Launch reload(KernelArgs& p) {
  asm volatile("" : "+s"(p));
  return *(const Launch*)p;
}

template <int D, bool kBig>
__global__ __launch_bounds__((Form<D, kBig>::NT), 2) void attn_paged_kernel(const Launch launch) {
  using F = Form<D, kBig>;
  constexpr int CH = Swz<D>::CH, KS = D / 16, DT = D / 32, NJ = (F::KW + 31) / 32;
  constexpr int NR = F::KW == 16 ? 8 : 16;  // registers of a product of 32 keys (8: of its first 16) that are used
  constexpr int NT = F::NT;
  constexpr int GR = kBig ? 1 : F::KW / 16;  // granules of 16 keys that a wave loads of a block
  constexpr int GL = 16 * CH / 64;           // loads of a granule of K (and of V)
  constexpr int RL = 16 / GL;                // rows of a load
  constexpr int JOIN = kBig ? 0 : 4 * 32 * (D + 6) * 4;  // the waves' sums are joined in the stages
  __shared__ __attribute__((aligned(1024))) char lds[2 * F::STAGE > JOIN ? 2 * F::STAGE : JOIN];
  __shared__ Share shares[NT / 64];  // the request, of every wave

  const int64_t b = blockIdx.x;
  if (b >= launch.groups) {
    const PagedArgs& c = launch.c;
    const AttnPagedArgs& x = launch.x;
    const int64_t j = b - launch.groups, n = gridDim.x - launch.groups, end = covered_tokens(c.cu, c.R, c.N);
    zero_tail(x.o, end, c.N, int64_t(x.Hq) * D * 2, j, n);
    if (x.lse != nullptr)
      for (int64_t i = j * NT + threadIdx.x; i < (c.N - end) * x.Hq; i += n * NT)
        x.lse[(i / (c.N - end)) * c.N + end + i % (c.N - end)] = -INFINITY;
    if (j == 0) check_requests(c);
    return;
  }
  // Consecutive work-groups run on different XCDs: units that share keys go to one.
  const int32_t w = kBig ? int32_t(b) % 8 * (F::GROUPS / 8) + int32_t(b) / 8 : int32_t(b);
  KernelArgs args = (KernelArgs)__builtin_amdgcn_kernarg_segment_ptr();
  Place<D, kBig> pl;
  int64_t unit, end;
  if (threadIdx.x == 0) launch.cuts[w].last = -1;
  if (!pl.find(launch.c, launch.x, w, launch.groups, unit)) return;
  {
    const int64_t all = pl.per_head * launch.c.Hkv;
    end = unit + pl.per < all ? unit + pl.per : all;
    // the tile whose second part is here
    const int32_t rep = launch.x.Hq / launch.c.Hkv;
    const Part pt = part_at<D, kBig>(pl, launch.x, rep, unit);
    if (pt.j >= 0 && pt.b0 > 0 && unit - pt.b0 >= unit - pl.per && threadIdx.x == 0) {
      const int64_t row0 = int64_t(pt.j) * F::BM, left = int64_t(pl.s.q.n) * rep - row0;
      launch.cuts[w] = {int32_t((unit - pt.b0 + pt.sp.blocks - 1) / pl.per),
                        left < F::BM ? int32_t(left) : F::BM,
                        pl.hk,
                        int32_t(row0 / rep),
                        pl.s.q.a,
                        int32_t(row0 % rep)};
    }
  }
  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
  const int half = lane >> 5, col = lane & 31;
  shares[wave] = pl.s;

  // the lane's place in a load: row lrow of RL, chunk lpos
  const int lrow = lane / CH, lpos = lane % CH;
  // (in the big form waves 0 to 3 load K, the others V)
  const bool loads_v = kBig && wave >= 4;
  // LDS addresses of the lane's operand chunks
  const int kx = Swz<D>::k(col);
  const int vr = 4 * half + ((lane & 15) >> 2), vc = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1), vb = (lane & 1) * 8;
  const int vx = Swz<D>::v(vr);

  const int32_t wrow = kBig ? wave * 32 : 0;  // the wave's first row in a tile
  // The part at `unit`, the wave's rows of its tile and the lane's row: its token and head
  // (of the tile's first row where there is none). Formed where they are needed: a walk,
  // another one and the outputs each have their own and hold nothing for one another.
  struct Piece {
    Launch a;
    Share s;
    Part pt;
    int32_t rep, b1, mine, tok, head;
  };
  auto piece = [&] {
    Piece p;
    p.a = reload(args);
    asm volatile("" ::: "memory");
    p.rep = p.a.x.Hq / p.a.c.Hkv;
    pl.s = p.s = uniform(shares[wave]);
    p.pt = part_at<D, kBig>(pl, p.a.x, p.rep, unit);
    p.b1 = p.pt.skip < end - unit ? p.pt.sp.blocks : int32_t(p.pt.b0 + (end - unit));
    const int64_t row0 = int64_t(p.pt.j) * F::BM, left = int64_t(p.s.q.n) * p.rep - row0;
    p.mine = (left < F::BM ? int32_t(left) : F::BM) - wrow;
    const int64_t row = col < p.mine ? row0 + wrow + col : row0;
    p.tok = int32_t(row / p.rep);
    p.head = pl.hk * p.rep + int32_t(row % p.rep);
    return p;
  };

  while (unit < end) {
    {
      const Launch a = reload(args);
      asm volatile("" ::: "memory");
      pl.s = uniform(shares[wave]);
      if (unit >= pl.at + pl.s.units()) {
        if (!pl.next(a.c, a.x)) return;
        shares[wave] = pl.s;
        continue;
      }
      const Part pt = part_at<D, kBig>(pl, a.x, a.x.Hq / a.c.Hkv, unit);
      if (pt.j < 0) {
        unit += pt.skip;
        continue;
      }
    }
    f32x16 acc[DT];
    float m = -FLT_MAX, l = 0.f;

    // mode 0: the sums; 1: with values that are not finite as 0; 2: those values added.
    // Whether some sum of the lane's row is not finite.
    auto walk = [&](int mode) {
      const Piece pc = piece();
      const Launch& a = pc.a;
      const Part& pt = pc.pt;
      const int32_t mine = pc.mine, tok = pc.tok, head = pc.head, b0 = pt.b0, b1 = pc.b1;
      pl.s = pc.s;
      // (a place is below kPlaces: no window is one of that many)
      const int32_t window = a.x.window > 0 && a.x.window < kPlaces ? a.x.window : kPlaces;
      const int32_t sinks = a.x.window > 0 ? a.x.sinks : 0;
      const int32_t place = col < mine ? pl.s.q.len - pl.s.q.n + tok : -1;
      // places of the wave's first and last row
      const int32_t wlo = uni(place);
      const int32_t whi = __builtin_amdgcn_readlane(place, mine >= 32 ? 31 : (mine > 0 ? mine - 1 : 0));
      const bool rows_here = mine > 0;
      const float cs = a.x.scale == 0.f ? 1.f : fabsf(a.x.scale) * kLog2e;  // (as in attn_fwd.hip)

      bf16x8 qf[KS];
      {
        const uint32_t flip = a.x.scale < 0.f ? 0x80008000u : 0u, keep = a.x.scale == 0.f ? 0u : ~0u;
        const bf16* q = static_cast<const bf16*>(a.x.q) + ((int64_t(pl.s.q.a) + tok) * a.x.Hq + head) * D + half * 8;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          i32x4 y = {0, 0, 0, 0};
          if (col < mine) y = *reinterpret_cast<const i32x4*>(q + i * 16);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = int((uint32_t(y[e]) ^ flip) & keep);
          qf[i] = __builtin_bit_cast(bf16x8, y);
        }
      }
      const int32_t ps = a.c.page_size, num_pages = a.c.num_pages, kstride = a.c.Hkv * D * 2;
      const char* kbase = static_cast<const char*>(a.x.k_pages) + int64_t(pl.hk) * D * 2;
      const char* vbase = static_cast<const char*>(a.x.v_pages) + int64_t(pl.hk) * D * 2;
      const int32_t wkey = kBig ? 16 * (wave & 3) : F::KW * wave;  // the wave's first key to load of a block
      uint32_t koff[GL], voff[GL];
#pragma unroll
      for (int u = 0; u < GL; ++u) {
        const int row = RL * u + lrow;
        koff[u] = row * kstride + uint32_t(lpos ^ (loads_v ? Swz<D>::v(row) : Swz<D>::k(row))) * 16;
        voff[u] = row * kstride + uint32_t(lpos ^ Swz<D>::v(row)) * 16;
      }
      const int32_t far = pt.sp.ww.far, low = pt.sp.ww.low - far;
      // (a granule past `oldest` is in the window)
      const int32_t limit = pt.sp.hi + 1, oldest = pt.sp.lo - window - 15;
      auto first_key = [&](int32_t blk) { return (blk < far ? blk : blk + low) * F::BK; };
      // 64 entries of the request's row of the table from `ids0` on, one a lane: loads of
      // entries would make every block wait for all loads before them
      int32_t ids = 0, ids0 = -64;
      // page and place in it of the wave's first key of the block to load next
      int32_t npg = 0, no = 0;
      const int32_t step_pg = F::BK / ps, step_o = F::BK % ps;
      auto issue = [&](int32_t blk, int st, bool start) {
        const uint32_t dst = lds_addr(lds) + st * F::STAGE +
                             (kBig ? (wave & 3) * (16 * D * 2) + (loads_v ? F::HALF : 0) : wave * 2 * F::HALF);
        const int32_t key = first_key(blk) + wkey;
        if (start || blk == far) {
          npg = key / ps;
          no = key - npg * ps;
        }
        int32_t pg = npg, o = no;
#pragma unroll
        for (int g = 0; g < GR; ++g) {
          const int32_t first = key + 16 * g, left = limit - first;
          // (what no row of the tile sees is not loaded)
          const bool seen = left > 0 && (first > oldest || first < sinks);
          if (seen && (pg < ids0 || pg >= ids0 + 64)) {
            const Launch a = reload(args);
            ids0 = pg;
            // (waited for here, not at every use)
            const int32_t at = pg + lane < a.c.max_pages ? pg + lane : a.c.max_pages - 1;
            ids = fresh(a.c.table[int64_t(pl.r) * a.c.max_pages + at]);
          }
          const int32_t page = __builtin_amdgcn_readlane(ids, (pg - ids0) & 63);
          const bool ok = seen && page >= 0 && page < num_pages;
          if (seen && !ok) {
            const Launch a = reload(args);
            if (a.c.flags != nullptr && lane == 0) atomicOr(a.c.flags, kFlagBadPage);
          }
          const int64_t from = ok ? int64_t(page * ps + o) * kstride : 0;
          const uint32_t bytes = ok ? ((left < 16 ? left : 16) - 1) * kstride + D * 2 : 0;
          load_lds16_async<GL, 1024>(descriptor((loads_v ? vbase : kbase) + from, bytes), koff, dst + g * (16 * D * 2));
          if constexpr (!kBig)
            load_lds16_async<GL, 1024>(descriptor(vbase + from, bytes), voff, dst + F::HALF + g * (16 * D * 2));
          o += 16;
          if (o == ps) {
            o = 0;
            ++pg;
          }
        }
        npg += step_pg;
        no += step_o;
        if (no >= ps) {
          no -= ps;
          ++npg;
        }
      };

      if (mode < 2) {
        m = -FLT_MAX;
        l = 0.f;
#pragma unroll
        for (int i = 0; i < DT; ++i) acc[i] = f32x16{};
      }
      issue(b0, 0, true);
      for (int32_t blk = b0; blk < b1; ++blk) {
        const int st = (blk - b0) & 1;
        if constexpr (kBig) {
          wait_vm();
          bar();
          if (blk + 1 < b1) issue(blk + 1, st ^ 1, false);
        } else {
          asm volatile("" ::: "memory");
          if (blk + 1 < b1) {
            issue(blk + 1, st ^ 1, false);
            wait_loads<2 * GR * GL>();
          } else {
            wait_loads<0>();
          }
          asm volatile("" ::: "memory");
        }
        char* kt = lds + st * F::STAGE + (kBig ? 0 : wave * 2 * F::HALF);
        char* vt = kt + F::HALF;
        const int32_t s0 = first_key(blk) + (kBig ? 0 : wkey);  // the wave's first key
        if (mode > 0) {
          // keys with a value that is not finite
          __shared__ uint64_t odd_lds[1];
          uint64_t odd = 0;
          if constexpr (kBig) {
            __syncthreads();
            if (tid == 0) odd_lds[0] = 0;
            __syncthreads();
          }
          for (int i = kBig ? tid : lane; i < F::HALF / 4; i += kBig ? NT : 64) {
            uint32_t y = reinterpret_cast<uint32_t*>(vt)[i];
            const bool p = (y & 0x7f80u) == 0x7f80u, e = (y & 0x7f800000u) == 0x7f800000u;
            if (p || e) odd |= uint64_t(1) << (i / (D / 2));
            if (mode == 1 && (p || e))
              reinterpret_cast<uint32_t*>(vt)[i] = y & (p ? 0xffff0000u : ~0u) & (e ? 0xffffu : ~0u);
          }
          if constexpr (kBig) {
            if (odd != 0) atomicOr(reinterpret_cast<unsigned long long*>(odd_lds), (unsigned long long)odd);
            __syncthreads();
            odd = odd_lds[0];
          } else {
#pragma unroll
            for (int d = 1; d < 64; d *= 2) odd |= uint64_t(__shfl_xor((long long)odd, d, 64));
            wait_all();
            asm volatile("" ::: "memory");
          }
          if (mode == 2) {
            for (int s = 0; s < F::KW; ++s) {
              if ((odd >> s & 1) == 0) continue;
              const int32_t p = s0 + s;
              const bool sees = p <= place && (place - p < window || p < sinks);
#pragma unroll
              for (int i = 0; i < DT; ++i)
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                  const int ch = 32 * i + 8 * (j / 4) + 4 * half + j % 4;
                  const float y = to_f32(*reinterpret_cast<const bf16*>(
                      vt + s * (D * 2) + (((ch / 8) ^ Swz<D>::v(s)) * 16) + ch % 8 * 2));
                  if (sees && !finite(y)) acc[i][j] += y;
                }
            }
            continue;
          }
        }
        if (!rows_here || s0 > whi || (s0 + F::KW - 1 <= wlo - window && s0 >= sinks)) continue;

        f32x16 s[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          s[j] = f32x16{};
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            const char* at = kt + (32 * j + col) * (D * 2) + (((2 * i + half) ^ kx) * 16);
            const bf16x8 y = *reinterpret_cast<const bf16x8*>(at);
            s[j] = mfma32(y, qf[i], s[j]);
          }
        }
        // (a wave of less than 32 rows has lanes that see nothing: their sums are not used)
        if (s0 + F::KW - 1 > wlo || s0 <= whi - window) {
          const int32_t last = place - s0 - 4 * half, old = last - window, sink = sinks - s0 - 4 * half;
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int i = 0; i < NR; ++i) {
              const int32_t k = 32 * j + 8 * (i / 4) + i % 4;
              s[j][i] = k <= last && (k > old || k < sink) ? s[j][i] : -INFINITY;
            }
        }
        float mx = s[0][0];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int i = 0; i < NR; ++i) mx = fmaxf(mx, s[j][i]);
        mx = fmaxf(mx, other_half(mx)) * cs;
        const bool grew = mx > m + kGrow;
        if (__builtin_amdgcn_ballot_w64(grew) != 0) {
          const float f = grew ? ex2(m - mx) : 1.f;
          m = grew ? mx : m;
          l *= f;
#pragma unroll
          for (int i = 0; i < DT; ++i)
#pragma unroll
            for (int j = 0; j < 16; ++j) acc[i][j] *= f;
        }
        bf16x8 p[F::KW / 16];
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int i = 0; i < NR; ++i) {
            const float y = ex2(fmaf(s[j][i], cs, -m));
            l += y;
            p[2 * j + i / 8][i % 8] = static_cast<bf16>(y);
          }
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int j = 0; j < F::KW / 16; ++j) {
            const char* y = vt + (16 * j + vr) * (D * 2) + (((4 * i + vc) ^ vx) * 16) + vb;
            acc[i] = mfma32(join(read_tr(y), read_tr(y + 8 * (D * 2))), p[j], acc[i]);
          }
      }
      bool bad = false;
      if (mode == 0) {
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int j = 0; j < 16; ++j) bad |= !finite(acc[i][j]);
      }
      return bad && place >= 0;
    };
    const bool bad = walk(0);
    // (in the big form also: every wave is done with the stages)
    if (kBig ? __syncthreads_or(bad) != 0 : __builtin_amdgcn_ballot_w64(bad) != 0) {
      walk(1);
      if constexpr (kBig) __syncthreads();
      walk(2);
      if constexpr (kBig) __syncthreads();
    }
    l += other_half(l);
    if constexpr (!kBig) __syncthreads();  // every wave is done with the stages

    // The tile's outputs, or the part's sums (a part with the tile's first block is the
    // work-group's last one, any other its first).
    const Piece pc = piece();
    const Launch& a = pc.a;
    const Share& sh = pc.s;
    const int32_t rep = pc.rep, mine = pc.mine, tok = pc.tok, head = pc.head, b0 = pc.pt.b0;
    const bool whole = b0 == 0 && pc.b1 == pc.pt.sp.blocks;
    const int64_t slot = 2 * int64_t(w) + (b0 == 0 ? 1 : 0);
    float* psum = a.sums + slot * F::BM * D;
    float* pst = a.sums + F::STATS + slot * F::BM * 2;
    bf16* o = static_cast<bf16*>(a.x.o);
    if constexpr (kBig) {
      if (col < mine) {
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // (NaN stays)
        bf16* to = o + ((int64_t(sh.q.a) + tok) * a.x.Hq + head) * D;
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int ch = 32 * i + 8 * j + 4 * half;
            if (whole) {
              bf16x4 y;
#pragma unroll
              for (int e = 0; e < 4; ++e) y[e] = static_cast<bf16>(acc[i][4 * j + e] * inv);
              *reinterpret_cast<bf16x4*>(to + ch) = y;
            } else {
              *reinterpret_cast<f32x4*>(psum + (wrow + col) * D + ch) =
                  f32x4{acc[i][4 * j], acc[i][4 * j + 1], acc[i][4 * j + 2], acc[i][4 * j + 3]};
            }
          }
        if (half == 0) {
          if (!whole) {
            pst[2 * (wrow + col)] = m;
            pst[2 * (wrow + col) + 1] = l;
          } else if (a.x.lse != nullptr) {
            a.x.lse[int64_t(head) * a.c.N + sh.q.a + tok] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
          }
        }
      }
    } else {
      // [wave][row][D + 4] and then [wave][row] m, l
      float* js = reinterpret_cast<float*>(lds);
      float* jst = js + 4 * 32 * (D + 4);
      if (col < mine) {
#pragma unroll
        for (int i = 0; i < DT; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<f32x4*>(js + (wave * 32 + col) * (D + 4) + 32 * i + 8 * j + 4 * half) =
                f32x4{acc[i][4 * j], acc[i][4 * j + 1], acc[i][4 * j + 2], acc[i][4 * j + 3]};
        if (half == 0) {
          jst[2 * (wave * 32 + col)] = m;
          jst[2 * (wave * 32 + col) + 1] = l;
        }
      }
      __syncthreads();
      for (int i = tid; i < mine * (D / 4); i += NT) {
        const int q = i / (D / 4), d = i % (D / 4) * 4;
        float top = jst[2 * q], sum = 0.f;
#pragma unroll
        for (int v = 1; v < 4; ++v) top = fmaxf(top, jst[2 * (v * 32 + q)]);
        f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float f = ex2(jst[2 * (v * 32 + q)] - top);
          sum += f * jst[2 * (v * 32 + q) + 1];
          const f32x4 z = *reinterpret_cast<const f32x4*>(js + (v * 32 + q) * (D + 4) + d);
          // (an infinity stays one, however small its wave's share)
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] += finite(z[e]) ? f * z[e] : z[e];
        }
        if (!whole) {
          *reinterpret_cast<f32x4*>(psum + q * D + d) = y;
          if (d == 0) {
            pst[2 * q] = top;
            pst[2 * q + 1] = sum;
          }
          continue;
        }
        const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
        const int32_t t = q / rep, hh = pl.hk * rep + q % rep;
        bf16x4 z;
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = static_cast<bf16>(y[e] * inv);
        *reinterpret_cast<bf16x4*>(o + ((int64_t(sh.q.a) + t) * a.x.Hq + hh) * D + d) = z;
        if (a.x.lse != nullptr && d == 0)
          a.x.lse[int64_t(hh) * a.c.N + sh.q.a + t] = sum == 0.f ? -INFINITY : top * kLn2 + logf(sum);
      }
      __syncthreads();  // the sums have left LDS
    }
    unit += pc.b1 - b0;
  }
}

// Joins the parts of cut tiles: work-group w the tile whose second part was in the main
// launch's work-group w. A thread sums 4 channels of a row over every n-th part, the
// loads of 8 parts going out together, and the n threads of a row's channels are joined
// at the end: many parts (one long request) and few rows, or few parts and many rows.
template <int D, bool kBig>
__device__ __forceinline__ void join_parts(const PagedArgs& c, const AttnPagedArgs& x, const float* __restrict__ sums,
                                           const Cut* __restrict__ cuts, int64_t w) {
  using F = Form<D, kBig>;
  constexpr int kQ = D / 4, kAtOnce = 8;
  __shared__ f32x4 ly[kThreads];
  __shared__ float lm[kThreads], ll[kThreads];
  const Cut t = cuts[w];
  if (t.last < 0) return;
  const int parts = t.last - int(w) + 2, n = parts > 2 * kAtOnce ? 8 : parts > kAtOnce ? 2 : 1;
  const int rep = x.Hq / c.Hkv, d = threadIdx.x % kQ * 4, i = threadIdx.x / kQ, mine = i % n;
  const int block = kThreads / kQ / n;  // rows at a time
  const float* st = sums + F::STATS;
  for (int q0 = blockIdx.y * block; q0 < t.rows; q0 += gridDim.y * block) {
    const int q = q0 + i / n < t.rows ? q0 + i / n : t.rows - 1;
    float m = -FLT_MAX, l = 0.f;
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
    for (int p0 = mine; p0 < parts; p0 += n * kAtOnce) {
      float pm[kAtOnce], pl[kAtOnce];
      f32x4 z[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int p = p0 + u * n < parts ? p0 + u * n : mine;
        const int64_t at = (2 * (w - 1 + p) + (p == 0 ? 1 : 0)) * F::BM + q;
        pm[u] = st[2 * at];
        pl[u] = st[2 * at + 1];
        z[u] = *reinterpret_cast<const f32x4*>(sums + at * D + d);
      }
      float top = m;
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) top = p0 + u * n < parts ? fmaxf(top, pm[u]) : top;
      const float f = ex2(m - top);
      m = top;
      l *= f;
      // (an infinity stays one, however small its part's share)
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = finite(y[e]) ? f * y[e] : y[e];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        if (p0 + u * n >= parts) break;
        const float g = ex2(pm[u] - top);
        l += g * pl[u];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] += finite(z[u][e]) ? g * z[u][e] : z[u][e];
      }
    }
    __syncthreads();  // the last rows are read
    ly[threadIdx.x] = y;
    lm[threadIdx.x] = m;
    ll[threadIdx.x] = l;
    __syncthreads();
    if (mine != 0 || q0 + i / n >= t.rows) continue;
    float top = m, sum = 0.f;
    for (int v = 1; v < n; ++v) top = fmaxf(top, lm[threadIdx.x + v * kQ]);
    y = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int v = 0; v < n; ++v) {
      const int at = threadIdx.x + v * kQ;
      const float g = ex2(lm[at] - top);
      sum += g * ll[at];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] += finite(ly[at][e]) ? g * ly[at][e] : ly[at][e];
    }
    const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
    const int row = t.rep_mod + q, tok = t.a + t.rep_first + row / rep, hh = t.hk * rep + row % rep;
    bf16x4 z;
#pragma unroll
    for (int e = 0; e < 4; ++e) z[e] = static_cast<bf16>(y[e] * inv);
    *reinterpret_cast<bf16x4*>(static_cast<bf16*>(x.o) + (int64_t(tok) * x.Hq + hh) * D + d) = z;
    if (x.lse != nullptr && d == 0) x.lse[int64_t(hh) * c.N + tok] = sum == 0.f ? -INFINITY : top * kLn2 + logf(sum);
  }
}

// The workspace: the small form's parts and cuts, and those of the big form where a call can
// have it.
template <int D>
struct Workspace {
  using S = Form<D, false>;
  using B = Form<D, true>;
  static constexpr size_t SMALL = S::PARTS + S::GROUPS * sizeof(Cut), BIG = B::PARTS + B::GROUPS * sizeof(Cut);
  static_assert(S::PARTS % 16 == 0 && SMALL % 16 == 0 && B::PARTS % 16 == 0, "16-byte stores");
  float *small, *big;
  Cut *small_cuts, *big_cuts;
  explicit Workspace(void* ws) {
    char* p = static_cast<char*>(ws);
    small = reinterpret_cast<float*>(p);
    small_cuts = reinterpret_cast<Cut*>(p + S::PARTS);
    big = reinterpret_cast<float*>(p + SMALL);
    big_cuts = reinterpret_cast<Cut*>(p + SMALL + B::PARTS);
  }
};

// Work-groups [0, small) join what the small form's work-groups 1 .. small cut.
template <int D>
__global__ __launch_bounds__(kThreads) void attn_paged_join_kernel(const PagedArgs c, const AttnPagedArgs x,
                                                                   const Workspace<D> ws, int small) {
  if (int(blockIdx.x) < small)
    join_parts<D, false>(c, x, ws.small, ws.small_cuts, int64_t(blockIdx.x) + 1);
  else
    join_parts<D, true>(c, x, ws.big, ws.big_cuts, int64_t(blockIdx.x) - small + 1);
}

// Which forms a call's requests can have: at most 32 rows of one, and more (all N tokens may
// be one request's, but without cu_seqlens each has its own).
bool any_small(int32_t rep) { return rep <= 32; }
bool any_big(int64_t N, int32_t rep, bool chunks) { return (chunks ? N : 1) * rep > 32; }

template <int D>
hipError_t run(const PagedArgs& c, const AttnPagedArgs& x, hipStream_t stream) {
  const bool s = any_small(x.Hq / c.Hkv), b = any_big(c.N, x.Hq / c.Hkv, c.cu != nullptr);
  const Workspace<D> ws(x.workspace);
  // (the first launch also zeroes the rows that no request has)
  const int64_t tail = c.cu == nullptr ? 1 : tail_groups(c.N * x.Hq * D * 2);
  // Two work-groups of the small form fit a compute unit: one hides the other's start and
  // end, which counts where walks are many and short, and costs a longer join and parts of
  // half the length. One token each, H 32, Hkv 8, D 128, 256 / 512 work-groups:
  //   1 request of 131072 tokens (8 walks)      108 / 112 us
  //   64 of about 2000 (512)                    146 / 149
  //   128 of 300, of 2000 (1024)                 47 / 36, 194 / 202
  //   256 of 300, of 1500 (2048)                 90 / 66, 290 / 294
  //   1024 of 130, of 600 (8192)                269 / 171, 518 / 481
  // D 64, the same, 512 the better nearly everywhere: 64 of 4096 117 / 110, 256 of 300 60 / 41.
  constexpr int64_t gb = Form<D, true>::GROUPS;
  const int64_t gs = D == 128 && int64_t(c.R) * c.Hkv < 1024 ? Form<D, false>::GROUPS / 2 : Form<D, false>::GROUPS;
  if (b)
    attn_paged_kernel<D, true><<<dim3(uint32_t(gb + tail)), dim3(Form<D, true>::NT), 0, stream>>>(
        Launch{c, x, ws.big, ws.big_cuts, gb});
  if (s)
    attn_paged_kernel<D, false><<<dim3(uint32_t(gs + (b ? 0 : tail))), dim3(Form<D, false>::NT), 0, stream>>>(
        Launch{c, x, ws.small, ws.small_cuts, gs});
  const int js = s ? int(gs) - 1 : 0, jb = b ? int(gb) - 1 : 0;
  // (the big form's tiles have 8 times the rows: 4 and 16 work-groups to a tile, 27 and 23 us
  // of 1007 us of a long prompt's chunk)
  attn_paged_join_kernel<D><<<dim3(js + jb, b ? 16 : 4), dim3(kThreads), 0, stream>>>(c, x, ws, js);
  return hipGetLastError();
}

}  // namespace

size_t attn_paged_workspace_bytes(int64_t N, int32_t Hq, int32_t Hkv, int32_t D, bool chunks) {
  const size_t big = any_big(N, Hq / Hkv, chunks) ? (D == 64 ? Workspace<64>::BIG : Workspace<128>::BIG) : 0;
  return (D == 64 ? Workspace<64>::SMALL : Workspace<128>::SMALL) + big;
}

hipError_t launch_attn_paged(const PagedArgs& c, const AttnPagedArgs& x, hipStream_t stream) {
  return c.D == 64 ? run<64>(c, x, stream) : run<128>(c, x, stream);
}

}  // namespace pkv
