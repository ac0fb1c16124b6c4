// New tokens' keys and values into the paged cache.
//
// A work-group takes 16 tokens of one request (a tile aligned to the request's first
// new token, found as in segments.h), a wave one token at a time: the token's row of
// all kv heads, 16 bytes a lane. With one token per request a work-group takes 4.
// A copy: bound by memory, in small calls by the chain request, page, row. 6236 tokens of
// four prompts, Hkv 8, D 128: 11.7 us for 51 MB; 64 requests' single tokens: 3 us, in a call
// of 9 us from Python.

#include "paged.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kTile = 16;

typedef int i32x4 __attribute__((ext_vector_type(4)));

// units: 16-byte pieces of a token's row; strides in pieces.
__global__ __launch_bounds__(kThreads) void paged_append_kernel(const PagedArgs c, const i32x4* __restrict__ k,
                                                                const i32x4* __restrict__ v, int64_t ks, int64_t vs,
                                                                i32x4* __restrict__ kp, i32x4* __restrict__ vp,
                                                                int32_t units, int64_t groups) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (int64_t(blockIdx.x) == groups) {
    check_requests(c);
    return;
  }
  int32_t r, from, to;  // the work-group's tokens
  if (c.cu == nullptr) {
    r = blockIdx.x * kWaves + wave;
    if (r >= c.R) return;
    from = r;
    to = r + 1;
  } else {
    SegTile t;
    if (!find_tile(c.cu, c.R, c.N, kTile, blockIdx.x, t)) return;
    r = t.seg;
    from = t.start + wave;
    to = t.e < t.start + kTile ? t.e : t.start + kTile;
  }
  const Request q = request(c, r);
  for (int32_t n = from; n < to; n += kWaves) {
    const int32_t p = q.len - q.n + (n - q.a);
    if (!q.ok || p < 0) continue;
    const int32_t page = page_of(c, r, p);
    if (page < 0) continue;
    const i32x4 *sk = k + n * ks, *sv = v + n * vs;
    const int64_t at = page_row(c, page, p) * units;
    for (int32_t i = lane; i < units; i += 64) {
      const i32x4 x = sk[i], y = sv[i];
      kp[at + i] = x;
      vp[at + i] = y;
    }
  }
}

}  // namespace

hipError_t launch_paged_append(const PagedArgs& c, const AppendArgs& x, int32_t dtype, hipStream_t stream) {
  const int64_t es = dtype == 0 ? 2 : 4, groups = c.cu == nullptr ? (c.R + kWaves - 1) / kWaves : tile_slots(c.N, c.R, kTile);
  paged_append_kernel<<<dim3(uint32_t(groups + 1)), dim3(kThreads), 0, stream>>>(
      c, static_cast<const i32x4*>(x.k), static_cast<const i32x4*>(x.v), x.k_stride * es / 16, x.v_stride * es / 16,
      static_cast<i32x4*>(x.k_pages), static_cast<i32x4*>(x.v_pages), int32_t(c.Hkv * c.D * es / 16), groups);
  return hipGetLastError();
}

}  // namespace pkv
