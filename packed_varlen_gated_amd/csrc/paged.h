// The paged cache: where a request's tokens lie (shared by the kernels that fill it
// and those that read it).
#pragma once

#include "segments.h"

namespace pkv {

// Request r of a call: its new tokens are rows [a, a + n) of the packed ones and lie
// at places [len - n, len). ok: its numbers are within the call's tensors.
struct Request {
  int32_t a, n, len;
  bool ok;
};
__device__ __forceinline__ Request request(const PagedArgs& c, int32_t r) {
  Request q;
  q.a = c.cu == nullptr ? r : c.cu[r];
  const int64_t e = c.cu == nullptr ? int64_t(r) + 1 : c.cu[r + 1];
  q.len = c.lens[r];
  q.ok = segment_ok(r, q.a, e, c.N) && q.len >= 0 && q.len <= int64_t(c.max_pages) * c.page_size;
  q.n = q.ok ? int32_t(e - q.a) : 0;
  return q;
}

// One work-group's check of the whole call's numbers.
__device__ __forceinline__ void check_requests(const PagedArgs& c) {
  if (c.flags == nullptr) return;
  check_cu(c.cu, c.R, c.N, c.flags);
  bool bad = false;
  for (int32_t r = threadIdx.x; r < c.R; r += blockDim.x)
    bad |= c.lens[r] < 0 || c.lens[r] > int64_t(c.max_pages) * c.page_size;
  if (bad) atomicOr(c.flags, kFlagBadLength);
}

// The page of place p of request r, or -1 (and the flag) where the table holds none.
__device__ __forceinline__ int32_t page_of(const PagedArgs& c, int32_t r, int32_t p) {
  const int32_t page = c.table[int64_t(r) * c.max_pages + p / c.page_size];
  if (page >= 0 && page < c.num_pages) return page;
  if (c.flags != nullptr) atomicOr(c.flags, kFlagBadPage);
  return -1;
}
// The row (of Hkv heads) of place p in a page.
__device__ __forceinline__ int64_t page_row(const PagedArgs& c, int32_t page, int32_t p) {
  return int64_t(page) * c.page_size + p % c.page_size;
}

}  // namespace pkv
