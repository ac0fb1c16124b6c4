// Argument checks shared by the entry points of include/pkv_mixers.h and
// include/pkv_softmax.h. Every check runs before any HIP call, so invalid arguments are
// reported synchronously and nothing is enqueued.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <initializer_list>

#include "pkv.h"

namespace pkv {

constexpr int64_t kInt32Max = 2147483647;
// Work-groups of a launch: a grid holds less than 2^32 work-items, of at most 512
// a group.
constexpr int64_t kMaxGroups = int64_t(1) << 23;
constexpr int32_t kMaxHeads = 65536;

inline bool supported_head_dim(int32_t d) { return d == 32 || d == 64 || d == 128; }
inline bool known_dtype(int32_t dt) { return dt == PKV_BF16 || dt == PKV_F32; }
inline int64_t elem_size(int32_t dt) { return dt == PKV_BF16 ? 2 : 4; }
inline pkv_status from_hip(hipError_t e) { return e == hipSuccess ? PKV_OK : PKV_ERR_HIP; }
inline bool heads_ok(int32_t Hq, int32_t Hkv) { return Hq >= 1 && Hkv >= 1 && Hq <= kMaxHeads && Hkv <= kMaxHeads; }

struct Span {
  const void* p;
  int64_t bytes;
  int64_t align;
};

inline bool overlap(const Span& a, const Span& b) {
  if (a.p == nullptr || b.p == nullptr) return false;
  const char *x = static_cast<const char*>(a.p), *y = static_cast<const char*>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}

// Alignment of every span, and no output on an input or another output.
inline bool spans_ok(std::initializer_list<Span> ins, std::initializer_list<Span> outs) {
  for (const Span& s : ins)
    if (reinterpret_cast<uintptr_t>(s.p) % s.align != 0) return false;
  for (const Span* o = outs.begin(); o != outs.end(); ++o) {
    if (reinterpret_cast<uintptr_t>(o->p) % o->align != 0) return false;
    for (const Span& s : ins)
      if (overlap(*o, s)) return false;
    for (const Span* p = outs.begin(); p != o; ++p)
      if (overlap(*o, *p)) return false;
  }
  return true;
}

inline bool any_null(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (p == nullptr) return true;
  return false;
}

inline bool workspace_ok(const void* ws, size_t bytes, size_t need) {
  return need == 0 || (ws != nullptr && bytes >= need && reinterpret_cast<uintptr_t>(ws) % 256 == 0);
}

// The bytes of N tokens of `heads` heads, `stride` elements apart.
inline int64_t strided_bytes(int64_t N, int64_t stride, int64_t heads, int64_t D, int64_t es) {
  return ((N - 1) * stride + heads * D) * es;
}
// N tokens of `heads` dense heads, 16-byte aligned and not on each other, whose bytes (at
// most 2^46, more than an address space has) do not overflow.
inline bool stride_ok(int64_t N, int64_t stride, int64_t heads, int64_t D, int64_t es) {
  return stride >= heads * D && stride <= (int64_t(1) << 46) / es / N && stride * es % 16 == 0;
}

}  // namespace pkv
