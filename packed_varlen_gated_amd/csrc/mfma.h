// Device helpers of the mixers' matrix-core kernels (gfx950).
//
// v_mfma_f32_32x32x16_bf16: A operand lane l holds row l % 32 and contraction
// slots 8 (l / 32) .. + 7, B likewise for column l % 32; the 32x32 fp32 result
// has column l % 32 and, in register i, row 8 (i / 4) + 4 (l / 32) + i % 4.
// v_mfma_f32_16x16x32_bf16: row / column l % 16, slots 8 (l / 16) .. + 7; the
// 16x16 result has column l % 16 and rows 4 (l / 16) + i. The contraction index
// may be permuted freely when A and B agree.
#pragma once

#include "common.h"

namespace pkv {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, int(bytes), 0x00020000);
}
// Out-of-range reads give 0, out-of-range stores are dropped.
__device__ __forceinline__ bf16x8 load8(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(bf16x8, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
__device__ __forceinline__ void store16(__amdgpu_buffer_rsrc_t r, uint32_t off, i32x4 x) {
  __builtin_amdgcn_raw_buffer_store_b128(x, r, off, 0, 0);
}

// 16 bytes per lane from a buffer straight into LDS, at `lds` (the same in
// every lane) + 16 lane; out-of-range reads write 0.
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, uint32_t off, void* lds) {
  // (a scalar offset would not take part in the range check)
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, off, 0, 0, 0);
}
// The same, with the waits left to the caller. Behind the builtin the compiler waits for
// all loads before the next read of LDS that it cannot tell apart, that is, for those of
// the next tile before this one is used. `lds` is a byte address (lds_addr). The loads
// count for wait_vm and wait_loads; no register is written. The descriptor is that of
// buffer(), the same in every lane.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ u32x4 descriptor(const void* base, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uintptr_t>(base);
  return u32x4{uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(b))),
               uint32_t(__builtin_amdgcn_readfirstlane(uint32_t(b >> 32) & 0xffffu)),
               uint32_t(__builtin_amdgcn_readfirstlane(bytes)), 0x00020000u};
}
// Load u of N goes to lds + u kStep, from off[u]. What the hardware does not check has its
// wait states here, where no schedule can take them away: a load reads a scalar register
// that a vector instruction wrote (readfirstlane in descriptor(), or readlane where the
// compiler had spilled it) five states after the write at the earliest, which the compiler
// keeps for its own loads but not for those in a text: two moves and s_nop 2. And a load
// into LDS reads m0 one state after its change. (m0 is the compiler's own and put back.)
template <int N, int kStep>
__device__ __forceinline__ void load_lds16_async(u32x4 r, const uint32_t (&off)[N], uint32_t lds) {
  static_assert(N == 2 || N == 4, "the loads of a tile or of a granule");
  uint32_t m0;
#define PKV_FIRST(x) "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 2\n\tbuffer_load_dwordx4 " x ", %2, 0 offen lds\n\t"
#define PKV_NEXT(x) "s_add_u32 m0, m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 " x ", %2, 0 offen lds\n\t"
  if constexpr (N == 2)
    asm volatile(PKV_FIRST("%4") PKV_NEXT("%5") "s_mov_b32 m0, %0"
                 : "=&s"(m0)
                 : "s"(lds), "s"(r), "i"(kStep), "v"(off[0]), "v"(off[1])
                 : "memory", "scc");
  else
    asm volatile(PKV_FIRST("%4") PKV_NEXT("%5") PKV_NEXT("%6") PKV_NEXT("%7") "s_mov_b32 m0, %0"
                 : "=&s"(m0)
                 : "s"(lds), "s"(r), "i"(kStep), "v"(off[0]), "v"(off[1]), "v"(off[2]), "v"(off[3])
                 : "memory", "scc");
#undef PKV_FIRST
#undef PKV_NEXT
}
// 4 bytes per lane, with the same wait states.
__device__ __forceinline__ void load_lds4_async(u32x4 r, uint32_t off, uint32_t lds) {
  uint32_t m0;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 2\n\tbuffer_load_dword %2, %3, 0 offen lds\n\ts_mov_b32 m0, %0"
               : "=&s"(m0)
               : "s"(lds), "v"(off), "s"(r)
               : "memory");
}
// x, recomputed from here on: what is derived from it in a loop is not kept in
// registers across the loop.
__device__ __forceinline__ uint32_t fresh(uint32_t x) {
  asm volatile("" : "+v"(x));
  return x;
}

__device__ __forceinline__ uint32_t fresh_uniform(uint32_t x) {
  x = __builtin_amdgcn_readfirstlane(x);
  asm volatile("" : "+s"(x));
  return x;
}

// LDS by byte address.
typedef __attribute__((address_space(3))) char lds_char;
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return uint32_t(reinterpret_cast<uintptr_t>((const lds_char*)(p)));
}
__device__ __forceinline__ bf16x8 read_lds8(uint32_t a) {
  typedef const __attribute__((address_space(3))) bf16x8 lds_bf16x8;
  return *(lds_bf16x8*)(uintptr_t(a));
}
// Transposing LDS read: within each group of 16 lanes, lane k points at 4
// consecutive bf16; with lane k at row r0 + k / 4, column c0 + 4 (k % 4) of a
// tile, lane j gets column c0 + j of rows r0 .. r0 + 3.
__device__ __forceinline__ s16x4 read_tr(uint32_t a) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(uintptr_t(a)));
}
__device__ __forceinline__ s16x4 read_tr(const void* p) { return read_tr(lds_addr(p)); }
__device__ __forceinline__ bf16x8 join(s16x4 lo, s16x4 hi) {
  return __builtin_bit_cast(bf16x8, s16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
}

// The value of lane l ^ 32.
__device__ __forceinline__ float other_half(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }

// All of this wave's vector-memory operations (loads into LDS among them) done.
__device__ __forceinline__ void wait_vm() { __builtin_amdgcn_s_waitcnt(0x0F70); }
// ... and its LDS operations.
__device__ __forceinline__ void wait_all() { __builtin_amdgcn_s_waitcnt(0x0070); }
// All LDS operations done, and all vector-memory operations but the last n (they
// complete in order).
template <int n>
__device__ __forceinline__ void wait_loads() {
  static_assert(n >= 0 && n < 64, "a 6-bit counter");
  __builtin_amdgcn_s_waitcnt(0x0070 | (n & 15) | (n >> 4) << 14);
}
// A work-group barrier that waits for nothing but the other waves.
__device__ __forceinline__ void bar() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace pkv
