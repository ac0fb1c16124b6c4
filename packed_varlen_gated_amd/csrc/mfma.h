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
