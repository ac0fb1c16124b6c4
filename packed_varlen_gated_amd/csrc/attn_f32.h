// What the fp32 attention kernels share (attn_simple.hip, packed, and attn_paged_simple.hip,
// over the paged cache): a wave's tile in LDS and the layouts of the fp32 matrix product.
#pragma once

#include "common.h"

namespace pkv {
namespace {

constexpr int kT = 32;        // tokens per tile, both sides
constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr float kFinite = 3.4028234663852886e38f;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

template <int D>
struct alignas(16) Tile {  // of one wave
  float x[kT][D + 4];      // (rows 4 banks apart)
  __device__ __forceinline__ f32x4 at(int r, int d) const { return *reinterpret_cast<const f32x4*>(&x[r][d]); }
};

__device__ __forceinline__ f32x4 load4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ f32x4 load4(const bf16* p) {
  typedef bf16 b16x4 __attribute__((ext_vector_type(4)));
  const b16x4 x = *reinterpret_cast<const b16x4*>(p);
  return f32x4{to_f32(x[0]), to_f32(x[1]), to_f32(x[2]), to_f32(x[3])};
}
__device__ __forceinline__ void store4(float* p, f32x4 x) { *reinterpret_cast<f32x4*>(p) = x; }
__device__ __forceinline__ void store4(bf16* p, f32x4 x) {
  typedef bf16 b16x4 __attribute__((ext_vector_type(4)));
  *reinterpret_cast<b16x4*>(p) = b16x4{from_f32<bf16>(x[0]), from_f32<bf16>(x[1]), from_f32<bf16>(x[2]), from_f32<bf16>(x[3])};
}

// The wave's LDS accesses are in order; nothing is moved across.
__device__ __forceinline__ void wave_fence() { asm volatile("" ::: "memory"); }

__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32, 64); }
// Row of register i of a product's result; the lane's column is lane % 32.
__device__ __forceinline__ int row_of(int i, int half) { return 8 * (i / 4) + 4 * half + i % 4; }

}  // namespace
}  // namespace pkv
