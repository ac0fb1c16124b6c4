// Linear attention with one decay per head, token by token in fp32 (fp32
// tensors, and bf16 tensors with a head dimension of 32).
//
//   S_t = e^{g_h} S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t
// with S reset (or set to the slot's initial state) at every segment start: the
// recurrence of RFC-0026 Background with one decay in place of a gate per
// channel and no beta.
//
// One kernel runs the recurrence in either direction of time, and the reverse
// pass is three runs of it with the tensors in other roles:
//   dq_t = scale S_t do_t                      (a, b, c) = (do, v, k), forward, on S^T;
//   dv_t = dS_t^T k_t                          (k, q, do), backward, on dS;
//   dk_t = dS_t v_t                            (v, do, q), backward, on dS^T,
// where dS_t = e^{g} dS_{t+1} + scale q_t do_t^T and dS after the last token is
// the final state's cotangent. out_t = out_scale X_t^T a_t, X <- X + in_scale b_t c_t^T;
// forward the decay comes before a token's update, backward after its readout,
// so the state that leaves the walk backwards is the initial state's cotangent.
//
// A work-group of 256 threads takes 16 columns of X of one (slot, head): thread
// (rg, e) keeps column e, rows [rg R, rg R + R) in registers. Tokens go through LDS
// in blocks, the next block's loads under way while one is used, and each block's
// partial readouts are summed over the 16 row groups. The three walks of the reverse
// pass are one launch where Dk = Dv. The chain of tokens bounds it, 80 to 180 ns each;
// these are the shapes that models are debugged on. One segment of 4096 tokens, fp32,
// forward / reverse: H 4, D 64 437 / 456 us, H 16, D 128 724 / 1108 us; bf16, H 16, D 32
// 330 / 344 us; 512 tokens, H 4, D 32, fp32 41 / 41 us. With all columns in one work-group and three launches
// 1482 / 4521, 5045 / 15007 and 73 / 221 us.

#include "segments.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kCols = 16;  // columns of a work-group
constexpr int kGroups = kThreads / kCols;
constexpr int kTail = 64;

typedef float f32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 load4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ f32x4 load4(const bf16* p) {
  typedef bf16 b16x4 __attribute__((ext_vector_type(4)));
  const b16x4 x = *reinterpret_cast<const b16x4*>(p);
  return f32x4{to_f32(x[0]), to_f32(x[1]), to_f32(x[2]), to_f32(x[3])};
}

struct Walk {
  const void *a, *b, *c;
  const float* init;
  void* out;
  float* fin;
  float in_scale, out_scale;
  bool reverse, transposed;
};
struct Walks {
  Walk w[3];
};

// blockIdx: (slot, head), slice of columns, walk.
template <typename T, int DA, int DB>
__global__ __launch_bounds__(kThreads) void linear_serial_kernel(const Walks walks, const float* __restrict__ g,
                                                                 const int32_t* __restrict__ cu, int32_t max_segs,
                                                                 int64_t N, int32_t H, int32_t* __restrict__ flags) {
  const Walk& w = walks.w[blockIdx.z];
  const T *__restrict__ a = static_cast<const T*>(w.a), *__restrict__ b = static_cast<const T*>(w.b),
          *__restrict__ c = static_cast<const T*>(w.c);
  const float* __restrict__ init = w.init;
  T* __restrict__ out = static_cast<T*>(w.out);
  float* __restrict__ fin = w.fin;
  const float in_scale = w.in_scale, out_scale = w.out_scale;
  const bool reverse = w.reverse, transposed = w.transposed;
  constexpr int R = DA / kGroups, TB = DA == 128 ? 16 : 32;  // rows of a thread, tokens of a block
  constexpr int LA = TB * DA / 4 / kThreads, LC = TB * kCols / 4;  // 16-byte loads: per thread, of a block's c
  static_assert(LA * kThreads * 4 == TB * DA && LC <= kThreads, "bad tile");
  __shared__ __attribute__((aligned(16))) float sa[2][TB][DA], sb[2][TB][DA], sc[2][TB][kCols];
  __shared__ float part[TB][kGroups][kCols];
  const int tid = threadIdx.x;
  const int64_t items = int64_t(max_segs) * H;
  if (int64_t(blockIdx.x) >= items) {
    if (blockIdx.y != 0) return;
    const int64_t j = blockIdx.x - items;
    zero_tail(out, covered_tokens(cu, max_segs, N), N, int64_t(H) * DB * sizeof(T), j, kTail);
    if (j == 0) check_cu(cu, max_segs, N, flags);
    return;
  }
  const int32_t slot = int32_t(blockIdx.x / H), h = int32_t(blockIdx.x % H);
  const int64_t start = cu ? cu[slot] : 0, end = cu ? cu[slot + 1] : N;
  if (!segment_ok(slot, start, end, N)) return;

  const int col = tid % kCols, rg = tid / kCols, e0 = int(blockIdx.y) * kCols, e = e0 + col;
  const float decay = expf(g[h]);
  const int64_t state0 = (int64_t(slot) * H + h) * DA * DB;
  float X[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int d = rg * R + r;
    X[r] = init == nullptr ? 0.f : init[state0 + (transposed ? e * DA + d : d * DB + e)];
  }
  const int64_t n = end - start;
  auto token = [&](int64_t i) { return reverse ? end - 1 - i : start + i; };
  f32x4 na[LA] = {}, nb[LA] = {}, nc = {};  // of the next block
  auto load = [&](int64_t t0) {
#pragma unroll
    for (int u = 0; u < LA; ++u) {
      const int i = (u * kThreads + tid) * 4;
      if (t0 + i / DA >= n) continue;
      const int64_t off = (token(t0 + i / DA) * H + h) * DA + i % DA;
      na[u] = load4(a + off);
      nb[u] = load4(b + off);
    }
    const int i = tid * 4;
    if (tid < LC && t0 + i / kCols < n) nc = load4(c + (token(t0 + i / kCols) * H + h) * DB + e0 + i % kCols);
  };
  auto put = [&](int s) {
#pragma unroll
    for (int u = 0; u < LA; ++u) {
      const int i = (u * kThreads + tid) * 4;
      *reinterpret_cast<f32x4*>(&sa[s][i / DA][i % DA]) = na[u] * out_scale;
      *reinterpret_cast<f32x4*>(&sb[s][i / DA][i % DA]) = nb[u] * in_scale;
    }
    if (tid < LC) *reinterpret_cast<f32x4*>(&sc[s][tid * 4 / kCols][tid * 4 % kCols]) = nc;
  };
  load(0);
  put(0);
  int s = 0;
  for (int64_t t0 = 0; t0 < n; t0 += TB, s ^= 1) {
    const int nt = n - t0 < TB ? int(n - t0) : TB;
    __syncthreads();  // the block is in LDS, the last one's readouts are out of it
    load(t0 + TB);
#pragma unroll 4
    for (int tt = 0; tt < nt; ++tt) {
      const float y = sc[s][tt][col];
      float p = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float z = sb[s][tt][rg * R + r] * y;
        X[r] = reverse ? X[r] + z : fmaf(X[r], decay, z);
        p += X[r] * sa[s][tt][rg * R + r];
        if (reverse) X[r] *= decay;
      }
      part[tt][rg][col] = p;
    }
    __syncthreads();
    for (int i = tid; i < nt * kCols; i += kThreads) {
      float p = 0.f;
#pragma unroll
      for (int j = 0; j < kGroups; ++j) p += part[i / kCols][j][i % kCols];
      out[(token(t0 + i / kCols) * H + h) * DB + e0 + i % kCols] = from_f32<T>(p);
    }
    put(s ^ 1);
  }
  if (fin != nullptr) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int d = rg * R + r;
      fin[state0 + (transposed ? e * DA + d : d * DB + e)] = X[r];
    }
  }
}

template <typename T, int DA, int DB>
void run(const LinearArgs& x, const Walks& walks, int count, hipStream_t stream) {
  const int64_t grid = int64_t(x.max_segs) * x.H + kTail;
  linear_serial_kernel<T, DA, DB><<<dim3(uint32_t(grid), DB / kCols, count), dim3(kThreads), 0, stream>>>(
      walks, x.g, x.cu, x.max_segs, x.N, x.H, x.flags);
}

template <typename T, int DK, int DV>
hipError_t fwd(const LinearArgs& x, hipStream_t s) {
  run<T, DK, DV>(x, {{{x.q, x.k, x.v, x.initial_state, x.o, x.final_state, 1.f, x.scale, false, false}}}, 1, s);
  return hipGetLastError();
}

template <typename T, int DK, int DV>
hipError_t bwd(const LinearArgs& x, const LinearGradArgs& y, hipStream_t s) {
  const Walk dq = {y.dout, x.v, x.k, x.initial_state, y.dq, nullptr, 1.f, x.scale, false, true};
  const Walk dk = {x.v, y.dout, x.q, y.dfinal_state, y.dk, nullptr, x.scale, 1.f, true, true};
  const Walk dv = {x.k, x.q, y.dout, y.dfinal_state, y.dv, y.d_initial_state, x.scale, 1.f, true, false};
  if constexpr (DK == DV) {
    run<T, DK, DV>(x, {{dq, dk, dv}}, 3, s);
  } else {
    run<T, DV, DK>(x, {{dq, dk}}, 2, s);
    run<T, DK, DV>(x, {{dv}}, 1, s);
  }
  return hipGetLastError();
}

// The pairs with a dimension of 32, for either type, and the others, for fp32 alone
// (with bf16 they are linear_chunk.hip's).
#define PKV_LINEAR_32(fn, T, ...)                                     \
  if (x.Dk == 32 && x.Dv == 32) return fn<T, 32, 32>(__VA_ARGS__);    \
  if (x.Dk == 32 && x.Dv == 64) return fn<T, 32, 64>(__VA_ARGS__);    \
  if (x.Dk == 32 && x.Dv == 128) return fn<T, 32, 128>(__VA_ARGS__);  \
  if (x.Dk == 64 && x.Dv == 32) return fn<T, 64, 32>(__VA_ARGS__);    \
  if (x.Dk == 128 && x.Dv == 32) return fn<T, 128, 32>(__VA_ARGS__)
#define PKV_LINEAR_64(fn, T, ...)                                     \
  if (x.Dk == 64 && x.Dv == 64) return fn<T, 64, 64>(__VA_ARGS__);    \
  if (x.Dk == 64 && x.Dv == 128) return fn<T, 64, 128>(__VA_ARGS__);  \
  if (x.Dk == 128 && x.Dv == 64) return fn<T, 128, 64>(__VA_ARGS__);  \
  if (x.Dk == 128 && x.Dv == 128) return fn<T, 128, 128>(__VA_ARGS__)

}  // namespace

hipError_t launch_linear_serial(const LinearArgs& x, int32_t dtype, hipStream_t stream) {
  if (dtype == 0) {
    PKV_LINEAR_32(fwd, bf16, x, stream);
  } else {
    PKV_LINEAR_32(fwd, float, x, stream);
    PKV_LINEAR_64(fwd, float, x, stream);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_linear_serial_backward(const LinearArgs& x, const LinearGradArgs& y, int32_t dtype,
                                         hipStream_t stream) {
  if (dtype == 0) {
    PKV_LINEAR_32(bwd, bf16, x, y, stream);
  } else {
    PKV_LINEAR_32(bwd, float, x, y, stream);
    PKV_LINEAR_64(bwd, float, x, y, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace pkv
