// Gated activation y = silu(gate) up, silu(g) = g / (1 + exp(-g)), with an
// 8-bit output and 8-bit checkpoints of gate and up, and its backward pass
// from the checkpoints:
//   dgate = dy up sigma (1 + g (1 - sigma)),   dup = dy g sigma,
//   sigma = 1 / (1 + exp(-g)).
//
// A warp takes 512 columns of one row: 8 lanes a block of 128, 16 columns each,
// so a block's largest magnitude is found with three shuffles and nothing is
// read twice.
//
// Measured, bf16, 16384 x 4096: forward with checkpoints 81 us, 5.8 TB/s, 71% of
// the issue slots (exp, reciprocal and three conversions to 8 bits an element);
// backward 84.5 us, 6.4 TB/s, bound by memory (a plain copy: 6.7 TB/s).

#include "fp8_block.cuh"

namespace taco {

namespace {

constexpr int kThreads = 256;

// s = 1 / (1 + exp(-g)) and 1 - s, each to its own relative precision: with
// e = exp(-|g|) <= 1 they are 1 / (1 + e) and e / (1 + e) in one order or the
// other, and the divisor lies in [1, 2].
__device__ __forceinline__ void sigmoid(float g, float& s, float& one_minus_s) {
  const float e = __expf(-fabsf(g));
  const float r = __fdividef(1.0f, 1.0f + e);
  s = g >= 0.0f ? r : e * r;
  one_minus_s = g >= 0.0f ? e * r : r;
}

// CTAs per SM that the registers are held to (16-bit types, 16384 x 4096 with
// checkpoints): forward 4 (3: 90 us, 4: 81, 5 spills), backward 6 (4: 95 us,
// 5: 87, 6: 85).
template <typename T>
constexpr int forward_ctas() { return sizeof(T) == 2 ? 4 : 3; }
template <typename T>
constexpr int backward_ctas() { return sizeof(T) == 2 ? 6 : 4; }

template <typename T, bool VEC, bool CKPT>
__global__ void __launch_bounds__(kThreads, forward_ctas<T>()) swiglu_kernel(SwigluArgs a, Divider per_row, bool wide) {
  const int lane8 = threadIdx.x & 7;
  const uint64_t w = static_cast<uint64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t row = per_row.quotient(w);
  const int64_t k = static_cast<int64_t>(w - row * per_row.d) * 4 + ((threadIdx.x >> 3) & 3);
  const int64_t col = k * kFp8Block + 16 * lane8;
  grid_launch_dependents();
  grid_dependency_wait();
  if (row >= a.M) return;   // whole warps
  const int n = clamp16(a.F - col);
  const Row16<T> gr = load16<T, VEC>(static_cast<const T*>(a.gate) + row * a.ldg + col, n, wide);
  const Row16<T> ur = load16<T, VEC>(static_cast<const T*>(a.up) + row * a.ldu + col, n, wide);
  float g[16], u[16], y[16];
  unpack<T>(gr, g);
  unpack<T>(ur, u);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float s, r;
    sigmoid(g[i], s, r);
    y[i] = g[i] * s * u[i];
  }
  quantize16(y, n, a.codes + row * a.ldc + col, a.scales + row * a.lds + k, lane8);
  if (CKPT) {
    quantize16(g, n, a.g_codes + row * a.g_ld + col, a.g_scales + row * a.g_lds + k, lane8);
    quantize16(u, n, a.u_codes + row * a.u_ld + col, a.u_scales + row * a.u_lds + k, lane8);
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, backward_ctas<T>())
swiglu_backward_kernel(SwigluBackwardArgs a, Divider per_row, bool wide) {
  const int lane8 = threadIdx.x & 7;
  const uint64_t w = static_cast<uint64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t row = per_row.quotient(w);
  const int64_t k = static_cast<int64_t>(w - row * per_row.d) * 4 + ((threadIdx.x >> 3) & 3);
  const int64_t col = k * kFp8Block + 16 * lane8;
  grid_launch_dependents();
  grid_dependency_wait();
  const int n = clamp16(a.F - col);
  if (row >= a.M || (VEC && n == 0)) return;   // unaligned rows are stored by whole warps
  const Row16<T> dr = load16<T, VEC>(static_cast<const T*>(a.dy) + row * a.lddy + col, n, wide);
  const uint4 gc = load_codes16(a.g_codes + row * a.g_ld + col, n);
  const uint4 uc = load_codes16(a.u_codes + row * a.u_ld + col, n);
  const bool any = VEC || n > 0;
  const float gs = any ? fp8_scale(a.g_scales[row * a.g_lds + k]) : 1.0f;
  const float us = any ? fp8_scale(a.u_scales[row * a.u_lds + k]) : 1.0f;
  float d[16], g[16], u[16];
  unpack<T>(dr, d);
  decode16(gc, gs, g);
  decode16(uc, us, u);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float s, r;
    sigmoid(g[i], s, r);
    const float ds = d[i] * s;
    u[i] = ds * u[i] * fmaf(g[i], r, 1.0f);
    g[i] = ds * g[i];
  }
  store16<T, VEC>(static_cast<T*>(a.dgate) + row * a.lddg + col, n, wide, pack<T>(u));
  store16<T, VEC>(static_cast<T*>(a.dup) + row * a.lddu + col, n, wide, pack<T>(g));
}

struct Shape {
  Divider per_row;
  dim3 grid;
  Shape(int64_t M, int64_t F) : per_row((F + 4 * kFp8Block - 1) / (4 * kFp8Block)) {
    grid = dim3(static_cast<unsigned>((M * static_cast<int64_t>(per_row.d) + kThreads / 32 - 1) / (kThreads / 32)));
  }
};

}  // namespace

cudaError_t launch_swiglu(const SwigluArgs& a, int dtype, int vec, cudaStream_t st) {
  const Shape s(a.M, a.F);
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    auto k = vec ? (a.g_codes ? swiglu_kernel<T, true, true> : swiglu_kernel<T, true, false>)
                 : (a.g_codes ? swiglu_kernel<T, false, true> : swiglu_kernel<T, false, false>);
    return launch_dependent(k, s.grid, kThreads, 0, st, a, s.per_row, vec == kVec32);
  });
}

cudaError_t launch_swiglu_backward(const SwigluBackwardArgs& a, int dtype, int vec, cudaStream_t st) {
  const Shape s(a.M, a.F);
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    return launch_dependent(vec ? swiglu_backward_kernel<T, true> : swiglu_backward_kernel<T, false>, s.grid,
                            kThreads, 0, st, a, s.per_row, vec == kVec32);
  });
}

}  // namespace taco
