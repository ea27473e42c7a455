// Gated activation y = silu(gate) up, silu(g) = g / (1 + exp(-g)), with an
// 8-bit output and 8-bit checkpoints of gate and up, and its backward pass
// from the checkpoints:
//   dgate = dy up sigma (1 + g (1 - sigma)),   dup = dy g sigma,
//   sigma = 1 / (1 + exp(-g)).
//
// 16 lanes take one row's block of 128 columns, 8 columns each, so a block's
// largest magnitude is found with four shuffles and nothing is read twice.

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

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) swiglu_kernel(SwigluArgs a) {
  const T* gate = static_cast<const T*>(a.gate);
  const T* up = static_cast<const T*>(a.up);
  const int lane = threadIdx.x & 15;
  const int64_t kb = (a.F + kFp8Block - 1) / kFp8Block;
  const int64_t groups = static_cast<int64_t>(gridDim.x) * (kThreads / 16);
  const int64_t total = a.M * kb;
  // both halves of a warp run the same number of steps (they shuffle together)
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads / 16) + (threadIdx.x >> 5) * 2;
  grid_launch_dependents();
  grid_dependency_wait();
  for (int64_t pair = first; pair < total; pair += groups) {
    const int64_t blk = pair + ((threadIdx.x >> 4) & 1);
    const int64_t row = blk / kb, k = blk - row * kb;
    const int64_t col = k * kFp8Block + 8 * lane;
    const int n = blk < total ? clamp8(a.F - col) : 0;
    float g[8], u[8], y[8];
    load8<T, VEC>(gate + row * a.ldg + col, n, g);
    load8<T, VEC>(up + row * a.ldu + col, n, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s, r;
      sigmoid(g[i], s, r);
      y[i] = g[i] * s * u[i];
    }
    const uint32_t b = fp8_scale_byte(group_umax<16>(amax8(y)));
    if (n > 0) {
      store_codes8(a.codes + row * a.ldc + col, n, codes8(y, fp8_inverse_scale(b)));
      if (lane == 0) a.scales[row * a.lds + k] = static_cast<uint8_t>(b);
    }
    if (a.g_codes) {
      const uint32_t bg = fp8_scale_byte(group_umax<16>(amax8(g)));
      const uint32_t bu = fp8_scale_byte(group_umax<16>(amax8(u)));
      if (n > 0) {
        store_codes8(a.g_codes + row * a.g_ld + col, n, codes8(g, fp8_inverse_scale(bg)));
        store_codes8(a.u_codes + row * a.u_ld + col, n, codes8(u, fp8_inverse_scale(bu)));
        if (lane == 0) {
          a.g_scales[row * a.g_lds + k] = static_cast<uint8_t>(bg);
          a.u_scales[row * a.u_lds + k] = static_cast<uint8_t>(bu);
        }
      }
    }
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) swiglu_backward_kernel(SwigluBackwardArgs a) {
  const T* dy = static_cast<const T*>(a.dy);
  T* dgate = static_cast<T*>(a.dgate);
  T* dup = static_cast<T*>(a.dup);
  const int lane = threadIdx.x & 15;
  const int64_t kb = (a.F + kFp8Block - 1) / kFp8Block;
  const int64_t groups = static_cast<int64_t>(gridDim.x) * (kThreads / 16);
  const int64_t total = a.M * kb;
  grid_launch_dependents();
  grid_dependency_wait();
  for (int64_t blk = static_cast<int64_t>(blockIdx.x) * (kThreads / 16) + (threadIdx.x >> 4); blk < total;
       blk += groups) {
    const int64_t row = blk / kb, k = blk - row * kb;
    const int64_t col = k * kFp8Block + 8 * lane;
    const int n = clamp8(a.F - col);
    if (n == 0) continue;
    float d[8], g[8], u[8], dg[8], du[8];
    load8<T, VEC>(dy + row * a.lddy + col, n, d);
    decode8(load_codes8(a.g_codes + row * a.g_ld + col, n), fp8_scale(a.g_scales[row * a.g_lds + k]), g);
    decode8(load_codes8(a.u_codes + row * a.u_ld + col, n), fp8_scale(a.u_scales[row * a.u_lds + k]), u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s, r;
      sigmoid(g[i], s, r);
      dg[i] = d[i] * u[i] * s * fmaf(g[i], r, 1.0f);
      du[i] = d[i] * g[i] * s;
    }
    store8<T, VEC>(dgate + row * a.lddg + col, n, dg);
    store8<T, VEC>(dup + row * a.lddu + col, n, du);
  }
}

int grid_for(int64_t M, int64_t F, int sms) {
  const int64_t blocks = M * ((F + kFp8Block - 1) / kFp8Block);
  const int64_t want = (blocks + kThreads / 16 - 1) / (kThreads / 16);
  const int64_t most = 8 * static_cast<int64_t>(sms);
  return static_cast<int>(want < most ? want : most);
}

}  // namespace

cudaError_t launch_swiglu(const SwigluArgs& a, int dtype, bool vec, int sms, cudaStream_t st) {
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    return launch_dependent(vec ? swiglu_kernel<T, true> : swiglu_kernel<T, false>,
                            dim3(grid_for(a.M, a.F, sms)), kThreads, 0, st, a);
  });
}

cudaError_t launch_swiglu_backward(const SwigluBackwardArgs& a, int dtype, bool vec, int sms, cudaStream_t st) {
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    return launch_dependent(vec ? swiglu_backward_kernel<T, true> : swiglu_backward_kernel<T, false>,
                            dim3(grid_for(a.M, a.F, sms)), kThreads, 0, st, a);
  });
}

}  // namespace taco
