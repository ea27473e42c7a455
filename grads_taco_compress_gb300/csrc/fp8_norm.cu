// Root-mean-square norm with the residual's addition, 8-bit output and 8-bit
// checkpoint, and its backward pass from the checkpoint.
//
//   forward   h = T(x + residual)          rounded once to the tensors' type:
//                                          the residual stream that the next
//                                          layer reads is the h normalised here
//             rstd = (mean h^2 + eps)^(-1/2)
//             y = h rstd w                 fp32, quantised directly
//   backward  xh = dec(checkpoint) rstd    (or h rstd from h itself)
//             g = dy w,  c = mean(g xh)
//             dx = rstd (g - xh c) + dh,   dw = sum over rows of dy xh
//
// A CTA takes a row at a time; thread t holds the 16-column chunks t, t + T,
// ... in registers, so a row is read once and a block of 128 columns is 8
// consecutive lanes. Sums are fp32.

#include "fp8_block.cuh"

namespace taco {

namespace {

template <typename T, int NC, bool VEC>
__global__ void __launch_bounds__(512) norm_kernel(NormArgs a, bool wide) {
  __shared__ float red[16];
  const int warps = blockDim.x >> 5, lane8 = threadIdx.x & 7;
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t row = blockIdx.x;
  Row16<T> h[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t col = 16 * (static_cast<int64_t>(threadIdx.x) + c * blockDim.x);
    h[c] = load16<T, VEC>(static_cast<const T*>(a.x) + row * a.ldx + col, clamp16(a.H - col), wide);
  }
  if (a.residual) {
    Row16<T> r[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = 16 * (static_cast<int64_t>(threadIdx.x) + c * blockDim.x);
      r[c] = load16<T, VEC>(static_cast<const T*>(a.residual) + row * a.ldr + col, clamp16(a.H - col), wide);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = 16 * (static_cast<int64_t>(threadIdx.x) + c * blockDim.x);
      float x[16], y[16];
      unpack<T>(h[c], x);
      unpack<T>(r[c], y);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] += y[i];
      h[c] = pack<T>(x);
      store16<T, VEC>(static_cast<T*>(a.h) + row * a.ldh + col, clamp16(a.H - col), wide, h[c]);
    }
  }
  float sum = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float v[16];
    unpack<T>(h[c], v);
#pragma unroll
    for (int i = 0; i < 16; ++i) sum = fmaf(v[i], v[i], sum);
  }
  sum = cta_sum(sum, red, warps);
  const float rstd = 1.0f / sqrtf(sum / static_cast<float>(a.H) + a.eps);
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t col = 16 * (static_cast<int64_t>(threadIdx.x) + c * blockDim.x);
    const int n = clamp16(a.H - col);
    float v[16], w[16];
    unpack<T>(h[c], v);
    if (a.ck_codes)
      quantize16(v, n, a.ck_codes + row * a.ck_ld + col, a.ck_scales + row * a.ck_lds + col / kFp8Block, lane8);
    load_weight16<VEC>(a.weight, a.weight_dtype, col, n, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] *= v[i] * rstd;
    quantize16(w, n, a.codes + row * a.ldc + col, a.scales + row * a.lds + col / kFp8Block, lane8);
  }
}

// Rows blockIdx.x, blockIdx.x + gridDim.x, ... of the backward pass, the next
// row's loads in flight while one is worked on; the CTA's column sums of
// dy xh go to its row of `partial`.
template <typename T, bool H>
struct BackwardRow {
  Row16<T> dy, dh;
  Row16<T> h;      // H
  uint4 codes;     // !H
  uint32_t scale;
};

template <typename T, int NC, bool VEC, bool H>
__global__ void __launch_bounds__(512) norm_backward_kernel(NormBackwardArgs a, bool wide) {
  __shared__ float red[16];
  const int warps = blockDim.x >> 5;
  float dw[NC][16];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 16; ++i) dw[c][i] = 0.0f;
  grid_launch_dependents();
  grid_dependency_wait();
  BackwardRow<T, H> next[NC];
  float next_rstd = 0.0f;
  const auto fetch = [&](int64_t row) {
    next_rstd = a.rstd[row];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = 16 * (static_cast<int64_t>(threadIdx.x) + c * blockDim.x);
      const int n = clamp16(a.H - col);
      next[c].dy = load16<T, VEC>(static_cast<const T*>(a.dy) + row * a.lddy + col, n, wide);
      if (H) {
        next[c].h = load16<T, VEC>(static_cast<const T*>(a.h) + row * a.ldh + col, n, wide);
      } else {
        next[c].codes = load_codes16(a.ck_codes + row * a.ck_ld + col, n);
        next[c].scale = n > 0 ? a.ck_scales[row * a.ck_lds + col / kFp8Block] : kScaleOne;
      }
      if (a.dh) next[c].dh = load16<T, VEC>(static_cast<const T*>(a.dh) + row * a.lddh + col, n, wide);
    }
  };
  if (blockIdx.x < a.M) fetch(blockIdx.x);
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    BackwardRow<T, H> cur[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) cur[c] = next[c];
    const float rstd = next_rstd;
    if (row + gridDim.x < a.M) fetch(row + gridDim.x);
    float g[NC][16], xh[NC][16];
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = 16 * (static_cast<int64_t>(threadIdx.x) + c * blockDim.x);
      const int n = clamp16(a.H - col);
      unpack<T>(cur[c].dy, g[c]);
      if (H)
        unpack<T>(cur[c].h, xh[c]);
      else
        decode16(cur[c].codes, fp8_scale(cur[c].scale), xh[c]);
      float w[16];
      load_weight16<VEC>(a.weight, a.weight_dtype, col, n, w);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        xh[c][i] = n == 16 || i < n ? xh[c][i] * rstd : 0.0f;
        dw[c][i] = fmaf(g[c][i], xh[c][i], dw[c][i]);
        g[c][i] *= w[i];
        sum = fmaf(g[c][i], xh[c][i], sum);
      }
    }
    const float mean = cta_sum(sum, red, warps) / static_cast<float>(a.H);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = 16 * (static_cast<int64_t>(threadIdx.x) + c * blockDim.x);
#pragma unroll
      for (int i = 0; i < 16; ++i) g[c][i] = rstd * fmaf(-xh[c][i], mean, g[c][i]);
      if (a.dh) {
        float d[16];
        unpack<T>(cur[c].dh, d);
#pragma unroll
        for (int i = 0; i < 16; ++i) g[c][i] += d[i];
      }
      store16<T, VEC>(static_cast<T*>(a.dx) + row * a.lddx + col, clamp16(a.H - col), wide, pack<T>(g[c]));
    }
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t col = 16 * (static_cast<int64_t>(threadIdx.x) + c * blockDim.x);
    const int n = clamp16(a.H - col);
    float* p = a.partial + blockIdx.x * a.H + col;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) p[i] = dw[c][i];
  }
}

// dw = the sum of the G rows of partial sums, in a fixed order: a CTA takes 32
// columns, warp w adds rows w, w + 8, ..., and the 8 sums meet in order.
__global__ void __launch_bounds__(256) norm_dw_kernel(const float* partial, int G, int64_t H, float* dw) {
  __shared__ float part[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  grid_launch_dependents();
  grid_dependency_wait();
  float s = 0.0f;
  if (col < H) {
#pragma unroll 8
    for (int g = warp; g < G; g += 8) s += partial[g * H + col];
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < H) {
    s = part[0][lane];
#pragma unroll
    for (int w = 1; w < 8; ++w) s += part[w][lane];
    dw[col] = s;
  }
}

// Threads and 16-column chunks per thread for H columns: at most 512 threads.
void norm_shape(int64_t H, int* threads, int* nc) {
  const int64_t chunks = (H + 15) / 16;
  *nc = chunks <= 512 ? 1 : chunks <= 1024 ? 2 : 4;
  const int64_t t = (chunks + *nc - 1) / *nc;
  *threads = static_cast<int>((t + 31) / 32 * 32);
}

template <typename T, int NC>
cudaError_t launch_norm_t(const NormArgs& a, int threads, int vec, cudaStream_t st) {
  return launch_dependent(vec ? norm_kernel<T, NC, true> : norm_kernel<T, NC, false>,
                          dim3(static_cast<unsigned>(a.M)), threads, 0, st, a, vec == kVec32);
}

template <typename T, int NC, bool H>
cudaError_t launch_norm_backward_t(const NormBackwardArgs& a, int threads, int vec, int grid, cudaStream_t st) {
  return launch_dependent(vec ? norm_backward_kernel<T, NC, true, H> : norm_backward_kernel<T, NC, false, H>,
                          dim3(grid), threads, 0, st, a, vec == kVec32);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, int dtype, int vec, int sms, cudaStream_t st) {
  (void)sms;
  int threads, nc;
  norm_shape(a.H, &threads, &nc);
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    return nc == 1   ? launch_norm_t<T, 1>(a, threads, vec, st)
           : nc == 2 ? launch_norm_t<T, 2>(a, threads, vec, st)
                     : launch_norm_t<T, 4>(a, threads, vec, st);
  });
}

int norm_backward_ctas(int64_t M, int sms) {
  int64_t most = 2 * static_cast<int64_t>(sms);
  if (most > kNormMaxPartials) most = kNormMaxPartials;
  return static_cast<int>(M < most ? M : most);
}

cudaError_t launch_norm_backward(const NormBackwardArgs& a, int dtype, int vec, int grid, cudaStream_t st) {
  int threads, nc;
  norm_shape(a.H, &threads, &nc);
  const auto launch = [&](auto t, auto held) {
    using T = decltype(t);
    constexpr bool H = decltype(held)::value;
    return nc == 1   ? launch_norm_backward_t<T, 1, H>(a, threads, vec, grid, st)
           : nc == 2 ? launch_norm_backward_t<T, 2, H>(a, threads, vec, grid, st)
                     : launch_norm_backward_t<T, 4, H>(a, threads, vec, grid, st);
  };
  if (grid > 0) {
    const cudaError_t e = with_dtype(dtype, [&](auto t) {
      return a.h ? launch(t, std::true_type{}) : launch(t, std::false_type{});
    });
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(norm_dw_kernel, dim3(static_cast<unsigned>((a.H + 31) / 32)), 256, 0, st,
                          static_cast<const float*>(a.partial), grid, a.H, a.dw);
}

}  // namespace taco
