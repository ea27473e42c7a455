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
// One CTA takes a row at a time; thread t holds the 8-column chunks t, t + T,
// ... in registers, so a row is read once and a block of 128 columns is 16
// consecutive lanes. Sums are fp32.

#include "fp8_block.cuh"

namespace taco {

namespace {

template <typename T, int NC, bool VEC>
__global__ void __launch_bounds__(512) norm_kernel(NormArgs a) {
  __shared__ float red[32];
  const int warps = blockDim.x >> 5;
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.residual);
  T* hout = static_cast<T*>(a.h);
  grid_launch_dependents();
  grid_dependency_wait();
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    float v[NC][8];
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = 8 * (static_cast<int64_t>(threadIdx.x) + c * blockDim.x);
      const int n = clamp8(a.H - col);
      load8<T, VEC>(x + row * a.ldx + col, n, v[c]);
      if (res) {
        float r[8];
        load8<T, VEC>(res + row * a.ldr + col, n, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] = to_f32(from_f32<T>(v[c][i] + r[i]));
        store8<T, VEC>(hout + row * a.ldh + col, n, v[c]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(v[c][i], v[c][i], sum);
    }
    sum = cta_sum(sum, red, warps);
    const float rstd = 1.0f / sqrtf(sum / static_cast<float>(a.H) + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = 8 * (static_cast<int64_t>(threadIdx.x) + c * blockDim.x);
      const int n = clamp8(a.H - col);
      if (a.ck_codes) {
        const uint32_t b = fp8_scale_byte(group_umax<16>(amax8(v[c])));
        if (n > 0) {
          store_codes8(a.ck_codes + row * a.ck_ld + col, n, codes8(v[c], fp8_inverse_scale(b)));
          if ((threadIdx.x & 15) == 0)
            a.ck_scales[row * a.ck_lds + col / kFp8Block] = static_cast<uint8_t>(b);
        }
      }
      float w[8], y[8];
      load_weight8<VEC>(a.weight, a.weight_dtype, col, n, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = v[c][i] * rstd * w[i];
      const uint32_t b = fp8_scale_byte(group_umax<16>(amax8(y)));
      if (n > 0) {
        store_codes8(a.codes + row * a.ldc + col, n, codes8(y, fp8_inverse_scale(b)));
        if ((threadIdx.x & 15) == 0) a.scales[row * a.lds + col / kFp8Block] = static_cast<uint8_t>(b);
      }
    }
  }
}

// Rows blockIdx.x, blockIdx.x + gridDim.x, ... of the backward pass; the
// CTA's column sums of dy xh go to its row of `partial`.
template <typename T, int NC, bool VEC>
__global__ void __launch_bounds__(512) norm_backward_kernel(NormBackwardArgs a) {
  __shared__ float red[32];
  const int warps = blockDim.x >> 5;
  const T* dy = static_cast<const T*>(a.dy);
  const T* h = static_cast<const T*>(a.h);
  const T* dh = static_cast<const T*>(a.dh);
  T* dx = static_cast<T*>(a.dx);
  float dw[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = 0.0f;
  grid_launch_dependents();
  grid_dependency_wait();
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    float g[NC][8], xh[NC][8];
    float sum = 0.0f;
    const float rstd = a.rstd[row];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = 8 * (static_cast<int64_t>(threadIdx.x) + c * blockDim.x);
      const int n = clamp8(a.H - col);
      load8<T, VEC>(dy + row * a.lddy + col, n, g[c]);
      if (h) {
        load8<T, VEC>(h + row * a.ldh + col, n, xh[c]);
      } else if (n > 0) {
        const uint32_t b = a.ck_scales[row * a.ck_lds + col / kFp8Block];
        decode8(load_codes8(a.ck_codes + row * a.ck_ld + col, n), fp8_scale(b), xh[c]);
      }
      float w[8];
      load_weight8<VEC>(a.weight, a.weight_dtype, col, n, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        xh[c][i] = n > 0 ? xh[c][i] * rstd : 0.0f;
        dw[c][i] = fmaf(g[c][i], xh[c][i], dw[c][i]);
        g[c][i] *= w[i];
        sum = fmaf(g[c][i], xh[c][i], sum);
      }
    }
    const float mean = cta_sum(sum, red, warps) / static_cast<float>(a.H);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = 8 * (static_cast<int64_t>(threadIdx.x) + c * blockDim.x);
      const int n = clamp8(a.H - col);
      float r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = rstd * fmaf(-xh[c][i], mean, g[c][i]);
      if (dh) {
        float d[8];
        load8<T, VEC>(dh + row * a.lddh + col, n, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] += d[i];
      }
      store8<T, VEC>(dx + row * a.lddx + col, n, r);
    }
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t col = 8 * (static_cast<int64_t>(threadIdx.x) + c * blockDim.x);
    const int n = clamp8(a.H - col);
    float* p = a.partial + blockIdx.x * a.H + col;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = dw[c][i];
  }
}

// dw = the sum of the G rows of partial sums, in order.
__global__ void norm_dw_kernel(const float* partial, int G, int64_t H, float* dw) {
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t col = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (col >= H) return;
  float s = 0.0f;
  for (int g = 0; g < G; ++g) s += partial[g * H + col];
  dw[col] = s;
}

// Threads and chunks per thread for H columns.
void norm_shape(int64_t H, int* threads, int* nc) {
  const int64_t chunks = (H + 7) / 8;
  *nc = chunks <= 512 ? 1 : chunks <= 1024 ? 2 : chunks <= 2048 ? 4 : 8;
  const int64_t t = (chunks + *nc - 1) / *nc;
  *threads = static_cast<int>((t + 31) / 32 * 32);
}

template <typename T, bool VEC>
cudaError_t launch_norm_t(const NormArgs& a, int sms, cudaStream_t st) {
  (void)sms;
  int threads, nc;
  norm_shape(a.H, &threads, &nc);
  const int64_t most = 1 << 30;
  const dim3 grid(static_cast<unsigned>(a.M < most ? a.M : most));
  switch (nc) {
    case 1: return launch_dependent(norm_kernel<T, 1, VEC>, grid, threads, 0, st, a);
    case 2: return launch_dependent(norm_kernel<T, 2, VEC>, grid, threads, 0, st, a);
    case 4: return launch_dependent(norm_kernel<T, 4, VEC>, grid, threads, 0, st, a);
    default: return launch_dependent(norm_kernel<T, 8, VEC>, grid, threads, 0, st, a);
  }
}

template <typename T, bool VEC>
cudaError_t launch_norm_backward_t(const NormBackwardArgs& a, int grid, cudaStream_t st) {
  int threads, nc;
  norm_shape(a.H, &threads, &nc);
  cudaError_t e = cudaSuccess;
  if (grid > 0) switch (nc) {
    case 1: e = launch_dependent(norm_backward_kernel<T, 1, VEC>, dim3(grid), threads, 0, st, a); break;
    case 2: e = launch_dependent(norm_backward_kernel<T, 2, VEC>, dim3(grid), threads, 0, st, a); break;
    case 4: e = launch_dependent(norm_backward_kernel<T, 4, VEC>, dim3(grid), threads, 0, st, a); break;
    default: e = launch_dependent(norm_backward_kernel<T, 8, VEC>, dim3(grid), threads, 0, st, a); break;
  }
  if (e != cudaSuccess) return e;
  return launch_dependent(norm_dw_kernel, dim3(static_cast<unsigned>((a.H + 127) / 128)), 128, 0, st,
                          static_cast<const float*>(a.partial), grid, a.H, a.dw);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, int dtype, bool vec, int sms, cudaStream_t st) {
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    return vec ? launch_norm_t<T, true>(a, sms, st) : launch_norm_t<T, false>(a, sms, st);
  });
}

int norm_backward_ctas(int64_t M, int sms) {
  int64_t most = 2 * static_cast<int64_t>(sms);
  if (most > kNormMaxPartials) most = kNormMaxPartials;
  return static_cast<int>(M < most ? M : most);
}

cudaError_t launch_norm_backward(const NormBackwardArgs& a, int dtype, bool vec, int grid,
                                 cudaStream_t st) {
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    return vec ? launch_norm_backward_t<T, true>(a, grid, st)
               : launch_norm_backward_t<T, false>(a, grid, st);
  });
}

}  // namespace taco
