// The norm of many tensors together, sqrt(sum of squares), and the factor that
// clips it. Squares are summed in fp32 by each thread (16 at a time, a few
// thousand at most), the threads' and CTAs' sums in fp64, in a fixed order.

#include "optim.cuh"

namespace taco {

namespace {

template <int CAP>
struct GradTable {
  uint32_t chunks;
  int count;
  GradEntry t[CAP];
};

template <typename T, bool VEC>
__device__ __forceinline__ float squares16(const void* p, int64_t i0, int n, bool wide) {
  float v[16];
  unpack<T>(load16<T, VEC>(static_cast<const T*>(p) + i0, n, wide), v);
  f2 s{0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 16; i += 2) s = fma2(f2{v[i], v[i + 1]}, f2{v[i], v[i + 1]}, s);
  return s.x + s.y;
}

__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(kFullMask, v, m);
  return v;
}

template <int CAP>
__global__ void __launch_bounds__(kOptimThreads)
grad_squares_kernel(const __grid_constant__ GradTable<CAP> table, double* partial) {
  __shared__ double sums[kOptimThreads / 32];
  grid_launch_dependents();
  grid_dependency_wait();
  float s = 0.0f;
  int e = 0;
  for (uint32_t c = blockIdx.x; c < table.chunks; c += gridDim.x) {
    e = tensor_of(table, c, e);
    const GradEntry& en = table.t[e];
    const int64_t i0 = static_cast<int64_t>(c - en.first) * kOptimChunk + 16 * threadIdx.x;
    const int n = clamp16(en.n - i0);
    if (n == 0) continue;
    if (en.dtype == TACO_DTYPE_F32)
      s += en.vec ? squares16<float, true>(en.p, i0, n, en.wide) : squares16<float, false>(en.p, i0, n, false);
    else if (en.dtype == TACO_DTYPE_BF16)
      s += en.vec ? squares16<__nv_bfloat16, true>(en.p, i0, n, en.wide)
                  : squares16<__nv_bfloat16, false>(en.p, i0, n, false);
    else
      s += en.vec ? squares16<__half, true>(en.p, i0, n, en.wide) : squares16<__half, false>(en.p, i0, n, false);
  }
  const double w = warp_sum64(static_cast<double>(s));
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = w;
  __syncthreads();
  if (threadIdx.x == 0) {
    double all = 0.0;
    for (int i = 0; i < kOptimThreads / 32; ++i) all += sums[i];
    partial[blockIdx.x] = all;
  }
}

__global__ void __launch_bounds__(kOptimThreads) grad_norm_kernel(const double* partial, int count, float most, float* out) {
  __shared__ double sums[kOptimThreads / 32];
  grid_launch_dependents();
  grid_dependency_wait();
  double s = 0.0;
  for (int i = threadIdx.x; i < count; i += kOptimThreads) s += partial[i];
  s = warp_sum64(s);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    double all = 0.0;
    for (int i = 0; i < kOptimThreads / 32; ++i) all += sums[i];
    const float norm = static_cast<float>(sqrt(all));
    out[0] = norm;
    out[1] = !isfinite(norm) ? __uint_as_float(0x7fffffffu) : norm > most ? most / norm : 1.0f;
  }
}

}  // namespace

cudaError_t launch_grad_squares(const GradEntry* entries, int count, uint32_t chunks, int sms, double* partial,
                                int* ctas, cudaStream_t st) {
  const uint32_t most = static_cast<uint32_t>(sms * 6 < kNormCtas ? sms * 6 : kNormCtas);
  const uint32_t grid = chunks < most ? chunks : most;
  *ctas = static_cast<int>(grid);
  const auto go = [&](auto cap) {
    constexpr int CAP = decltype(cap)::value;
    static_assert(sizeof(GradTable<CAP>) <= 32700, "kernel parameters");
    GradTable<CAP> table;
    table.chunks = chunks;
    table.count = count;
    for (int i = 0; i < count; ++i) table.t[i] = entries[i];
    return launch_dependent(grad_squares_kernel<CAP>, dim3(grid), kOptimThreads, 0, st, table, partial);
  };
  return count <= kNormFew ? go(std::integral_constant<int, kNormFew>{})
                           : go(std::integral_constant<int, kNormMany>{});
}

cudaError_t launch_grad_norm(const double* partial, int count, float most, float* out, cudaStream_t st) {
  return launch_dependent(grad_norm_kernel, dim3(1), kOptimThreads, 0, st, partial, count, most, out);
}

}  // namespace taco
