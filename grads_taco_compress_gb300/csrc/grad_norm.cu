// The norm of many tensors together, sqrt(sum of squares), and the factor that
// clips it. Squares are summed in fp32 by each thread 16 or 32 at a time, and all
// sums of those in fp64, in a fixed order: a thread's own sum may be one of
// millions of elements. (An addition in fp64 for 64 bytes costs 1%, for 512 bytes no
// less: 134M f32 81.3 us, 80.5 with all of a thread's in fp32.) Where a thread's
// squares may leave fp32 they are formed again of scaled values, so that every finite
// value counts whatever its magnitude.
//
// Measured: 134M f32 81 us, 6.6 TB/s (a plain copy: 6.78), bf16 43.6 us; 96 small
// vectors 5.4 us, two launches.

#include "optim.cuh"

namespace taco {

namespace {

// CTAs per SM. 64 bytes a thread at a time, 134M f32 and bf16 elements: 4: 86, 43.7 us,
// 6: 79.6 and 41.8 us (1.00 and 0.95 of the copy peak).
constexpr int kNormPerSm = 6;

template <int CAP>
struct GradTable {
  uint32_t chunks;
  int count;
  GradEntry t[CAP];
};

// The sum of the squares of a thread's elements (16 of every 4096 of a chunk) where
// the plain sum is below 2^-90 or not below 2^120, or none: the squares of values
// times a power of two that brings the largest one's well within fp32. Values so much
// smaller that theirs vanish count for nothing. They are read again, one at a time:
// registers for this would cost all others 2%.
template <typename T>
__device__ __forceinline__ double squares_at_the_ends(const T* p, int64_t left, int parts) {
  float top = 0.0f;
#pragma unroll 1
  for (int k = 0; k < parts; ++k) {
    const int n = clamp16(left - k * kOptimChunk);
#pragma unroll 1
    for (int i = 0; i < n; ++i) top = amax3(top, to_f32(p[k * kOptimChunk + i]), 0.0f);
  }
  if (!(top > 0.0f && top < __uint_as_float(0x7f800000u))) return static_cast<double>(top);   // 0, infinity, NaN
  const float f = top < 1.0f ? 0x1p100f : 0x1p-80f;
  float s = 0.0f;
#pragma unroll 1
  for (int k = 0; k < parts; ++k) {
    const int n = clamp16(left - k * kOptimChunk);
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const float v = to_f32(p[k * kOptimChunk + i]) * f;
      s += v * v;
    }
  }
  return static_cast<double>(s) * (top < 1.0f ? 0x1p-200 : 0x1p160);
}

// Of the thread's elements in a tensor's chunk, 64 bytes of them: 16 of every
// 4096, all loaded before the first is used.
template <typename T>
__device__ __forceinline__ double squares(const GradEntry& en, uint32_t chunk) {
  constexpr int64_t kElems = kNormChunkBytes / static_cast<int64_t>(sizeof(T));
  constexpr int kParts = static_cast<int>(kElems / kOptimChunk);
  const int64_t base = static_cast<int64_t>(chunk) * kElems + 16 * threadIdx.x;
  const T* const p = static_cast<const T*>(en.p) + base;
  Row16<T> r[kParts];
#pragma unroll
  for (int k = 0; k < kParts; ++k) {
    const int n = clamp16(en.n - base - k * kOptimChunk);
    const T* const q = n > 0 ? p + k * kOptimChunk : static_cast<const T*>(en.p);
    r[k] = en.vec ? load16<T, true>(q, n, en.wide) : load16<T, false>(q, n, false);
  }
  f2 s{0.0f, 0.0f}, t{0.0f, 0.0f};
  uint32_t any = 0;
#pragma unroll
  for (int k = 0; k < kParts; ++k) {
    float v[16];
    unpack<T>(r[k], v);
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      s = fma2(f2{v[i], v[i + 1]}, f2{v[i], v[i + 1]}, s);
      t = fma2(f2{v[i + 2], v[i + 3]}, f2{v[i + 2], v[i + 3]}, t);
    }
    for (const uint32_t w : r[k].w) any |= w;
  }
  s = add2(s, t);
  const float sum = s.x + s.y;
  if constexpr (!std::is_same<T, __half>::value) {   // whose squares are all between 2^-48 and 2^32
    if (!(sum >= 0x1p-90f && sum < 0x1p120f) && any) return squares_at_the_ends<T>(p, en.n - base, kParts);
  }
  return static_cast<double>(sum);
}

__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(kFullMask, v, m);
  return v;
}

template <int CAP>
__global__ void __launch_bounds__(kOptimThreads, kNormPerSm)
grad_squares_kernel(const __grid_constant__ GradTable<CAP> table, double* partial) {
  __shared__ double sums[kOptimThreads / 32];
  grid_launch_dependents();
  grid_dependency_wait();
  double s = 0.0;
  int e = 0;
  for (uint32_t c = blockIdx.x; c < table.chunks; c += gridDim.x) {
    e = tensor_of(table, c, e);
    const GradEntry& en = table.t[e];
    if (en.dtype == TACO_DTYPE_F32)
      s += squares<float>(en, c - en.first);
    else if (en.dtype == TACO_DTYPE_BF16)
      s += squares<__nv_bfloat16>(en, c - en.first);
    else
      s += squares<__half>(en, c - en.first);
  }
  const double w = warp_sum64(s);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = w;
  __syncthreads();
  if (threadIdx.x == 0) {
    double all = 0.0;
    for (int i = 0; i < kOptimThreads / 32; ++i) all += sums[i];
    partial[blockIdx.x] = all;
  }
}

__global__ void __launch_bounds__(kOptimThreads)
grad_norm_kernel(const double* partial, int count, float most, float* out) {
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
  const uint32_t most = static_cast<uint32_t>(sms * kNormPerSm < kNormCtas ? sms * kNormPerSm : kNormCtas);
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
