// A tensor [M, K] to FP8 block tensors: its rows (blocks of 128 columns), its
// transpose [K, M] (blocks of 128 of the M rows, what a product that sums
// over the rows reads) or both from one read, with one scale per row and
// block or per 128 x 128 tile. The source is bf16, f16, f32 or itself an FP8
// block tensor.
//
// Rows alone: 16 lanes take one row's block, 8 columns each. With the
// transpose: one CTA takes a 128 x 128 tile through shared memory.

#include "fp8_block.cuh"

namespace taco {

namespace {

constexpr int kThreads = 256;

struct Fp8Source {};   // the source is codes and scales

template <typename T, bool VEC>
__device__ __forceinline__ void read8(const QuantizeArgs& a, int64_t row, int64_t col, int n, float (&v)[8]) {
  if constexpr (std::is_same<T, Fp8Source>::value) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    if (n > 0)
      decode8(load_codes8(static_cast<const uint8_t*>(a.x) + row * a.ldx + col, n),
              fp8_scale(a.x_scales[(row / a.x_tile) * a.x_lds + col / kFp8Block]), v);
  } else {
    load8<T, VEC>(static_cast<const T*>(a.x) + row * a.ldx + col, n, v);
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(QuantizeArgs a) {
  const int lane = threadIdx.x & 15;
  const int64_t kb = (a.K + kFp8Block - 1) / kFp8Block;
  const int64_t groups = static_cast<int64_t>(gridDim.x) * (kThreads / 16);
  const int64_t total = a.M * kb;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads / 16) + (threadIdx.x >> 5) * 2;
  grid_launch_dependents();
  grid_dependency_wait();
  for (int64_t pair = first; pair < total; pair += groups) {
    const int64_t blk = pair + ((threadIdx.x >> 4) & 1);
    const int64_t row = blk / kb, k = blk - row * kb;
    const int64_t col = k * kFp8Block + 8 * lane;
    const int n = blk < total ? clamp8(a.K - col) : 0;
    float v[8];
    read8<T, VEC>(a, row, col, n, v);
    const uint32_t b = fp8_scale_byte(group_umax<16>(amax8(v)));
    if (n > 0) {
      store_codes8(a.codes + row * a.ldc + col, n, codes8(v, fp8_inverse_scale(b)));
      if (lane == 0) a.scales[row * a.lds + k] = static_cast<uint8_t>(b);
    }
  }
}

// Words of a tile's row in shared memory: 128 values and one of padding, so
// that 32 lanes reading down a column hit 32 banks.
constexpr int kPitch = kFp8Block + 1;
constexpr size_t kTileSmem = sizeof(float) * kFp8Block * kPitch;

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) quantize_tile_kernel(QuantizeArgs a) {
  extern __shared__ float tile[];   // [128][kPitch]
  __shared__ uint32_t tile_max;
  const int64_t kb = (a.K + kFp8Block - 1) / kFp8Block;
  const int64_t rb = blockIdx.x / kb, cb = blockIdx.x - rb * kb;   // this tile's row and column of tiles
  const int64_t r0 = rb * kFp8Block, c0 = cb * kFp8Block;
  const int lane = threadIdx.x & 15, slot = threadIdx.x >> 4;
  if (threadIdx.x == 0) tile_max = 0;
  __syncthreads();
  grid_launch_dependents();
  grid_dependency_wait();
  uint32_t m = 0;
  for (int r = slot; r < kFp8Block; r += kThreads / 16) {
    const int n = r0 + r < a.M ? clamp8(a.K - c0 - 8 * lane) : 0;
    float v[8];
    read8<T, VEC>(a, r0 + r, c0 + 8 * lane, n, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) tile[r * kPitch + 8 * lane + i] = v[i];
    const uint32_t top = group_umax<16>(amax8(v));
    m = max(m, top);
    if (a.codes && a.tile == 1 && n > 0) {
      const uint32_t b = fp8_scale_byte(top);
      store_codes8(a.codes + (r0 + r) * a.ldc + c0 + 8 * lane, n, codes8(v, fp8_inverse_scale(b)));
      if (lane == 0) a.scales[(r0 + r) * a.lds + cb] = static_cast<uint8_t>(b);
    }
  }
  if (a.tile != 1) atomicMax(&tile_max, m);
  __syncthreads();
  if (a.tile != 1) {
    const uint32_t b = fp8_scale_byte(tile_max);
    if (threadIdx.x == 0) {
      if (a.codes) a.scales[rb * a.lds + cb] = static_cast<uint8_t>(b);
      if (a.t_codes) a.t_scales[cb * a.t_lds + rb] = static_cast<uint8_t>(b);
    }
    if (a.codes)
      for (int r = slot; r < kFp8Block; r += kThreads / 16) {
        const int n = r0 + r < a.M ? clamp8(a.K - c0 - 8 * lane) : 0;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = tile[r * kPitch + 8 * lane + i];
        store_codes8(a.codes + (r0 + r) * a.ldc + c0 + 8 * lane, n, codes8(v, fp8_inverse_scale(b)));
      }
  }
  if (!a.t_codes) return;
  // the transpose: 16 lanes take one column, 8 rows each
  for (int c = slot; c < kFp8Block; c += kThreads / 16) {
    const int n = c0 + c < a.K ? clamp8(a.M - r0 - 8 * lane) : 0;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = tile[(8 * lane + i) * kPitch + c];
    const uint32_t b = fp8_scale_byte(a.tile == 1 ? group_umax<16>(amax8(v)) : tile_max);
    store_codes8(a.t_codes + (c0 + c) * a.t_ldc + r0 + 8 * lane, n, codes8(v, fp8_inverse_scale(b)));
    if (a.tile == 1 && lane == 0 && n > 0) a.t_scales[(c0 + c) * a.t_lds + rb] = static_cast<uint8_t>(b);
  }
}

template <typename T, bool VEC>
cudaError_t launch_t(const QuantizeArgs& a, int sms, cudaStream_t st) {
  const int64_t kb = (a.K + kFp8Block - 1) / kFp8Block;
  if (!a.t_codes && a.tile == 1) {
    const int64_t want = (a.M * kb + kThreads / 16 - 1) / (kThreads / 16);
    const int64_t most = 8 * static_cast<int64_t>(sms);
    return launch_dependent(quantize_rows_kernel<T, VEC>, dim3(static_cast<unsigned>(want < most ? want : most)),
                            kThreads, 0, st, a);
  }
  const dim3 grid(static_cast<unsigned>(kb * ((a.M + kFp8Block - 1) / kFp8Block)));
  return launch_dependent(quantize_tile_kernel<T, VEC>, grid, kThreads, kTileSmem, st, a);
}

template <typename F>
void each_tile_kernel(F&& f) {
  f(reinterpret_cast<const void*>(quantize_tile_kernel<__nv_bfloat16, true>));
  f(reinterpret_cast<const void*>(quantize_tile_kernel<__nv_bfloat16, false>));
  f(reinterpret_cast<const void*>(quantize_tile_kernel<__half, true>));
  f(reinterpret_cast<const void*>(quantize_tile_kernel<__half, false>));
  f(reinterpret_cast<const void*>(quantize_tile_kernel<float, true>));
  f(reinterpret_cast<const void*>(quantize_tile_kernel<float, false>));
  f(reinterpret_cast<const void*>(quantize_tile_kernel<Fp8Source, true>));
}

}  // namespace

cudaError_t prepare_quantize() {
  cudaError_t e = cudaSuccess;
  each_tile_kernel([&](const void* k) {
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kTileSmem));
  });
  return e;
}

cudaError_t launch_quantize(const QuantizeArgs& a, int dtype, bool vec, int sms, cudaStream_t st) {
  if (a.x_scales) return launch_t<Fp8Source, true>(a, sms, st);
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    return vec ? launch_t<T, true>(a, sms, st) : launch_t<T, false>(a, sms, st);
  });
}

}  // namespace taco
