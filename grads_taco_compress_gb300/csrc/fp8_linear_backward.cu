// The gradient at a layer's product, d = dy act'(pre), from the 8-bit checkpoint
// of pre: its FP8 rows (what the input's gradient reads), its FP8 transpose (what
// the weight's reads) and the bias's gradient, the sum of its rows, from one read
// of dy and of the checkpoint. d itself is never written: it is quantised from
// fp32, rounded once.
//
// A CTA takes a 128 x 128 tile, each thread 4 consecutive rows of 16 columns,
// whose d stay in registers. Largest magnitudes and sums of the columns meet in
// shared memory. Tiles write their column sums; a second kernel adds them in the
// order of the rows.

#include "fp8_activation.cuh"
#include "fp8_tile.cuh"

namespace taco {

namespace {

template <typename T, bool VEC>
__global__ void __launch_bounds__(kTileThreads, 2)
linear_backward_kernel(LinearBackwardArgs a, Divider per_row, bool wide) {
  __shared__ __align__(16) uint32_t words[kFp8Block * 32];
  __shared__ __align__(16) uint32_t col_max[kTileThreads / 32][kFp8Block];
  __shared__ __align__(16) float col_sum[kTileThreads / 32][kFp8Block];
  __shared__ __align__(16) float col_inv[kFp8Block];
  const int64_t rb = per_row.quotient(blockIdx.x);
  const int64_t cb = blockIdx.x - rb * static_cast<int64_t>(per_row.d);
  const int lane8 = threadIdx.x & 7, r4 = threadIdx.x >> 3, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r0 = rb * kFp8Block, c0 = cb * kFp8Block;
  const int64_t row = r0 + 4 * r4, col = c0 + 16 * lane8;
  const int n = clamp16(a.N - col), rows = clamp4(a.M - row);
  grid_launch_dependents();
  grid_dependency_wait();

  const T* const p = static_cast<const T*>(a.dy) + row * a.lddy + col;
  float d[4][16];
  {
    Row16<T> g[4];
    uint4 codes[4];
    uint32_t scale[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) g[i] = load16<T, VEC>(p + i * a.lddy, i < rows ? n : 0, wide);
    if (a.act != TACO_ACT_NONE) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool any = i < rows && n > 0;
        codes[i] = load_codes16(a.k_codes + (row + i) * a.k_ld + col, any ? n : 0);
        scale[i] = any ? a.k_scales[(row + i) * a.k_lds + cb] : kScaleOne;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack<T>(g[i], d[i]);
    with_act(a.act, [&](auto kind) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x[16];
        decode16(codes[i], fp8_scale(scale[i]), x);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const f2 y = mul2(f2{d[i][e], d[i][e + 1]}, slope2<decltype(kind)::value>(f2{x[e], x[e + 1]}));
          d[i][e] = y.x;
          d[i][e + 1] = y.y;
        }
        if (scale[i] == kScaleNan) {   // which must not reach columns that do not exist
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (e >= n) d[i][e] = 0.0f;
        }
      }
    });
  }
  if (a.codes) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      quantize16(d[i], i < rows ? n : 0, a.codes + (row + i) * a.ldc + col, a.scales + (row + i) * a.lds + cb, lane8);
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    // over the thread's 4 rows and the 4 lanes of the warp with the same columns
    uint32_t top = __float_as_uint(amax3(amax3(0.0f, d[0][e], d[1][e]), d[2][e], d[3][e]));
    float sum = (d[0][e] + d[1][e]) + (d[2][e] + d[3][e]);
#pragma unroll
    for (int m = 8; m < 32; m <<= 1) {
      top = max(top, __shfl_xor_sync(kFullMask, top, m));
      sum += __shfl_xor_sync(kFullMask, sum, m);
    }
    if (lane < 8) {
      col_max[warp][16 * lane8 + e] = top;
      col_sum[warp][16 * lane8 + e] = sum;
    }
  }
  __syncthreads();
  if (threadIdx.x < kFp8Block) {
    const int c = threadIdx.x;
    uint32_t top = 0;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kTileThreads / 32; ++w) {
      top = max(top, col_max[w][c]);
      sum += col_sum[w][c];
    }
    const uint32_t b = fp8_scale_byte(top);
    col_inv[c] = fp8_inverse_scale(b);
    if (c0 + c < a.N) {
      if (a.t_codes) a.t_scales[(c0 + c) * a.t_lds + rb] = static_cast<uint8_t>(b);
      if (a.sums) a.sums[rb * a.N + c0 + c] = sum;
    }
  }
  if (!a.t_codes) return;
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int c = 16 * lane8 + e;
    const float inv = col_inv[c];
    words[tile_word(c, r4)] = e4m3x4_from_f32(d[0][e] * inv, d[1][e] * inv, d[2][e] * inv, d[3][e] * inv);
  }
  __syncthreads();
  store_transposed(a.t_codes, a.t_ldc, a.M, a.N, words, r0, c0, lane8, r4);
}

// Sums of the columns of [rows, N], a warp 32 columns of every eighth row, joined
// in order.
__global__ void __launch_bounds__(256) column_sums_kernel(const float* sums, int64_t rows, int64_t N, float* out) {
  __shared__ float part[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  grid_launch_dependents();
  grid_dependency_wait();
  float s = 0.0f;
  if (c < N) {
#pragma unroll 4
    for (int64_t r = warp; r < rows; r += 8) s += sums[r * N + c];
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < N) {
    float all = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) all += part[w][lane];
    out[c] = all;
  }
}

}  // namespace

cudaError_t launch_linear_backward(const LinearBackwardArgs& args, int dtype, int vec, float* db, float* workspace,
                                   cudaStream_t st) {
  LinearBackwardArgs a = args;
  const Divider per_row((a.N + kFp8Block - 1) / kFp8Block);
  const int64_t tiles = (a.M + kFp8Block - 1) / kFp8Block;
  if (db) a.sums = tiles == 1 ? db : workspace;
  const dim3 grid(static_cast<unsigned>(per_row.d * tiles));
  const cudaError_t e = with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    return vec ? launch_dependent(linear_backward_kernel<T, true>, grid, kTileThreads, 0, st, a, per_row, vec == kVec32)
               : launch_dependent(linear_backward_kernel<T, false>, grid, kTileThreads, 0, st, a, per_row, false);
  });
  if (e != cudaSuccess || !db || tiles == 1) return e;
  return launch_dependent(column_sums_kernel, dim3(static_cast<unsigned>((a.N + 31) / 32)), 256, 0, st,
                          static_cast<const float*>(workspace), tiles, a.N, db);
}

}  // namespace taco
