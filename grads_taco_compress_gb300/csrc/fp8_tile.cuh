// What the kernels that quantise 128 x 128 tiles both ways share
// (fp8_quantize.cu, fp8_linear_backward.cu): 256 threads, each 4 consecutive
// rows of 16 columns; the transposed codes go through shared memory, 4 rows of a
// column to a word, so that they leave as whole 128-byte rows.
#pragma once

#include "fp8_block.cuh"

namespace taco {

constexpr int kTileThreads = 256;

__device__ __forceinline__ int clamp4(int64_t left) { return left < 0 ? 0 : (left > 4 ? 4 : static_cast<int>(left)); }

// Word of the transposed tile that holds rows 4 r4 .. 4 r4 + 3 of column c: 32
// words a column, in the order r4 ^ 4 (c / 16 % 8). A warp writes one column
// of each of its 8 lane groups at a time, 4 words apiece: 32 banks.
__device__ __forceinline__ int tile_word(int c, int r4) { return c * 32 + (r4 ^ (4 * ((c >> 4) & 7))); }

// 8 lanes write the 128 codes of one column of the transposed tile, 16 each; the
// tile begins at row r0 and column c0 of the matrix [M, K].
__device__ __forceinline__ void store_transposed(uint8_t* t_codes, int64_t t_ldc, int64_t M, int64_t K,
                                                 const uint32_t* words, int64_t r0, int64_t c0, int lane8, int r4) {
  const int n = clamp16(M - r0 - 16 * lane8);
  const int64_t left = K - c0 - r4;
  uint8_t* const p = t_codes + (c0 + r4) * t_ldc + r0 + 16 * lane8;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 w = *reinterpret_cast<const uint4*>(&words[tile_word(32 * i + r4, 4 * lane8)]);
    store_codes16(p + 32 * i * t_ldc, 32 * i < left ? n : 0, w);
  }
}

}  // namespace taco
