// A tensor [M, K] to FP8 block tensors: its rows (blocks of 128 columns), its
// transpose [K, M] (blocks of 128 of the M rows, what a product that sums
// over the rows reads) or both from one read, with one scale per row and
// block or per 128 x 128 tile. The source is bf16, f16, f32 or itself an FP8
// block tensor.
//
// Rows alone: a warp takes 512 columns of one row, 8 lanes a block of 128.
// With the transpose (or tiles): one CTA takes a 128 x 128 tile, each thread 4
// consecutive rows of 16 columns, which stay in registers. The largest
// magnitudes of the columns meet in shared memory; the transposed codes go
// through it too, 4 rows of a column to a word, so that they leave as whole
// 128-byte rows.
//
// The transpose of codes alone works on pairs of fp16 (below).
//
// Measured (a plain copy: 6.7 TB/s): rows of 8192 x 4096 bf16 15.4 us, 6.5 TB/s;
// rows and transpose from one read 25.0 us, 5.4 TB/s;
// the transpose of 8192 x 1600 codes 8.1 us at 780 instructions a thread, 53% of
// the issue slots and 1.4 waves of CTAs (13.7 us and 1500 in fp32).

#include "fp8_block.cuh"

namespace taco {

namespace {

constexpr int kThreads = 256;

struct Fp8Source {};   // the source is codes and scales

// 16 columns of a row as they lie in memory (of which n exist, the others are
// zero).
struct Fp8Row16 {
  uint4 codes;
  uint32_t scale, n;
};
template <typename T>
struct RowOf {
  using type = Row16<T>;
};
template <>
struct RowOf<Fp8Source> {
  using type = Fp8Row16;
};
template <typename T, bool VEC>
__device__ __forceinline__ typename RowOf<T>::type read16(const QuantizeArgs& a, int64_t row, int64_t col, int n,
                                                          bool wide) {
  if constexpr (std::is_same<T, Fp8Source>::value) {
    Fp8Row16 r{make_uint4(0, 0, 0, 0), kScaleOne, static_cast<uint32_t>(n)};
    if (n > 0) {
      r.codes = load_codes16(static_cast<const uint8_t*>(a.x) + row * a.ldx + col, n);
      r.scale = a.x_scales[(a.x_tile == 1 ? row : row / kFp8Block) * a.x_lds + col / kFp8Block];
    }
    return r;
  } else {
    return load16<T, VEC>(static_cast<const T*>(a.x) + row * a.ldx + col, n, wide);
  }
}
// Columns 4 q .. 4 q + 3 of them as fp32.
template <typename T>
__device__ __forceinline__ void values4(const typename RowOf<T>::type& r, int q, float* v) {
  if constexpr (std::is_same<T, Fp8Source>::value) {
    decode4(q == 0 ? r.codes.x : q == 1 ? r.codes.y : q == 2 ? r.codes.z : r.codes.w, fp8_scale(r.scale), v);
    if (r.scale == kScaleNan) {   // which must not reach columns that do not exist
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * q + i >= static_cast<int>(r.n)) v[i] = 0.0f;
    }
  } else if constexpr (std::is_same<T, float>::value) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r.w[4 * q + i]);
  } else if constexpr (std::is_same<T, __half>::value) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.w[2 * q + i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[2 * i] = bf16_lo(r.w[2 * q + i]);
      v[2 * i + 1] = bf16_hi(r.w[2 * q + i]);
    }
  }
}
template <typename T>
__device__ __forceinline__ void values16(const typename RowOf<T>::type& r, float (&v)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) values4<T>(r, q, v + 4 * q);
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(QuantizeArgs a, Divider per_row, bool wide) {
  const int lane8 = threadIdx.x & 7;
  const uint64_t w = static_cast<uint64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t row = per_row.quotient(w);
  const int64_t k = static_cast<int64_t>(w - row * per_row.d) * 4 + ((threadIdx.x >> 3) & 3);
  const int64_t col = k * kFp8Block + 16 * lane8;
  grid_launch_dependents();
  grid_dependency_wait();
  if (row >= a.M) return;   // whole warps
  const int n = clamp16(a.K - col);
  float v[16];
  values16<T>(read16<T, VEC>(a, row, col, n, wide), v);
  quantize16(v, n, a.codes + row * a.ldc + col, a.scales + row * a.lds + k, lane8);
}

// Four rows of 16 columns of a tile that begins at (rb, cb) blocks, the first at
// (row, col); n: the columns that exist, rows: the rows.
template <typename T, bool VEC>
__device__ __forceinline__ void read_tile(const QuantizeArgs& a, int64_t rb, int64_t cb, int64_t row, int64_t col,
                                          int n, int rows, bool wide, typename RowOf<T>::type (&r)[4]) {
  if constexpr (std::is_same<T, Fp8Source>::value) {
    const uint8_t* p = static_cast<const uint8_t*>(a.x) + row * a.ldx + col;
    const uint8_t* s = a.x_scales + (a.x_tile == 1 ? row : rb) * a.x_lds + cb;
    const int64_t step = a.x_tile == 1 ? a.x_lds : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool any = i < rows && n > 0;
      r[i] = Fp8Row16{make_uint4(0, 0, 0, 0), kScaleOne, static_cast<uint32_t>(any ? n : 0)};
      if (any) {
        r[i].codes = load_codes16(p + i * a.ldx, n);
        r[i].scale = s[i * step];
      }
    }
  } else {
    const T* p = static_cast<const T*>(a.x) + row * a.ldx + col;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = load16<T, VEC>(p + i * a.ldx, i < rows ? n : 0, wide);
  }
}
__device__ __forceinline__ int clamp4(int64_t left) { return left < 0 ? 0 : (left > 4 ? 4 : static_cast<int>(left)); }

// Word of the transposed tile that holds rows 4 r4 .. 4 r4 + 3 of column c: 32
// words a column, in the order r4 ^ 4 (c / 16 % 8). A warp writes one column
// of each of its 8 lane groups at a time, 4 words apiece: 32 banks.
__device__ __forceinline__ int tile_word(int c, int r4) { return c * 32 + (r4 ^ (4 * ((c >> 4) & 7))); }

// The largest magnitudes of a tile's columns. 16-bit types (and re-blocked
// codes, below) stay packed, pairs of columns to a word: with the sign cleared
// their order is that of unsigned integers, NaN above infinity. Every warp
// writes the 64 words of its 16 rows to `words`; after a barrier the first 64
// threads join them.
constexpr uint32_t kAbs2 = 0x7fff7fffu;
constexpr int kPairs = kFp8Block / 2;

__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  uint32_t m = __vmaxu2(__vimax3_u16x2(a & kAbs2, b & kAbs2, c & kAbs2), d & kAbs2);
  m = __vmaxu2(m, __shfl_xor_sync(kFullMask, m, 8));
  return __vmaxu2(m, __shfl_xor_sync(kFullMask, m, 16));
}
__device__ __forceinline__ void put_pairs(const uint32_t (&m)[8], uint32_t* words) {
  const int lane = threadIdx.x & 31;
  if (lane < 8) {
    uint4* to = reinterpret_cast<uint4*>(&words[(threadIdx.x >> 5) * kPairs + 8 * lane]);
    to[0] = make_uint4(m[0], m[1], m[2], m[3]);
    to[1] = make_uint4(m[4], m[5], m[6], m[7]);
  }
}
__device__ __forceinline__ uint32_t join_pairs(const uint32_t* words, int pair) {
  uint32_t all = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) all = __vmaxu2(all, words[i * kPairs + pair]);
  return all;
}
// 32-bit types: over the thread's 4 rows and the 4 lanes of the warp that hold
// other rows of the same columns, into col_max (fp32 bits).
template <typename T>
__device__ __forceinline__ void fold_columns(const typename RowOf<T>::type (&r)[4], uint32_t* col_max, int lane8) {
  const bool writes = (threadIdx.x & 31) < 8;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float v[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) values4<T>(r[i], q, v[i]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t w = __float_as_uint(amax3(amax3(0.0f, v[0][e], v[1][e]), v[2][e], v[3][e]));
      w = max(w, __shfl_xor_sync(kFullMask, w, 8));
      w = max(w, __shfl_xor_sync(kFullMask, w, 16));
      if (writes) atomicMax(&col_max[16 * lane8 + 4 * q + e], w);
    }
  }
}
// The two halves of a word as fp32 bits.
template <typename T>
__device__ __forceinline__ void pair_bits(uint32_t w, uint32_t (&b)[2]) {
  if constexpr (std::is_same<T, __half>::value) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    b[0] = __float_as_uint(f.x);
    b[1] = __float_as_uint(f.y);
  } else {
    b[0] = w << 16;
    b[1] = w & 0xffff0000u;
  }
}

// 8 lanes write the 128 codes of one column of the transposed tile, 16 each.
__device__ __forceinline__ void store_transposed(const QuantizeArgs& a, const uint32_t* words, int64_t r0, int64_t c0,
                                                 int lane8, int r4) {
  const int n = clamp16(a.M - r0 - 16 * lane8);
  const int64_t left = a.K - c0 - r4;
  uint8_t* const p = a.t_codes + (c0 + r4) * a.t_ldc + r0 + 16 * lane8;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 w = *reinterpret_cast<const uint4*>(&words[tile_word(32 * i + r4, 4 * lane8)]);
    store_codes16(p + 32 * i * a.t_ldc, 32 * i < left ? n : 0, w);
  }
}

// ------------------------------------------ re-blocking in half precision ----
// A code times 2^d is exact in fp16 down to 2^-23 and so takes half the
// instructions of fp32: the codes of a tile are decoded to w = code *
// 2^(scale - top), top the largest scale byte of its rows that hold anything
// but zeros, and the transposed codes are w * 2^(top - new scale), both
// products exact where the code does not round to zero (it does below 2^-10,
// fp16 loses bits only below 2^-24). Tiles whose rows' scales are further
// apart than kSpread, or that hold a NaN or scales near the end of the range,
// and columns that need a factor above 2^15, leave the tile to fp32.
constexpr int kSpread = 14;
constexpr uint32_t kTopLimit = 240;

__device__ __forceinline__ uint32_t e4m3x2_to_h2(uint32_t two_codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two_codes)));
  return h;
}
__device__ __forceinline__ uint32_t e4m3x2_from_h2(uint32_t h) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(h));
  return c;
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// fp16 bits of 2^d, -14 <= d <= 15.
__device__ __forceinline__ uint32_t h_pow2(int d) { return static_cast<uint32_t>(d + 15) << 10; }

// Largest and smallest scale byte of a warp's rows that hold anything but
// zeros, as top << 16 | 255 - low: a maximum over 16-bit halves joins them.
__device__ __forceinline__ uint32_t scale_range(const Fp8Row16 (&r)[4]) {
  uint32_t top = 0, low = 255;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4& c = r[i].codes;
    if (((c.x | c.y | c.z | c.w) & 0x7f7f7f7fu) != 0u || r[i].scale == kScaleNan) {
      top = max(top, r[i].scale);
      low = min(low, r[i].scale);
    }
  }
  return __reduce_max_sync(kFullMask, top) << 16 | (255u - __reduce_min_sync(kFullMask, low));
}

// The factor of a row, 2^(scale - top), in both halves.
__device__ __forceinline__ uint32_t row_factor(uint32_t scale, uint32_t top) {
  const int d = static_cast<int>(scale) - static_cast<int>(top);   // rows of zeros may lie anywhere
  return h_pow2(min(max(d, -kSpread), 0)) * 0x10001u;
}
// Columns 2 p and 2 p + 1 of a row as w (above).
__device__ __forceinline__ uint32_t packed_pair(const Fp8Row16& r, int p, uint32_t factor) {
  const uint32_t c = p < 2 ? r.codes.x : p < 4 ? r.codes.y : p < 6 ? r.codes.z : r.codes.w;
  return mul_h2(e4m3x2_to_h2(p & 1 ? c >> 16 : c & 0xffffu), factor);
}

// The new scale byte of a column whose largest |w| is m, and its factor as
// fp16 bits; false where fp16 cannot carry it.
__device__ __forceinline__ bool column_scale(float m, uint32_t top, uint32_t& byte, uint32_t& factor) {
  const uint32_t bits = __float_as_uint(m);
  byte = kScaleOne;
  factor = h_pow2(0);
  if (bits == 0u) return true;
  if (bits >= 0x7f800000u) return false;
  const int e = static_cast<int>((bits >> 23) + top) - 127;   // of m * 2^(top - 127); subnormal below 1
  byte = fp8_scale_byte(e < 1 ? 1u : static_cast<uint32_t>(e) << 23 | (bits & 0x7fffffu));
  const int d = static_cast<int>(top) - static_cast<int>(byte);
  if (d > 15) return false;
  factor = h_pow2(d);
  return true;
}

// The transpose of codes alone: quantize_tile_kernel's tile and threads. Held to
// 4 CTAs per SM (8192 x 1600 codes: 3: 8.5 us, 4: 8.0, 5 spills: 9.9).
__global__ void __launch_bounds__(kThreads, 4)
transpose_codes_kernel(QuantizeArgs a, Divider per_row) {
  static_assert(kThreads == 256, "eight warps");
  __shared__ __align__(16) uint32_t words[kFp8Block * 32];
  __shared__ uint32_t col_max[kFp8Block];
  __shared__ __align__(16) uint32_t factors[kFp8Block];   // pairs of fp16, or fp32
  __shared__ __align__(16) uint32_t ranges[8];
  __shared__ bool wide_range;   // fp16 cannot carry the tile
  const int64_t rb = per_row.quotient(blockIdx.x);
  const int64_t cb = blockIdx.x - rb * static_cast<int64_t>(per_row.d);
  const int lane8 = threadIdx.x & 7, r4 = threadIdx.x >> 3, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r0 = rb * kFp8Block, c0 = cb * kFp8Block;
  const int64_t row = r0 + 4 * r4, col = c0 + 16 * lane8;
  if (threadIdx.x < kFp8Block) col_max[threadIdx.x] = 0;
  if (threadIdx.x == 0) wide_range = false;
  grid_launch_dependents();
  grid_dependency_wait();

  Fp8Row16 r[4];
  read_tile<Fp8Source, true>(a, rb, cb, row, col, clamp16(a.K - col), clamp4(a.M - row), false, r);
  const uint32_t mine = scale_range(r);
  if (lane == 0) ranges[warp] = mine;
  __syncthreads();

  const uint4 x = reinterpret_cast<const uint4*>(ranges)[0], y = reinterpret_cast<const uint4*>(ranges)[1];
  const uint32_t range = __vmaxu2(__vimax3_u16x2(x.x, x.y, x.z),
                                  __vmaxu2(__vimax3_u16x2(x.w, y.x, y.y), __vmaxu2(y.z, y.w)));
  const uint32_t top = range >> 16, low = 255u - (range & 0xffffu);
  bool packed = top <= kTopLimit && static_cast<int>(top) - static_cast<int>(low) <= kSpread;
  uint32_t rf[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) rf[i] = row_factor(r[i].scale, top);
  if (packed) {
    uint32_t m[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = packed_pair(r[i], p, rf[i]);
      m[p] = max_abs2(w[0], w[1], w[2], w[3]);
    }
    put_pairs(m, words);
    __syncthreads();
    uint32_t b0 = 0, b1 = 0;
    if (threadIdx.x < kPairs) {
      const uint32_t all = join_pairs(words, threadIdx.x);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&all));
      uint32_t f0, f1;
      const bool fits0 = column_scale(f.x, top, b0, f0), fits1 = column_scale(f.y, top, b1, f1);
      if (!fits0 || !fits1) wide_range = true;
      factors[threadIdx.x] = f0 | f1 << 16;
    }
    __syncthreads();
    packed = !wide_range;
    if (packed && threadIdx.x < kPairs) {
      const int64_t c = c0 + 2 * threadIdx.x;
      if (c < a.K) a.t_scales[c * a.t_lds + rb] = static_cast<uint8_t>(b0);
      if (c + 1 < a.K) a.t_scales[(c + 1) * a.t_lds + rb] = static_cast<uint8_t>(b1);
    }
  }
  if (packed) {
    const uint4 g = *reinterpret_cast<const uint4*>(&factors[8 * lane8]);
    const uint4 h = *reinterpret_cast<const uint4*>(&factors[8 * lane8 + 4]);
    const uint32_t f[8] = {g.x, g.y, g.z, g.w, h.x, h.y, h.z, h.w};
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      uint32_t q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = e4m3x2_from_h2(mul_h2(packed_pair(r[i], p, rf[i]), f[p]));
      const uint32_t q01 = __byte_perm(q[0], q[1], 0x5410), q23 = __byte_perm(q[2], q[3], 0x5410);
      const int c = 16 * lane8 + 2 * p;
      words[tile_word(c, r4)] = __byte_perm(q01, q23, 0x6420);
      words[tile_word(c + 1, r4)] = __byte_perm(q01, q23, 0x7531);
    }
  } else {   // in fp32, four columns at a time
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      float v[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) values4<Fp8Source>(r[i], q, v[i]);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        atomicMax(&col_max[16 * lane8 + 4 * q + e],
                  __float_as_uint(amax3(amax3(0.0f, v[0][e], v[1][e]), v[2][e], v[3][e])));
    }
    __syncthreads();
    if (threadIdx.x < kFp8Block) {
      const uint32_t b = fp8_scale_byte(col_max[threadIdx.x]);
      factors[threadIdx.x] = __float_as_uint(fp8_inverse_scale(b));
      if (c0 + threadIdx.x < a.K) a.t_scales[(c0 + threadIdx.x) * a.t_lds + rb] = static_cast<uint8_t>(b);
    }
    __syncthreads();
#pragma unroll 1
    for (int q = 0; q < 4; ++q) {
      float v[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) values4<Fp8Source>(r[i], q, v[i]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = 16 * lane8 + 4 * q + e;
        const float inv = __uint_as_float(factors[c]);
        words[tile_word(c, r4)] = e4m3x4_from_f32(v[0][e] * inv, v[1][e] * inv, v[2][e] * inv, v[3][e] * inv);
      }
    }
  }
  __syncthreads();
  store_transposed(a, words, r0, c0, lane8, r4);
}

// CTAs per SM that the tile kernel's registers are held to, with 2, 3 and 4 (and
// the bytes that the aligned form with the transpose then spills):
//   16-bit rows and transpose, 8192 x 4096     27.4 (0), 27.7 (0), 25.5 us (8)
//   16-bit 128 x 128 tiles, 16384 x 4096       53.2 (0), 46.3 (108), 55.8 us (240)
//   codes, rows and transpose, 8192 x 4096     49.8 (0), 43.9 (92), 49.4 us (232)
//   codes, 128 x 128 tiles, 8192 x 4096        43.2 (0), 38.5 (84), 43.5 us (220)
//   f32 rows and transpose, 8192 x 4096        41.4 (0), 41.8 (156), 76.0 us (760)
//   f32 128 x 128 tiles, 16384 x 4096          62.3 (0), 61.1 (100), 125 us (864)
template <typename T, bool TILE>
constexpr int tile_ctas() {
  return std::is_same<T, float>::value ? 2 : std::is_same<T, Fp8Source>::value || TILE ? 3 : 4;
}

template <typename T, bool VEC, bool TILE, bool TRANSPOSE>
__global__ void __launch_bounds__(kThreads, (tile_ctas<T, TILE>()))
quantize_tile_kernel(QuantizeArgs a, Divider per_row, bool wide) {
  __shared__ __align__(16) uint32_t words[TRANSPOSE ? kFp8Block * 32 : 4];
  __shared__ uint32_t col_max[kFp8Block];   // TILE: entry 0 is the tile's
  __shared__ __align__(16) float col_inv[kFp8Block];
  const int64_t rb = per_row.quotient(blockIdx.x);
  const int64_t cb = blockIdx.x - rb * static_cast<int64_t>(per_row.d);
  const int lane8 = threadIdx.x & 7, r4 = threadIdx.x >> 3;
  const int64_t r0 = rb * kFp8Block, c0 = cb * kFp8Block;
  const int64_t row = r0 + 4 * r4, col = c0 + 16 * lane8;
  if (threadIdx.x < kFp8Block) col_max[threadIdx.x] = 0;
  grid_launch_dependents();
  grid_dependency_wait();

  typename RowOf<T>::type r[4];
  const int n = clamp16(a.K - col), rows = clamp4(a.M - row);
  read_tile<T, VEC>(a, rb, cb, row, col, n, rows, wide, r);
  __syncthreads();

  if (TILE) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[16];
      values16<T>(r[i], v);
      m = amax3(m, amax_of(v), 0.0f);
    }
    const uint32_t top = group_umax<32>(m);
    if ((threadIdx.x & 31) == 0) atomicMax(&col_max[0], top);
  } else {
    if (a.codes) {
      uint8_t* const codes = a.codes + row * a.ldc + col;
      uint8_t* const scales = a.scales + row * a.lds + cb;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v[16];
        values16<T>(r[i], v);
        quantize16(v, i < rows ? n : 0, codes + i * a.ldc, scales + i * a.lds, lane8);
      }
    }
    if constexpr (sizeof(T) == 2) {
      uint32_t m[8];
#pragma unroll
      for (int p = 0; p < 8; ++p) m[p] = max_abs2(r[0].w[p], r[1].w[p], r[2].w[p], r[3].w[p]);
      put_pairs(m, words);
    } else {
      fold_columns<T>(r, col_max, lane8);
    }
  }
  __syncthreads();
  if (TILE) {
    const uint32_t b = fp8_scale_byte(col_max[0]);
    const float inv = fp8_inverse_scale(b);
    if (threadIdx.x == 0) {
      if (a.codes) a.scales[rb * a.lds + cb] = static_cast<uint8_t>(b);
      if (TRANSPOSE) a.t_scales[cb * a.t_lds + rb] = static_cast<uint8_t>(b);
    }
    if (a.codes) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v[16];
        values16<T>(r[i], v);
        store_codes16(a.codes + (row + i) * a.ldc + col, i < rows ? n : 0, codes16(v, inv));
      }
    }
  }
  if constexpr (TRANSPOSE) {
    float tile_inv = 0.0f;
    if (TILE) {
      tile_inv = fp8_inverse_scale(fp8_scale_byte(col_max[0]));
    } else {
      const auto set = [&](int c, uint32_t amax) {
        const uint32_t b = fp8_scale_byte(amax);
        col_inv[c] = fp8_inverse_scale(b);
        if (c0 + c < a.K) a.t_scales[(c0 + c) * a.t_lds + rb] = static_cast<uint8_t>(b);
      };
      if constexpr (sizeof(T) == 2) {
        if (threadIdx.x < kPairs) {
          uint32_t b[2];
          pair_bits<T>(join_pairs(words, threadIdx.x), b);
          set(2 * threadIdx.x, b[0]);
          set(2 * threadIdx.x + 1, b[1]);
        }
      } else if (threadIdx.x < kFp8Block) {
        set(threadIdx.x, col_max[threadIdx.x]);
      }
      __syncthreads();
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) values4<T>(r[i], q, v[i]);
      float inv4[4];
      if (!TILE) *reinterpret_cast<float4*>(inv4) = *reinterpret_cast<const float4*>(&col_inv[16 * lane8 + 4 * q]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = 16 * lane8 + 4 * q + e;
        const float inv = TILE ? tile_inv : inv4[e];
        words[tile_word(c, r4)] = e4m3x4_from_f32(v[0][e] * inv, v[1][e] * inv, v[2][e] * inv, v[3][e] * inv);
      }
    }
    __syncthreads();
    store_transposed(a, words, r0, c0, lane8, r4);
  }
}

template <typename T, bool VEC>
cudaError_t launch_t(const QuantizeArgs& a, bool wide, cudaStream_t st) {
  if (!a.t_codes && a.tile == 1) {
    const Divider per_row((a.K + 4 * kFp8Block - 1) / (4 * kFp8Block));
    const int64_t warps = a.M * static_cast<int64_t>(per_row.d);
    return launch_dependent(quantize_rows_kernel<T, VEC>,
                            dim3(static_cast<unsigned>((warps + kThreads / 32 - 1) / (kThreads / 32))), kThreads, 0,
                            st, a, per_row, wide);
  }
  const Divider per_row((a.K + kFp8Block - 1) / kFp8Block);
  const dim3 grid(static_cast<unsigned>(per_row.d * ((a.M + kFp8Block - 1) / kFp8Block)));
  if constexpr (std::is_same<T, Fp8Source>::value)
    if (a.tile == 1 && !a.codes) return launch_dependent(transpose_codes_kernel, grid, kThreads, 0, st, a, per_row);
  auto k = a.tile == 1    ? quantize_tile_kernel<T, VEC, false, true>
           : a.t_codes ? quantize_tile_kernel<T, VEC, true, true>
                       : quantize_tile_kernel<T, VEC, true, false>;
  return launch_dependent(k, grid, kThreads, 0, st, a, per_row, wide);
}

}  // namespace

cudaError_t launch_quantize(const QuantizeArgs& a, int dtype, int vec, cudaStream_t st) {
  if (a.x_scales) return launch_t<Fp8Source, true>(a, false, st);
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    return vec ? launch_t<T, true>(a, vec == kVec32, st) : launch_t<T, false>(a, false, st);
  });
}

}  // namespace taco
