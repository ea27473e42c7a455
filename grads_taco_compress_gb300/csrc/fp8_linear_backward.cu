// The gradient at a layer's product, d = dy act'(pre), from the 8-bit checkpoint
// of pre: its FP8 rows (what the input's gradient reads), its FP8 transpose (what
// the weight's reads) and the bias's gradient, the sum of its rows, from one read
// of dy and of the checkpoint. d itself is never written: it is quantised from
// fp32, rounded once.
//
// A CTA takes a 128 x 128 tile, each of 512 threads 4 consecutive rows of 8
// columns, whose d stay in registers (with 256 threads and 16 columns they take
// twice the registers, and half the warps could not hide the latencies of the
// tile's phases). Largest magnitudes and sums of the columns meet in shared
// memory; the transposed codes go through it, 4 rows of a column to a word, so that
// they leave as whole 128-byte rows. Tiles write their column sums; a second kernel
// adds them in the order of the rows.
//
// Measured, 8192 x 16384 bf16 (a plain copy: 6.78 TB/s): tanh GELU 154-156 us, 4.4 TB/s,
// 62% of the issue slots at 27 instructions an element; without an activation 113
// us, 4.8 TB/s; f32 188 us, 5.0 TB/s.

#include "fp8_activation.cuh"

namespace taco {

namespace {

constexpr int kThreads = 512;
constexpr int kCols = 8;                        // of a thread
constexpr int kLanes = kFp8Block / kCols;       // that share a row's block

// Eight consecutive elements of a row, as they lie in memory.
template <typename T>
struct Row8 {
  static constexpr int kWords = 2 * static_cast<int>(sizeof(T));
  uint32_t w[kWords];
};
// n (0 .. 8) of them exist, the others read as zero. VEC: p is 16-byte aligned.
template <typename T, bool VEC>
__device__ __forceinline__ Row8<T> load8(const T* p, int n) {
  Row8<T> r;
  if (VEC && n == kCols) {
#pragma unroll
    for (int i = 0; i < Row8<T>::kWords / 4; ++i)
      asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(r.w[4 * i]), "=r"(r.w[4 * i + 1]), "=r"(r.w[4 * i + 2]), "=r"(r.w[4 * i + 3])
                   : "l"(reinterpret_cast<const char*>(p) + 16 * i));
  } else if constexpr (VEC) {   // the end of a row
    alignas(16) T v[kCols];
#pragma unroll
    for (int i = 0; i < kCols; ++i) v[i] = i < n ? p[i] : from_f32<T>(0.0f);
    memcpy(r.w, v, sizeof(v));
  } else {
    load_shifted(p, n, r.w);
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void unpack8(const Row8<T>& r, float (&v)[kCols]) {
#pragma unroll
  for (int i = 0; i < kCols / 2; ++i) {
    if constexpr (std::is_same<T, float>::value) {
      v[2 * i] = __uint_as_float(r.w[2 * i]);
      v[2 * i + 1] = __uint_as_float(r.w[2 * i + 1]);
    } else if constexpr (std::is_same<T, __half>::value) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    } else {
      v[2 * i] = bf16_lo(r.w[i]);
      v[2 * i + 1] = bf16_hi(r.w[i]);
    }
  }
}
__device__ __forceinline__ uint2 load_codes8(const uint8_t* p, int n) {
  if (n == kCols) {
    uint2 c;
    asm volatile("ld.global.L1::no_allocate.v2.b32 {%0,%1}, [%2];" : "=r"(c.x), "=r"(c.y) : "l"(p));
    return c;
  }
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < kCols; ++i)
    if (i < n) w[i >> 2] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store_codes8(uint8_t* p, int n, uint2 c) {
  if (n == kCols) {
    *reinterpret_cast<uint2*>(p) = c;
  } else {
#pragma unroll
    for (int i = 0; i < kCols; ++i)
      if (i < n) p[i] = static_cast<uint8_t>((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
  }
}
// Codes that leave for good, kept out of L1 (1% of the kernel's time).
__device__ __forceinline__ void store_past_l1(uint8_t* p, uint2 c) {
  asm volatile("st.global.L1::no_allocate.v2.b32 [%2], {%0,%1};" :: "r"(c.x), "r"(c.y), "l"(p) : "memory");
}
__device__ __forceinline__ void store_past_l1(uint8_t* p, uint4 c) {
  asm volatile("st.global.L1::no_allocate.v4.b32 [%4], {%0,%1,%2,%3};"
               :: "r"(c.x), "r"(c.y), "r"(c.z), "r"(c.w), "l"(p) : "memory");
}
__device__ __forceinline__ uint32_t codes4(f2 a, f2 b, float inv) {
  const f2 x = mul2(a, both(inv)), y = mul2(b, both(inv));
  return e4m3x4_from_f32(x.x, x.y, y.x, y.y);
}

// Word of the transposed tile that holds rows 4 r4 .. 4 r4 + 3 of column c: 32
// words a column, in the order r4 ^ 2 (c / 8), so that a warp, which writes one
// column of each of its 16 lane groups at a time, in two words, meets 32 banks.
__device__ __forceinline__ int word_of_tile(int c, int r4) { return c * 32 + (r4 ^ (2 * (c / kCols))); }

struct TileShared {
  uint4 words[kFp8Block * 32 / 4];              // the transposed codes
  uint4 tops[kThreads / 32][kFp8Block / 4];     // of a warp's rows, by column
  float4 sums[kThreads / 32][kFp8Block / 4];
  float4 inv[kFp8Block / 4];
};
// One tile. FULL: all of it exists, and nothing is checked.
template <typename T, bool VEC, bool FULL>
__device__ __forceinline__ void backward_tile(const LinearBackwardArgs& a, int64_t rb, int64_t cb, TileShared& sh) {
  constexpr int kWarps = kThreads / 32;
  const int group = threadIdx.x & (kLanes - 1), r4 = threadIdx.x / kLanes, lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int64_t r0 = rb * kFp8Block, c0 = cb * kFp8Block;
  const int64_t row = r0 + 4 * r4, col = c0 + kCols * group;
  const int n = FULL ? kCols : static_cast<int>(a.N - col < 0 ? 0 : a.N - col < kCols ? a.N - col : kCols);
  const int rows = FULL ? 4 : static_cast<int>(a.M - row < 0 ? 0 : a.M - row < 4 ? a.M - row : 4);

  float d[4][kCols];
  {
    Row8<T> g[4];
    uint2 codes[4];
    uint32_t scale[4];
    const T* const p = static_cast<const T*>(a.dy) + row * a.lddy + col;
#pragma unroll
    for (int i = 0; i < 4; ++i) g[i] = load8<T, VEC>(p + i * a.lddy, i < rows ? n : 0);
    if (a.act != TACO_ACT_NONE) {
      const uint8_t* const k = a.k_codes + row * a.k_ld + col;
      const uint8_t* const s = a.k_scales + row * a.k_lds + cb;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool any = i < rows && n > 0;
        codes[i] = load_codes8(k + i * a.k_ld, any ? n : 0);
        scale[i] = any ? s[i * a.k_lds] : kScaleOne;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack8<T>(g[i], d[i]);
    with_act(a.act, [&](auto kind) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float x[kCols];
        const float s = fp8_scale(scale[i]);
        decode4(codes[i].x, s, x);
        decode4(codes[i].y, s, x + 4);
        // beyond this values no slope's arithmetic holds as it is
        if (scale[i] > kScaleOne + kSlopeBinades) limit_for_slope<decltype(kind)::value>(x);
#pragma unroll
        for (int e = 0; e < kCols; e += 2) {
          const f2 y = mul2(f2{d[i][e], d[i][e + 1]}, slope2<decltype(kind)::value>(f2{x[e], x[e + 1]}));
          d[i][e] = y.x;
          d[i][e + 1] = y.y;
        }
        if (!FULL && scale[i] == kScaleNan) {   // which must not reach columns that do not exist
#pragma unroll
          for (int e = 0; e < kCols; ++e)
            if (e >= n) d[i][e] = 0.0f;
        }
      }
    });
  }
  if (a.codes) {
    // The largest magnitudes of the 4 rows over their 16 lanes: two exchanges hand
    // half of a lane's rows to the partner, so that lane l joins row l / 4 % 4 alone
    // and forms one scale.
    uint32_t m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = __float_as_uint(amax_of(d[i]));
    const bool b8 = lane & 8, b4 = lane & 4;
    const uint32_t o0 = __shfl_xor_sync(kFullMask, b8 ? m[0] : m[2], 8);
    const uint32_t o1 = __shfl_xor_sync(kFullMask, b8 ? m[1] : m[3], 8);
    const uint32_t k0 = max(b8 ? m[2] : m[0], o0), k1 = max(b8 ? m[3] : m[1], o1);
    uint32_t top = max(b4 ? k1 : k0, __shfl_xor_sync(kFullMask, b4 ? k0 : k1, 4));
    top = max(top, __shfl_xor_sync(kFullMask, top, 2));
    top = max(top, __shfl_xor_sync(kFullMask, top, 1));
    const uint32_t b = fp8_scale_byte(top);
    const float inv = fp8_inverse_scale(b);
    const int mine = (lane >> 2) & 3;
    if ((lane & 3) == 0 && (FULL || (row + mine < a.M)))
      a.scales[(row + mine) * a.lds + cb] = static_cast<uint8_t>(b);
    uint8_t* const q = a.codes + row * a.ldc + col;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = __shfl_sync(kFullMask, inv, (lane & 16) + 4 * i);
      const uint2 c = make_uint2(codes4(f2{d[i][0], d[i][1]}, f2{d[i][2], d[i][3]}, f),
                                 codes4(f2{d[i][4], d[i][5]}, f2{d[i][6], d[i][7]}, f));
      if (FULL)
        store_past_l1(q + i * a.ldc, c);
      else
        store_codes8(q + i * a.ldc, i < rows ? n : 0, c);
    }
  }
  {
    // The columns of the warp's two lanes that hold other rows of them: each hands
    // half of its columns to the other and keeps the other half.
    uint32_t top[kCols];
    float sum[kCols];
#pragma unroll
    for (int e = 0; e < kCols; ++e) {
      top[e] = __float_as_uint(amax3(amax3(0.0f, d[0][e], d[1][e]), d[2][e], d[3][e]));
    }
#pragma unroll
    for (int e = 0; e < kCols; e += 2) {
      const auto pair = [&](int r) { return f2{d[r][e], d[r][e + 1]}; };
      const f2 s = add2(add2(pair(0), pair(1)), add2(pair(2), pair(3)));
      sum[e] = s.x;
      sum[e + 1] = s.y;
    }
    const bool high = lane & 16;
    uint32_t t[4];
    float u[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t other = __shfl_xor_sync(kFullMask, high ? top[e] : top[e + 4], 16);
      t[e] = max(high ? top[e + 4] : top[e], other);
      const float more = __shfl_xor_sync(kFullMask, high ? sum[e] : sum[e + 4], 16);
      u[e] = (high ? sum[e + 4] : sum[e]) + more;
    }
    const int c = kCols * group + (high ? 4 : 0);
    sh.tops[warp][c / 4] = make_uint4(t[0], t[1], t[2], t[3]);
    sh.sums[warp][c / 4] = make_float4(u[0], u[1], u[2], u[3]);
  }
  __syncthreads();
  if (threadIdx.x < 2 * kFp8Block) {   // 128 threads join the maxima, 128 the sums
    const int c = threadIdx.x & (kFp8Block - 1);
    const bool exists = FULL || c0 + c < a.N;
    if (threadIdx.x < kFp8Block) {
      uint32_t top = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = max(top, reinterpret_cast<const uint32_t*>(sh.tops[w])[c]);
      const uint32_t b = fp8_scale_byte(top);
      reinterpret_cast<float*>(sh.inv)[c] = fp8_inverse_scale(b);
      if (exists && a.t_codes) a.t_scales[(c0 + c) * a.t_lds + rb] = static_cast<uint8_t>(b);
    } else if (a.sums) {
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) sum += reinterpret_cast<const float*>(sh.sums[w])[c];
      if (exists) a.sums[rb * a.N + c0 + c] = sum;
    }
  }
  if (!a.t_codes) return;
  __syncthreads();
  uint32_t* const words = reinterpret_cast<uint32_t*>(sh.words);
#pragma unroll
  for (int e = 0; e < kCols; e += 4) {
    const float4 inv = sh.inv[2 * group + e / 4];
#pragma unroll
    for (int j = 0; j < 4; j += 2) {   // columns in pairs, which lie in pairs of registers
      const f2 f = j ? f2{inv.z, inv.w} : f2{inv.x, inv.y};
      f2 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = mul2(f2{d[i][e + j], d[i][e + j + 1]}, f);
      words[word_of_tile(kCols * group + e + j, r4)] = e4m3x4_from_f32(x[0].x, x[1].x, x[2].x, x[3].x);
      words[word_of_tile(kCols * group + e + j + 1, r4)] = e4m3x4_from_f32(x[0].y, x[1].y, x[2].y, x[3].y);
    }
  }
  __syncthreads();
  // 8 lanes write the 128 codes of a column, 16 each
  const int lane8 = threadIdx.x & 7;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = (threadIdx.x >> 3) + 64 * i;
    const int at = word_of_tile(c, 4 * lane8);   // two words, the other two at ^ 2
    const uint2 lo = *reinterpret_cast<const uint2*>(&words[at]), hi = *reinterpret_cast<const uint2*>(&words[at ^ 2]);
    const uint4 w = make_uint4(lo.x, lo.y, hi.x, hi.y);
    uint8_t* const to = a.t_codes + (c0 + c) * a.t_ldc + r0 + 16 * lane8;
    if (FULL)
      store_past_l1(to, w);
    else if (c0 + c < a.N)
      store_codes16(to, clamp16(a.M - r0 - 16 * lane8), w);
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) linear_backward_kernel(LinearBackwardArgs a, Divider per_row) {
  __shared__ TileShared sh;
  const int64_t rb = per_row.quotient(blockIdx.x);
  const int64_t cb = blockIdx.x - rb * static_cast<int64_t>(per_row.d);
  grid_launch_dependents();
  grid_dependency_wait();
  if (VEC && (rb + 1) * kFp8Block <= a.M && (cb + 1) * kFp8Block <= a.N)
    backward_tile<T, VEC, true>(a, rb, cb, sh);
  else
    backward_tile<T, VEC, false>(a, rb, cb, sh);
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
    return launch_dependent(vec ? linear_backward_kernel<T, true> : linear_backward_kernel<T, false>, grid, kThreads, 0,
                            st, a, per_row);
  });
  if (e != cudaSuccess || !db || tiles == 1) return e;
  return launch_dependent(column_sums_kernel, dim3(static_cast<unsigned>((a.N + 31) / 32)), 256, 0, st,
                          static_cast<const float*>(workspace), tiles, a.N, db);
}

}  // namespace taco
