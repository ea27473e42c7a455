// Device helpers of the FP8 block tensors (fp8_quantize.cu, fp8_norm.cu,
// fp8_swiglu.cu, fp8_matmul.cu).
//
// An FP8 block tensor holds E4M3 codes and, per row and 128 columns (or per
// 128 x 128 tile), one E8M0 scale byte b that stands for 2^(b - 127). A scale
// that is a power of two multiplies a code exactly, so a value decoded to
// fp32 carries no rounding of its own, and the byte is what the block-scaled
// tensor-core instructions read.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <type_traits>

#include "taco_device.cuh"
#include "taco_launch.h"

namespace taco {

constexpr int kFp8Block = 128;          // columns per scale
constexpr uint32_t kScaleNan = 255;     // E8M0 NaN
constexpr uint32_t kScaleOne = 127;     // 2^0

// Scale byte of a block whose largest magnitude has the fp32 bits `amax`
// (sign cleared; integer order is the order of the values, with infinity and
// NaN above every finite one). The scale is the smallest power of two with
// amax / scale <= 448 = 1.75 * 2^8, not below 2^-126, so that it and its
// reciprocal are normal fp32 numbers; 1 for an all-zero block. A block that
// holds an infinity or a NaN has no finite scale: its byte is the E8M0 NaN,
// which decodes every element of the block, and every product with it, to NaN.
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t amax) {
  if (amax >= 0x7f800000u) return kScaleNan;
  if (amax == 0u) return kScaleOne;
  const int b = static_cast<int>(amax >> 23) - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(b < 1 ? 1 : b);
}
// 2^(127 - b), the factor that takes a value to its code (bytes 1 .. 247, as
// fp8_scale_byte gives them; for the NaN byte any finite factor will do).
__device__ __forceinline__ float fp8_inverse_scale(uint32_t b) {
  return __uint_as_float((b >= 248u ? 127u : 254u - b) << 23);
}
// 2^(b - 127) of any byte: 0 is 2^-127, a subnormal fp32 number, 255 is NaN.
__device__ __forceinline__ float fp8_scale(uint32_t b) {
  if (b == kScaleNan) return __uint_as_float(0x7fffffffu);
  return __uint_as_float(b == 0u ? 0x400000u : b << 23);
}

// max(|a|, |b|, |c|), NaN if any of them is.
__device__ __forceinline__ float amax3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Largest magnitude of N values (N even), NaN if any is.
template <int N>
__device__ __forceinline__ float amax_of(const float (&v)[N]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < N; i += 2) m = amax3(m, v[i], v[i + 1]);
  return m;
}
// Largest over the LANES consecutive lanes of an aligned group, as bits.
template <int LANES>
__device__ __forceinline__ uint32_t group_umax(float v) {
  uint32_t b = __float_as_uint(v);
#pragma unroll
  for (int m = 1; m < LANES; m <<= 1) b = max(b, __shfl_xor_sync(kFullMask, b, m));
  return b;
}

// Lanes that share a block of 128 columns, 16 columns each.
constexpr int kBlockLanes = 8;

// Sixteen codes of v * inv, element 0 in the low byte.
__device__ __forceinline__ uint4 codes16(const float (&v)[16], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f2 s{inv, inv};
    const f2 a = mul2(f2{v[4 * i], v[4 * i + 1]}, s), b = mul2(f2{v[4 * i + 2], v[4 * i + 3]}, s);
    w[i] = e4m3x4_from_f32(a.x, a.y, b.x, b.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Four codes -> fp32 values times s (a power of two: exact).
__device__ __forceinline__ void decode4(uint32_t w, float s, float* v) {
  const f2 ss{s, s}, a = mul2(e4m3x2_to_f2(w & 0xffffu), ss), b = mul2(e4m3x2_to_f2(w >> 16), ss);
  v[0] = a.x;
  v[1] = a.y;
  v[2] = b.x;
  v[3] = b.y;
}
__device__ __forceinline__ void decode16(uint4 c, float s, float (&v)[16]) {
  decode4(c.x, s, v);
  decode4(c.y, s, v + 4);
  decode4(c.z, s, v + 8);
  decode4(c.w, s, v + 12);
}

// ------------------------------------------------------- element types ----
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ float from_f32(float v) { return v; }

// Sixteen consecutive elements of a row, as they lie in memory.
template <typename T>
struct Row16 {
  uint32_t w[4 * sizeof(T)];
};
template <typename T>
__device__ __forceinline__ void unpack(const Row16<T>& r, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
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
template <typename T>
__device__ __forceinline__ Row16<T> pack(const float (&v)[16]) {
  Row16<T> r;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (std::is_same<T, float>::value) {
      r.w[2 * i] = __float_as_uint(v[2 * i]);
      r.w[2 * i + 1] = __float_as_uint(v[2 * i + 1]);
    } else if constexpr (std::is_same<T, __half>::value) {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      r.w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      r.w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    }
  }
  return r;
}
// Eight 32-bit words to and from global memory: one 32-byte access where p
// allows it (wide), else two of 16 bytes. Streamed data is kept out of L1.
__device__ __forceinline__ void load_words8(const void* p, bool wide, uint32_t* w) {
  if (wide) {
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      asm volatile("ld.global.v4.b32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                   : "l"(static_cast<const char*>(p) + 16 * i));
  }
}
__device__ __forceinline__ void store_words8(void* p, bool wide, const uint32_t* w) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};"
                 :: "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]), "l"(p)
                 : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<uint4*>(static_cast<char*>(p) + 16 * i) =
          make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
}
// ------------------------------------------- rows that start anywhere ----
// The W words of n consecutive elements (the others become zero) that start s
// bytes, a multiple of their size below 16, into the words v.
template <typename T, int W>
__device__ __forceinline__ void shift_words(uint32_t (&v)[W + 4], uint32_t s, int n, uint32_t (&w)[W]) {
  if (s & 8) {
#pragma unroll
    for (int i = 0; i < W + 2; ++i) v[i] = v[i + 2];
  }
  if (s & 4) {
#pragma unroll
    for (int i = 0; i < W + 1; ++i) v[i] = v[i + 1];
  }
#pragma unroll
  for (int i = 0; i < W; ++i) {
    w[i] = sizeof(T) == 4 ? v[i] : __funnelshift_r(v[i], v[i + 1], 8 * (s & 2));
    // elements beyond the row are zero
    if (sizeof(T) == 4) {
      if (i >= n) w[i] = 0u;
    } else {
      if (2 * i >= n) w[i] = 0u;
      else if (2 * i + 1 >= n) w[i] &= 0xffffu;
    }
  }
}
// The W words of a lane's consecutive elements at p, of which n exist (the
// others read as zero), through aligned 16-byte loads and a shift. Every load
// holds at least one byte of an element that exists.
template <typename T, int W>
__device__ __forceinline__ void load_shifted(const T* p, int n, uint32_t (&w)[W]) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const uint32_t s = static_cast<uint32_t>(at & 15);
  const uint4* from = reinterpret_cast<const uint4*>(at - s);
  const int bytes = n ? static_cast<int>(s) + n * static_cast<int>(sizeof(T)) : 0;
  uint32_t v[W + 4];
#pragma unroll
  for (int j = 0; j <= W / 4; ++j) {
    uint4 q = make_uint4(0, 0, 0, 0);
    if (16 * j < bytes) q = from[j];
    v[4 * j] = q.x;
    v[4 * j + 1] = q.y;
    v[4 * j + 2] = q.z;
    v[4 * j + 3] = q.w;
  }
  shift_words<T>(v, s, n, w);
}

// Writes the W words of each lane of a converged warp, whose lanes hold
// consecutive elements (n of a lane's exist; a lane after a partial one has
// none): whole aligned 16-byte pieces, each by the lane in whose place it
// starts, with the end of the lane before; what a piece at either end of the
// warp or of the row lacks goes element by element.
template <typename T, int W>
__device__ __forceinline__ void store_shifted(T* p, int n, const uint32_t (&w)[W]) {
  constexpr int kEs = sizeof(T), kPer = 16 / kEs, kElems = 4 * W / kEs;
  const int lane = threadIdx.x & 31;
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const uint32_t s = static_cast<uint32_t>(at & 15);   // the same in every lane
  const int before = static_cast<int>(s) / kEs;        // elements of the first piece that are the last lane's
  uint32_t v[W + 8];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __shfl_up_sync(kFullMask, w[W - 4 + i], 1);
  const int n_before = __shfl_up_sync(kFullMask, n, 1);
#pragma unroll
  for (int i = 0; i < W; ++i) v[4 + i] = w[i];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[4 + W + i] = 0u;
  // shift by the 16 - s bytes in front of the first piece
  const uint32_t d = 16u - s;
  if (d & 16) {
#pragma unroll
    for (int i = 0; i < W + 4; ++i) v[i] = v[i + 4];
  }
  if (d & 8) {
#pragma unroll
    for (int i = 0; i < W + 2; ++i) v[i] = v[i + 2];
  }
  if (d & 4) {
#pragma unroll
    for (int i = 0; i < W + 1; ++i) v[i] = v[i + 1];
  }
  if (kEs == 2) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = __funnelshift_r(v[i], v[i + 1], 8 * (d & 2));
  }
  T* first = reinterpret_cast<T*>(at - s);
#pragma unroll
  for (int j = 0; j < W / 4; ++j) {
    const auto exists = [&](int e) {   // e: element of the pieces, counted from the first one's start
      const int own = e - before;
      return own >= 0 ? own < n : lane > 0 && kElems + own < n_before;
    };
    if (exists(j * kPer) && exists(j * kPer + kPer - 1)) {
      *reinterpret_cast<uint4*>(first + j * kPer) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    } else {
#pragma unroll
      for (int k = 0; k < kPer; ++k)
        if (exists(j * kPer + k)) {
          const uint32_t word = v[4 * j + k * kEs / 4];
          if (kEs == 4)
            reinterpret_cast<uint32_t*>(first)[j * kPer + k] = word;
          else
            reinterpret_cast<uint16_t*>(first)[j * kPer + k] = static_cast<uint16_t>(word >> (16 * (k & 1)));
        }
    }
  }
  if (lane == 31) {   // the end of the last lane starts no piece of the warp
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int e = kElems - kPer + k;
      if (e >= kElems - before && e < n) {
        const uint32_t word = w[e * kEs / 4];
        if (kEs == 4)
          reinterpret_cast<uint32_t*>(p)[e] = word;
        else
          reinterpret_cast<uint16_t*>(p)[e] = static_cast<uint16_t>(word >> (16 * (e & 1)));
      }
    }
  }
}

// The elements of 16 consecutive columns, of which n (0 .. 16) exist; the
// others read as zero. VEC: p is 16-byte aligned, and 32-byte aligned if wide;
// without it a store takes whole warps on consecutive columns.
template <typename T, bool VEC>
__device__ __forceinline__ Row16<T> load16(const T* p, int n, bool wide) {
  Row16<T> r;
  if (VEC && n == 16) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
      load_words8(p + 8 * i * (4 / sizeof(T)), wide, r.w + 8 * i);
  } else if constexpr (VEC) {   // the end of a row
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = i < n ? to_f32(p[i]) : 0.0f;
    r = pack<T>(v);
  } else {
    load_shifted(p, n, r.w);
  }
  return r;
}
template <typename T, bool VEC>
__device__ __forceinline__ void store16(T* p, int n, bool wide, const Row16<T>& r) {
  if (VEC && n == 16) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
      store_words8(p + 8 * i * (4 / sizeof(T)), wide, r.w + 8 * i);
  } else if constexpr (VEC) {
    float v[16];
    unpack<T>(r, v);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) p[i] = from_f32<T>(v[i]);
  } else {
    store_shifted(p, n, r.w);
  }
}
// Codes of 16 consecutive columns: rows of codes start at multiples of 16
// bytes, so a full group is one access; a partial one goes byte by byte and
// leaves what lies behind the row alone.
__device__ __forceinline__ void store_codes16(uint8_t* p, int n, uint4 c) {
  if (n == 16) {
    *reinterpret_cast<uint4*>(p) = c;
  } else {
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) p[i] = static_cast<uint8_t>(w[i >> 2] >> (8 * (i & 3)));
  }
}
__device__ __forceinline__ uint4 load_codes16(const uint8_t* p, int n) {
  if (n == 16) {
    uint4 c;
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(c.x), "=r"(c.y), "=r"(c.z), "=r"(c.w) : "l"(p));
    return c;
  }
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (i < n) w[i >> 2] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 consecutive entries of a vector of any element type, kept in L1.
template <typename T, bool VEC>
__device__ __forceinline__ void load_vector16(const T* p, int n, float (&v)[16]) {
  if (VEC && n == 16) {
    Row16<T> r;
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)); ++i)
      *reinterpret_cast<uint4*>(r.w + 4 * i) = *reinterpret_cast<const uint4*>(p + 4 * i * (4 / sizeof(T)));
    unpack<T>(r, v);
  } else if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = i < n ? to_f32(p[i]) : 0.0f;
  } else {
    Row16<T> r;
    load_shifted(p, n, r.w);
    unpack<T>(r, v);
  }
}
template <bool VEC>
__device__ __forceinline__ void load_weight16(const void* w, int dtype, int64_t col, int n, float (&v)[16]) {
  if (dtype == TACO_DTYPE_F32)
    load_vector16<float, VEC>(static_cast<const float*>(w) + col, n, v);
  else if (dtype == TACO_DTYPE_BF16)
    load_vector16<__nv_bfloat16, VEC>(static_cast<const __nv_bfloat16*>(w) + col, n, v);
  else
    load_vector16<__half, VEC>(static_cast<const __half*>(w) + col, n, v);
}

__device__ __forceinline__ int clamp16(int64_t left) {
  return left < 0 ? 0 : (left > 16 ? 16 : static_cast<int>(left));
}

// Quantises 16 columns of a block whose 8 lanes all call this (n of the
// columns exist, the others hold zeros) and writes codes and scale byte.
__device__ __forceinline__ void quantize16(const float (&v)[16], int n, uint8_t* codes, uint8_t* scale, int lane8) {
  const uint32_t b = fp8_scale_byte(group_umax<kBlockLanes>(amax_of(v)));
  if (n > 0) {
    store_codes16(codes, n, codes16(v, fp8_inverse_scale(b)));
    if (lane8 == 0) *scale = static_cast<uint8_t>(b);
  }
}

// Quotient by a divisor fixed per launch: floor(n / d) = high half of
// n * (floor(2^64 / d) + 1) for n d < 2^64.
struct Divider {
  uint64_t magic;
  uint64_t d;
  explicit Divider(uint64_t d_ = 1) : magic(d_ == 1 ? 0 : ~uint64_t{0} / d_ + 1), d(d_) {}
  __device__ __forceinline__ uint64_t quotient(uint64_t n) const { return d == 1 ? n : __umul64hi(n, magic); }
};

// Sum over a warp, the same in every lane.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(kFullMask, v, m);
  return v;
}
// Sum over the CTA's warps, added in the same order in every thread. `red`
// holds 32 floats, zero beyond the warps, and must not be the buffer of the
// call before (a thread may still be reading that one). WIDE: more than 16
// warps may take part.
template <bool WIDE>
__device__ __forceinline__ float cta_sum(float v, float* red) {
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = red[threadIdx.x & (WIDE ? 31 : 15)];
#pragma unroll
  for (int m = WIDE ? 16 : 8; m > 0; m >>= 1) s += __shfl_xor_sync(kFullMask, s, m);
  return s;
}

// 16 bytes global -> shared, of which the first `bytes` (0 .. 16) are read and
// the others zero-filled; src 16-byte aligned.
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
// The same of 8 bytes.
__device__ __forceinline__ void copy_async8(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest N groups of this thread have landed.
template <int N>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}

// ------------------------------------------------------------- launches ----
// A launch that may begin while the preceding kernel of the stream drains
// (each kernel waits for it before its first global access).
template <typename... P, typename... A>
inline cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, int threads, size_t smem,
                                    cudaStream_t stream, A&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<A&&>(args)...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// f(T{}) for the element type of a TACO_DTYPE_* value.
template <typename F>
inline cudaError_t with_dtype(int dtype, F&& f) {
  switch (dtype) {
    case TACO_DTYPE_BF16: return f(__nv_bfloat16{});
    case TACO_DTYPE_F16: return f(__half{});
    default: return f(float{});
  }
}

}  // namespace taco
