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

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Largest magnitude (as bits) of 8 values.
__device__ __forceinline__ uint32_t amax8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
  return m;
}
// Largest over the LANES consecutive lanes of an aligned group.
template <int LANES>
__device__ __forceinline__ uint32_t group_umax(uint32_t v) {
#pragma unroll
  for (int m = 1; m < LANES; m <<= 1) v = max(v, __shfl_xor_sync(kFullMask, v, m));
  return v;
}

// Eight codes of v * inv, element 0 in the low byte.
__device__ __forceinline__ uint2 codes8(const float (&v)[8], float inv) {
  return make_uint2(e4m3x4_from_f32(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                    e4m3x4_from_f32(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}
// Eight codes -> fp32 values times s (a power of two: exact).
__device__ __forceinline__ void decode8(uint2 c, float s, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? c.x : c.y;
    const f2 p = e4m3x2_to_f2((i & 1) ? w >> 16 : w);
    v[2 * i] = p.x * s;
    v[2 * i + 1] = p.y * s;
  }
}

// ------------------------------------------------------- element types ----
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ float from_f32(float v) { return v; }

// The elements of 8 consecutive columns; n (0 .. 8) of them exist, the others
// read as 0. VEC: p is 16-byte aligned.
template <typename T>
struct alignas(16) Pack8 {
  T v[8];
};
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int n, float (&v)[8]) {
  if (VEC && n == 8) {
    Pack8<T> q;
    const uint4* s = reinterpret_cast<const uint4*>(p);
    uint4* d = reinterpret_cast<uint4*>(&q);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(q) / 16); ++i) d[i] = s[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(q.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? to_f32(p[i]) : 0.0f;
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, int n, const float (&v)[8]) {
  if (VEC && n == 8) {
    Pack8<T> q;
#pragma unroll
    for (int i = 0; i < 8; ++i) q.v[i] = from_f32<T>(v[i]);
    const uint4* s = reinterpret_cast<const uint4*>(&q);
    uint4* d = reinterpret_cast<uint4*>(p);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(q) / 16); ++i) d[i] = s[i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = from_f32<T>(v[i]);
  }
}
// Codes of 8 consecutive columns: rows of codes start at multiples of 16
// bytes, so a full group is 8-byte aligned; a partial one is written byte by
// byte and leaves what lies behind the row alone.
__device__ __forceinline__ void store_codes8(uint8_t* p, int n, uint2 c) {
  if (n == 8) {
    *reinterpret_cast<uint2*>(p) = c;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = static_cast<uint8_t>((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
  }
}
__device__ __forceinline__ uint2 load_codes8(const uint8_t* p, int n) {
  if (n == 8) return *reinterpret_cast<const uint2*>(p);
  uint2 c = make_uint2(0, 0);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) (i < 4 ? c.x : c.y) |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
  return c;
}

// 8 consecutive entries of a weight vector of any element type.
template <bool VEC>
__device__ __forceinline__ void load_weight8(const void* w, int dtype, int64_t col, int n, float (&v)[8]) {
  if (dtype == TACO_DTYPE_F32)
    load8<float, VEC>(static_cast<const float*>(w) + col, n, v);
  else if (dtype == TACO_DTYPE_BF16)
    load8<__nv_bfloat16, VEC>(static_cast<const __nv_bfloat16*>(w) + col, n, v);
  else
    load8<__half, VEC>(static_cast<const __half*>(w) + col, n, v);
}

__device__ __forceinline__ int clamp8(int64_t left) {
  return left < 0 ? 0 : (left > 8 ? 8 : static_cast<int>(left));
}

// Sum over a CTA of WARPS warps (WARPS a runtime count <= 32); `red` holds one
// float per warp. Every thread gets the same sum, added in the same order.
__device__ __forceinline__ float cta_sum(float v, float* red, int warps) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(kFullMask, v, m);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < warps; ++i) s += red[i];
  __syncthreads();   // `red` may be written again
  return s;
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
