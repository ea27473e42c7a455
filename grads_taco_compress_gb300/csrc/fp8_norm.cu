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
// A CTA takes a row at a time; thread t holds the 16-column chunks t, t + T,
// ... in registers, so a row is read once and a block of 128 columns is 8
// consecutive lanes. Sums are fp32.
//
// Measured, bf16 (a plain copy: 6.7 TB/s): forward of 16384 x 3584 with residual
// and checkpoint 72.5 us, 6.5 TB/s, bound by memory; backward of 8192 x 4096
// with dh 45 us, 5.2 TB/s with the column sums' second kernel (4 us), 67% of
// the issue slots taken.

#include "fp8_block.cuh"

namespace taco {

namespace {

//
// WARP: rows of at most 512 columns, one to a warp, kWarpRows to a CTA (65536
// rows of 512: 67 us with a CTA of one warp a row, 42 us so).
constexpr int kWarpRows = 8;

template <typename T, int NC, bool VEC, bool WARP>
__global__ void __launch_bounds__(512) norm_kernel(NormArgs a, bool wide) {
  __shared__ float red[32];
  const int lane8 = threadIdx.x & 7;
  const uint32_t slot = WARP ? threadIdx.x & 31 : threadIdx.x;   // place in the row
  const uint32_t threads = WARP ? 32 : blockDim.x;
  if (!WARP && threadIdx.x < 32 && threadIdx.x >= blockDim.x >> 5) red[threadIdx.x] = 0.0f;
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t row = WARP ? static_cast<int64_t>(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && row >= a.M) return;   // whole warps
  Row16<T> h[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t col = 16 * (static_cast<int64_t>(slot) + c * threads);
    h[c] = load16<T, VEC>(static_cast<const T*>(a.x) + row * a.ldx + col, clamp16(a.H - col), wide);
  }
  if (a.residual) {
    Row16<T> r[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = 16 * (static_cast<int64_t>(slot) + c * threads);
      r[c] = load16<T, VEC>(static_cast<const T*>(a.residual) + row * a.ldr + col, clamp16(a.H - col), wide);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = 16 * (static_cast<int64_t>(slot) + c * threads);
      float x[16], y[16];
      unpack<T>(h[c], x);
      unpack<T>(r[c], y);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] += y[i];
      h[c] = pack<T>(x);
      store16<T, VEC>(static_cast<T*>(a.h) + row * a.ldh + col, clamp16(a.H - col), wide, h[c]);
    }
  }
  float sum = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float v[16];
    unpack<T>(h[c], v);
#pragma unroll
    for (int i = 0; i < 16; ++i) sum = fmaf(v[i], v[i], sum);
  }
  sum = WARP ? warp_sum(sum) : cta_sum<false>(sum, red);
  const float rstd = 1.0f / sqrtf(sum / static_cast<float>(a.H) + a.eps);
  if (a.rstd && slot == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t col = 16 * (static_cast<int64_t>(slot) + c * threads);
    const int n = clamp16(a.H - col);
    float v[16], w[16];
    unpack<T>(h[c], v);
    if (a.ck_codes)
      quantize16(v, n, a.ck_codes + row * a.ck_ld + col, a.ck_scales + row * a.ck_lds + col / kFp8Block, lane8);
    load_weight16<VEC>(a.weight, a.weight_dtype, col, n, w);
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] *= v[i] * rstd;
    quantize16(w, n, a.codes + row * a.ldc + col, a.scales + row * a.lds + col / kFp8Block, lane8);
  }
}

// The backward pass holds no block's maximum, so a thread takes 8 columns: twice
// the warps of the forward's 16 at the same registers in all, and the row's
// chain of loads, sum and stores needs them (two CTAs of 256 threads with 16
// columns each, 4 warps a scheduler: 59 us at 8192 x 4096).
template <typename T>
struct Row8 {
  uint32_t w[2 * sizeof(T)];
};
template <typename T>
__device__ __forceinline__ void unpack8(const Row8<T>& r, f2 (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<T, float>::value) {
      v[i] = f2{__uint_as_float(r.w[2 * i]), __uint_as_float(r.w[2 * i + 1])};
    } else if constexpr (std::is_same<T, __half>::value) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.w[i]));
      v[i] = f2{f.x, f.y};
    } else {
      v[i] = f2{bf16_lo(r.w[i]), bf16_hi(r.w[i])};
    }
  }
}
template <typename T>
__device__ __forceinline__ Row8<T> pack8(const f2 (&v)[4]) {
  Row8<T> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (std::is_same<T, float>::value) {
      r.w[2 * i] = __float_as_uint(v[i].x);
      r.w[2 * i + 1] = __float_as_uint(v[i].y);
    } else if constexpr (std::is_same<T, __half>::value) {
      const __half2 h = __floats2half2_rn(v[i].x, v[i].y);
      r.w[i] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      r.w[i] = pack_bf16x2(v[i].x, v[i].y);
    }
  }
  return r;
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, int n, const Row8<T>& r) {
  if (VEC && n == 8) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
      *reinterpret_cast<uint4*>(p + 4 * i) = make_uint4(r.w[4 * i], r.w[4 * i + 1], r.w[4 * i + 2], r.w[4 * i + 3]);
  } else if constexpr (VEC) {
    f2 v[4];
    unpack8<T>(r, v);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = from_f32<T>(i & 1 ? v[i >> 1].y : v[i >> 1].x);
  } else {
    store_shifted(p, n, r.w);
  }
}
// 8 entries of a vector or row.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int n, f2 (&v)[4]) {
  Row8<T> r;
  if (VEC && n == 8) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
      *reinterpret_cast<uint4*>(r.w + 4 * i) = *reinterpret_cast<const uint4*>(p + 4 * i);
  } else {
    load_shifted(p, n, r.w);
  }
  unpack8<T>(r, v);
}
template <bool VEC>
__device__ __forceinline__ void load_weight8(const void* w, int dtype, int64_t col, int n, f2 (&v)[4]) {
  if (dtype == TACO_DTYPE_F32)
    load8<float, VEC>(static_cast<const float*>(w) + col, n, v);
  else if (dtype == TACO_DTYPE_BF16)
    load8<__nv_bfloat16, VEC>(static_cast<const __nv_bfloat16*>(w) + col, n, v);
  else
    load8<__half, VEC>(static_cast<const __half*>(w) + col, n, v);
}
__device__ __forceinline__ void decode8(uint2 c, float s, f2 (&v)[4]) {
  const f2 ss{s, s};
  v[0] = mul2(e4m3x2_to_f2(c.x & 0xffffu), ss);
  v[1] = mul2(e4m3x2_to_f2(c.x >> 16), ss);
  v[2] = mul2(e4m3x2_to_f2(c.y & 0xffffu), ss);
  v[3] = mul2(e4m3x2_to_f2(c.y >> 16), ss);
}
__device__ __forceinline__ uint2 load_codes8(const uint8_t* p, int n) {
  if (n == 8) return *reinterpret_cast<const uint2*>(p);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) w[i >> 2] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}

// Rows blockIdx.x, blockIdx.x + gridDim.x, ... of the backward pass; the CTA's
// column sums of dy xh go to its row of `partial`. Each thread copies its own
// columns of the next DEPTH - 1 rows to shared memory while it works on one
// (DEPTH 0, where no two stages fit: rows are loaded as they come), so the
// copies need no barrier and what is in flight costs no registers. SHIFT: rows
// start anywhere; a thread copies the aligned 16-byte pieces that hold its
// columns, one more than they fill, and shifts as it reads them (9240 x 2804
// bf16: 87 us with rows loaded as they come, 68 so).
template <typename T, int NC, bool H, bool SHIFT>
struct BackwardStage {
  // 8 columns: 16-byte pieces of dy, dh and h, and bytes of h or codes
  static constexpr int kPieces = sizeof(T) / 2 + (SHIFT ? 1 : 0), kRow = 16 * kPieces, kSaved = H ? kRow : 8;
  static constexpr int kThread = 2 * kRow + kSaved;
  static constexpr size_t bytes(int threads) { return static_cast<size_t>(NC) * kThread * threads; }
};

template <typename T, int NC, int DEPTH, bool H, bool SHIFT>
__global__ void __launch_bounds__(1024) norm_backward_kernel(NormBackwardArgs a) {
  using S = BackwardStage<T, NC, H, SHIFT>;
  constexpr bool RING = DEPTH > 0, VEC = RING && !SHIFT;
  constexpr int kPieces = S::kPieces;
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ float red[2][32];
  if (threadIdx.x < 32 && threadIdx.x >= blockDim.x >> 5) red[0][threadIdx.x] = red[1][threadIdx.x] = 0.0f;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  const uint32_t threads = blockDim.x, step = gridDim.x;

  // Everything that does not change from row to row: this thread's columns and
  // how many exist (copies of none read zero bytes at the row's start), and its
  // place in a stage of the ring.
  int64_t col[NC];
  int n[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    col[c] = 8 * (static_cast<int64_t>(threadIdx.x) + c * threads);
    const int64_t left = a.H - col[c];
    n[c] = left < 0 ? 0 : left > 8 ? 8 : static_cast<int>(left);
    if (VEC && n[c] == 0) col[c] = 0;
  }
  const uint32_t stage_bytes = NC * S::kThread * threads;
  const uint32_t slot16 = smem_u32(ring) + 16 * threadIdx.x;
  const uint32_t slot8 = smem_u32(ring) + 2 * S::kRow * threads + 8 * threadIdx.x;   // codes: after dy and dh
  f2 dw[NC][4];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[c][i] = f2{0.0f, 0.0f};
  grid_launch_dependents();
  grid_dependency_wait();

  const T* dy = static_cast<const T*>(a.dy) + blockIdx.x * a.lddy;
  const T* dh = a.dh ? static_cast<const T*>(a.dh) + blockIdx.x * a.lddh : nullptr;
  const T* h = H ? static_cast<const T*>(a.h) + blockIdx.x * a.ldh : nullptr;
  const uint8_t* codes = H ? nullptr : a.ck_codes + blockIdx.x * a.ck_ld;
  const uint8_t* scales = H ? nullptr : a.ck_scales + blockIdx.x * a.ck_lds;
  T* dx = static_cast<T*>(a.dx) + blockIdx.x * a.lddx;
  const int64_t dy_step = step * a.lddy, dh_step = step * a.lddh, h_step = step * a.ldh, codes_step = step * a.ck_ld,
                scales_step = step * a.ck_lds, dx_step = step * a.lddx;

  // dy, dh, h and codes run ahead of the row that is worked on by the ring's
  // depth (RING), scales and rstd by one row
  int64_t ahead = blockIdx.x;
  uint32_t put = 0, get = 0;   // byte offsets of the stages written and read next
  const auto begin_copy = [&]() {
    if (ahead < a.M) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const uint32_t to = put + c * (S::kThread * threads);
        const auto copy = [&](const T* from, int first) {
#pragma unroll
          for (int i = 0; i < kPieces; ++i) {
            if (SHIFT) {
              const uintptr_t at = reinterpret_cast<uintptr_t>(from);
              const int s = static_cast<int>(at & 15);
              const bool any = n[c] && 16 * i < s + n[c] * static_cast<int>(sizeof(T));
              copy_async16(slot16 + to + (first + i) * 16 * threads,
                           reinterpret_cast<const T*>(at - s + (any ? col[c] * sizeof(T) + 16 * i : 0)), any ? 16 : 0);
              continue;
            }
            constexpr int kPer = 16 / static_cast<int>(sizeof(T));
            const int left = n[c] - kPer * i;   // elements of this piece that exist
            const int bytes = (left < 0 ? 0 : left > kPer ? kPer : left) * static_cast<int>(sizeof(T));
            copy_async16(slot16 + to + (first + i) * 16 * threads, from + col[c] + (left > 0 ? kPer * i : 0), bytes);
          }
        };
        copy(dy, 0);
        if (dh) copy(dh, kPieces);
        if (H)
          copy(h, 2 * kPieces);
        else
          copy_async8(slot8 + to, codes + (SHIFT && n[c] == 0 ? 0 : col[c]), n[c]);
      }
      dy += dy_step;
      if (dh) dh += dh_step;
      if (H) h += h_step;
      else codes += codes_step;
    }
    ahead += step;
    copy_async_commit();
    put = put + stage_bytes == DEPTH * stage_bytes ? 0 : put + stage_bytes;
  };
  const auto staged = [&](int c, int first, const void* base, int64_t ld, int64_t row, f2 (&v)[4]) {
    Row8<T> r;
    uint32_t q[4 * kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint4 piece = lds128(slot16 + get + c * (S::kThread * threads) + (first + i) * 16 * threads);
      q[4 * i] = piece.x;
      q[4 * i + 1] = piece.y;
      q[4 * i + 2] = piece.z;
      q[4 * i + 3] = piece.w;
    }
    if constexpr (SHIFT) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(static_cast<const T*>(base) + row * ld);
      const uint32_t s = static_cast<uint32_t>(at & 15);
      shift_words<T>(q, s, n[c], r.w);
    } else {
#pragma unroll
      for (int i = 0; i < 4 * kPieces; ++i) r.w[i] = q[i];
    }
    unpack8<T>(r, v);
  };
  uint32_t next_scale[NC];
  float next_rstd = 0.0f;
  const float* rstds = a.rstd + blockIdx.x;
  const auto peek = [&](int64_t row) {
    if (row >= a.M) return;
    next_rstd = *rstds;
    rstds += step;
    if (!H) {
#pragma unroll
      for (int c = 0; c < NC; ++c) next_scale[c] = scales[n[c] ? static_cast<uint32_t>(col[c]) / kFp8Block : 0u];
      scales += scales_step;
    }
  };

  if (RING)
    for (int s = 0; s < DEPTH - 1; ++s) begin_copy();
  peek(blockIdx.x);
  f2 w[4];   // in registers for the whole call where a thread has one chunk
  if (NC == 1) load_weight8<VEC>(a.weight, a.weight_dtype, col[0], n[0], w);
  uint32_t turn = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += step, turn ^= 1u) {
    if (RING) begin_copy();
    float scale[NC];
    const float rstd = next_rstd;
    // a code times its scale is exact, so scale and rstd may be multiplied first
#pragma unroll
    for (int c = 0; c < NC; ++c) scale[c] = H ? rstd : fp8_scale(next_scale[c]) * rstd;
    peek(row + step);
    if (RING) copy_async_wait<RING ? DEPTH - 1 : 0>();
    f2 g[NC][4], xh[NC][4], part{0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (RING)
        staged(c, 0, a.dy, a.lddy, row, g[c]);
      else
        load8<T, false>(dy + col[c], n[c], g[c]);
      if (H) {
        if (RING)
          staged(c, 2 * kPieces, a.h, a.ldh, row, xh[c]);
        else
          load8<T, false>(h + col[c], n[c], xh[c]);
      } else {
        const uint2 q = RING ? lds64(slot8 + get + c * (S::kThread * threads)) : load_codes8(codes + col[c], n[c]);
        decode8(q, scale[c], xh[c]);
      }
      if (NC > 1) load_weight8<VEC>(a.weight, a.weight_dtype, col[c], n[c], w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // columns that do not exist are 0, or NaN in a block whose scale is:
        // there the row's sum is NaN by those that do
        if (H) xh[c][i] = mul2(xh[c][i], f2{rstd, rstd});
        dw[c][i] = fma2(g[c][i], xh[c][i], dw[c][i]);
        g[c][i] = mul2(g[c][i], w[i]);
        part = fma2(g[c][i], xh[c][i], part);
      }
    }
    const float mean = cta_sum<true>(part.x + part.y, red[turn]) * inv_h;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      f2 d[4];
      if (a.dh) {
        if (RING)
          staged(c, kPieces, a.dh, a.lddh, row, d);
        else
          load8<T, false>(dh + col[c], n[c], d);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        g[c][i] = fma2(xh[c][i], f2{-mean, -mean}, g[c][i]);
        g[c][i] = a.dh ? fma2(g[c][i], f2{rstd, rstd}, d[i]) : mul2(g[c][i], f2{rstd, rstd});
      }
      store8<T, VEC>(dx + col[c], n[c], pack8<T>(g[c]));
    }
    dx += dx_step;
    if (!RING) {
      dy += dy_step;
      if (dh) dh += dh_step;
      if (H) h += h_step;
      else codes += codes_step;
    }
    get = get + stage_bytes == DEPTH * stage_bytes ? 0 : get + stage_bytes;
  }
  if (RING) copy_async_wait<0>();
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float* p = a.partial + blockIdx.x * a.H + col[c];
    if (n[c] == 8 && a.H % 4 == 0) {   // every CTA's row of partial sums starts on 16 bytes
#pragma unroll
      for (int i = 0; i < 4; i += 2)
        *reinterpret_cast<float4*>(p + 2 * i) = make_float4(dw[c][i].x, dw[c][i].y, dw[c][i + 1].x, dw[c][i + 1].y);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n[c]) p[i] = i & 1 ? dw[c][i >> 1].y : dw[c][i >> 1].x;
    }
  }
}

// dw = the sum of the G rows of partial sums, in a fixed order: a CTA takes 32
// columns, warp w adds rows w, w + 32, ..., and the 32 sums meet in order.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* partial, int G, int64_t H, float* dw) {
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  grid_launch_dependents();
  grid_dependency_wait();
  float s = 0.0f;
  if (col < H) {
#pragma unroll 16
    for (int g = warp; g < G; g += 32) s += partial[g * H + col];
  }
  part[warp][lane] = s;
  __syncthreads();
  // warp w: column w, one sum per lane
  s = part[lane][warp];
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(kFullMask, s, m);
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + warp;
  if (lane == 0 && c < H) dw[c] = s;
}

// Threads and 8-column chunks per thread of the backward pass: at most 1024.
void backward_shape(int64_t H, int* threads, int* nc) {
  const int64_t chunks = (H + 7) / 8;
  *nc = chunks <= 1024 ? 1 : chunks <= 2048 ? 2 : 4;
  const int64_t t = (chunks + *nc - 1) / *nc;
  *threads = static_cast<int>((t + 31) / 32 * 32);
}

// Threads and 16-column chunks per thread for H columns: at most 512 threads.
void norm_shape(int64_t H, int* threads, int* nc) {
  const int64_t chunks = (H + 15) / 16;
  *nc = chunks <= 512 ? 1 : chunks <= 1024 ? 2 : 4;
  const int64_t t = (chunks + *nc - 1) / *nc;
  *threads = static_cast<int>((t + 31) / 32 * 32);
}

template <typename T, int NC>
cudaError_t launch_norm_t(const NormArgs& a, int threads, int vec, cudaStream_t st) {
  if (NC == 1 && threads == 32)
    return launch_dependent(vec ? norm_kernel<T, 1, true, true> : norm_kernel<T, 1, false, true>,
                            dim3(static_cast<unsigned>((a.M + kWarpRows - 1) / kWarpRows)), 32 * kWarpRows, 0, st, a,
                            vec == kVec32);
  return launch_dependent(vec ? norm_kernel<T, NC, true, false> : norm_kernel<T, NC, false, false>,
                          dim3(static_cast<unsigned>(a.M)), threads, 0, st, a, vec == kVec32);
}

// CTAs of the backward pass that an SM holds at 64 registers a thread.
int backward_ctas_per_sm(int threads) { return 1024 / threads < 16 ? 1024 / threads : 16; }

// Shared memory that the rings of an SM's CTAs may take together, and the
// ring's depth for a stage of this size (0: no ring).
constexpr size_t kRingRoom = 222 * 1024;
constexpr int kMaxDepth = 4;
int ring_depth(size_t stage, int per_sm) {
  const size_t depth = kRingRoom / per_sm / stage;
  return depth < 2 ? 0 : depth < kMaxDepth ? static_cast<int>(depth) : kMaxDepth;
}

// Rows that start anywhere: rings of 2 or 4 stages for threads of one chunk of
// a 16-bit type (fp32 copies half as much again as it uses: 4096 x 8191 takes
// 158 us so, 124 us with rows loaded as they come).
template <typename T>
constexpr bool shifted_ring() { return sizeof(T) == 2; }
template <typename T, int NC, bool H, bool SHIFT, typename F>
auto with_backward_kernel(int depth, F&& f) {
  if constexpr (SHIFT)
    return depth == 4 ? f(norm_backward_kernel<T, NC, 4, H, true>) : f(norm_backward_kernel<T, NC, 2, H, true>);
  else
    return depth == 4   ? f(norm_backward_kernel<T, NC, 4, H, false>)
           : depth == 3 ? f(norm_backward_kernel<T, NC, 3, H, false>)
           : depth == 2 ? f(norm_backward_kernel<T, NC, 2, H, false>)
                        : f(norm_backward_kernel<T, NC, 0, H, false>);
}

template <typename T, int NC, bool H>
cudaError_t launch_norm_backward_t(const NormBackwardArgs& a, int threads, bool vec, int grid, cudaStream_t st) {
  const int per_sm = backward_ctas_per_sm(threads);
  if constexpr (NC == 1 && shifted_ring<T>()) {
    const size_t stage = BackwardStage<T, 1, H, true>::bytes(threads);
    const int depth = vec ? 0 : ring_depth(stage, per_sm) & ~1;
    if (depth)
      return with_backward_kernel<T, 1, H, true>(depth, [&](auto k) {
        return launch_dependent(k, dim3(grid), threads, depth * stage, st, a);
      });
  }
  const size_t stage = BackwardStage<T, NC, H, false>::bytes(threads);
  const int depth = vec ? ring_depth(stage, per_sm) : 0;
  return with_backward_kernel<T, NC, H, false>(depth, [&](auto k) {
    return launch_dependent(k, dim3(grid), threads, depth * stage, st, a);
  });
}

template <typename T, int NC, bool H, bool SHIFT>
cudaError_t prepare_rings() {
  cudaError_t e = cudaSuccess;
  for (int depth = 2; depth <= kMaxDepth; depth += SHIFT ? 2 : 1)
    if (e == cudaSuccess)
      e = with_backward_kernel<T, NC, H, SHIFT>(depth, [&](auto k) {
        const size_t most = depth * BackwardStage<T, NC, H, SHIFT>::bytes(1024);
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(most < kRingRoom ? most : kRingRoom));
      });
  return e;
}
template <typename T, int NC, bool H>
cudaError_t prepare_backward_t() {
  const cudaError_t e = prepare_rings<T, NC, H, false>();
  if constexpr (NC == 1 && shifted_ring<T>())
    if (e == cudaSuccess) return prepare_rings<T, 1, H, true>();
  return e;
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, int dtype, int vec, cudaStream_t st) {
  int threads, nc;
  norm_shape(a.H, &threads, &nc);
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    return nc == 1   ? launch_norm_t<T, 1>(a, threads, vec, st)
           : nc == 2 ? launch_norm_t<T, 2>(a, threads, vec, st)
                     : launch_norm_t<T, 4>(a, threads, vec, st);
  });
}

cudaError_t prepare_norm() {
  cudaError_t e = cudaSuccess;
  for (int dtype : {TACO_DTYPE_BF16, TACO_DTYPE_F16, TACO_DTYPE_F32})
    if (e == cudaSuccess)
      e = with_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        for (cudaError_t r : {prepare_backward_t<T, 1, true>(), prepare_backward_t<T, 1, false>(),
                              prepare_backward_t<T, 2, true>(), prepare_backward_t<T, 2, false>(),
                              prepare_backward_t<T, 4, true>(), prepare_backward_t<T, 4, false>()})
          if (r != cudaSuccess) return r;
        return cudaSuccess;
      });
  return e;
}

int64_t norm_max_partials(int64_t H) { return H >= 2048 ? 512 : H >= 512 ? 512 * 2048 / H : 2048; }

// CTAs of the backward pass: as many as stay resident, no more than rows, and
// no more than rows of partial sums.
int norm_backward_ctas(int64_t M, int64_t H, int sms) {
  int threads, nc;
  backward_shape(H, &threads, &nc);
  int64_t most = static_cast<int64_t>(backward_ctas_per_sm(threads)) * sms;
  const int64_t partials = norm_max_partials(H);
  if (most > partials) most = partials;
  return static_cast<int>(M < most ? M : most);
}

cudaError_t launch_norm_backward(const NormBackwardArgs& a, int dtype, int vec, int grid, cudaStream_t st) {
  int threads, nc;
  backward_shape(a.H, &threads, &nc);
  const auto launch = [&](auto t, auto held) {
    using T = decltype(t);
    constexpr bool H = decltype(held)::value;
    return nc == 1   ? launch_norm_backward_t<T, 1, H>(a, threads, vec != kVecNone, grid, st)
           : nc == 2 ? launch_norm_backward_t<T, 2, H>(a, threads, vec != kVecNone, grid, st)
                     : launch_norm_backward_t<T, 4, H>(a, threads, vec != kVecNone, grid, st);
  };
  if (grid > 0) {
    const cudaError_t e = with_dtype(dtype, [&](auto t) {
      return a.h ? launch(t, std::true_type{}) : launch(t, std::false_type{});
    });
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(norm_dw_kernel, dim3(static_cast<unsigned>((a.H + 31) / 32)), 1024, 0, st,
                          static_cast<const float*>(a.partial), grid, a.H, a.dw);
}

}  // namespace taco
