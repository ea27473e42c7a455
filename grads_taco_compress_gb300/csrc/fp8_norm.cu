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

#include "fp8_block.cuh"

namespace taco {

namespace {

template <typename T, int NC, bool VEC>
__global__ void __launch_bounds__(512) norm_kernel(NormArgs a, bool wide) {
  __shared__ float red[16];
  const int warps = blockDim.x >> 5, lane8 = threadIdx.x & 7;
  grid_launch_dependents();
  grid_dependency_wait();
  const int64_t row = blockIdx.x;
  Row16<T> h[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t col = 16 * (static_cast<int64_t>(threadIdx.x) + c * blockDim.x);
    h[c] = load16<T, VEC>(static_cast<const T*>(a.x) + row * a.ldx + col, clamp16(a.H - col), wide);
  }
  if (a.residual) {
    Row16<T> r[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = 16 * (static_cast<int64_t>(threadIdx.x) + c * blockDim.x);
      r[c] = load16<T, VEC>(static_cast<const T*>(a.residual) + row * a.ldr + col, clamp16(a.H - col), wide);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = 16 * (static_cast<int64_t>(threadIdx.x) + c * blockDim.x);
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
  sum = cta_sum(sum, red, warps);
  const float rstd = 1.0f / sqrtf(sum / static_cast<float>(a.H) + a.eps);
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t col = 16 * (static_cast<int64_t>(threadIdx.x) + c * blockDim.x);
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

// Rows blockIdx.x, blockIdx.x + gridDim.x, ... of the backward pass; the CTA's
// column sums of dy xh go to its row of `partial`. Each thread copies its own
// columns of the next DEPTH - 1 rows to shared memory while it works on one
// (rows that do not start on 16 bytes are loaded as they come: DEPTH 0), so the
// copies need no barrier and what is in flight costs no registers.
template <typename T, int NC, bool H>
struct BackwardStage {
  static constexpr int kT = sizeof(T);                  // 16-byte pieces of 16 columns
  static constexpr int kSaved = H ? kT : 1;
  static constexpr int kPieces = 2 * kT + kSaved;       // dy, dh, saved
  static constexpr size_t bytes(int threads) { return static_cast<size_t>(16) * NC * kPieces * threads; }
};

template <typename T, int NC, int DEPTH, bool H>
__global__ void __launch_bounds__(512) norm_backward_kernel(NormBackwardArgs a, bool wide) {
  using S = BackwardStage<T, NC, H>;
  constexpr bool VEC = DEPTH > 0;
  constexpr int kBufs = VEC ? DEPTH : 1;
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ float red[2][16];
  const int warps = blockDim.x >> 5;
  const uint32_t slot = smem_u32(ring) + 16 * threadIdx.x;
  const uint32_t pitch = 16 * blockDim.x;
  float dw[NC][16];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 16; ++i) dw[c][i] = 0.0f;
  grid_launch_dependents();
  grid_dependency_wait();

  const auto column = [&](int c) { return 16 * (static_cast<int64_t>(threadIdx.x) + c * blockDim.x); };
  // piece p of chunk c of a row in stage s
  const auto place = [&](int s, int c, int p) { return slot + ((s * NC + c) * S::kPieces + p) * pitch; };
  const auto begin_copy = [&](int64_t row, int s) {
    if (row < a.M) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const int64_t col = column(c);
        const int n = clamp16(a.H - col);
        const auto copy = [&](const void* base, int64_t ld, int first, int pieces, int es) {
          const char* p = static_cast<const char*>(base) + (row * ld + (n ? col : 0)) * es;
#pragma unroll
          for (int i = 0; i < pieces; ++i) {
            const int left = n * es - 16 * i;
            copy_async16(place(s, c, first + i), p + (left > 0 ? 16 * i : 0), left < 0 ? 0 : left > 16 ? 16 : left);
          }
        };
        copy(a.dy, a.lddy, 0, S::kT, sizeof(T));
        if (a.dh) copy(a.dh, a.lddh, S::kT, S::kT, sizeof(T));
        if (H)
          copy(a.h, a.ldh, 2 * S::kT, S::kT, sizeof(T));
        else
          copy(a.ck_codes, a.ck_ld, 2 * S::kT, 1, 1);
      }
    }
    copy_async_commit();
  };
  const auto staged = [&](int s, int c, int first) {
    Row16<T> r;
#pragma unroll
    for (int i = 0; i < S::kT; ++i) {
      const uint4 w = lds128(place(s, c, first + i));
      r.w[4 * i] = w.x;
      r.w[4 * i + 1] = w.y;
      r.w[4 * i + 2] = w.z;
      r.w[4 * i + 3] = w.w;
    }
    return r;
  };
  // read a row ahead: they are one byte and one word
  uint32_t next_scale[NC];
  float next_rstd = 0.0f;
  const auto peek = [&](int64_t row) {
    if (row >= a.M) return;
    next_rstd = a.rstd[row];
    if (!H)
#pragma unroll
      for (int c = 0; c < NC; ++c)
        next_scale[c] = column(c) < a.H ? a.ck_scales[row * a.ck_lds + column(c) / kFp8Block] : kScaleOne;
  };

  if (VEC)
    for (int s = 0; s < DEPTH - 1; ++s) begin_copy(blockIdx.x + static_cast<int64_t>(s) * gridDim.x, s);
  peek(blockIdx.x);
  float w[16];   // in registers for the whole call where a thread has one chunk
  if (NC == 1) load_weight16<VEC>(a.weight, a.weight_dtype, column(0), clamp16(a.H - column(0)), w);
  int s = 0;
  uint32_t turn = 0;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, turn ^= 1u) {
    if (VEC) begin_copy(row + static_cast<int64_t>(DEPTH - 1) * gridDim.x, (s + DEPTH - 1) % kBufs);
    uint32_t scale[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) scale[c] = next_scale[c];
    const float rstd = next_rstd;
    peek(row + gridDim.x);
    if (VEC) copy_async_wait<VEC ? DEPTH - 1 : 0>();
    float g[NC][16], xh[NC][16];
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = column(c);
      const int n = clamp16(a.H - col);
      if (VEC) {
        unpack<T>(staged(s, c, 0), g[c]);
        if (H)
          unpack<T>(staged(s, c, 2 * S::kT), xh[c]);
        else
          decode16(lds128(place(s, c, 2 * S::kT)), fp8_scale(scale[c]), xh[c]);
      } else {
        unpack<T>(load16<T, false>(static_cast<const T*>(a.dy) + row * a.lddy + col, n, false), g[c]);
        if (H)
          unpack<T>(load16<T, false>(static_cast<const T*>(a.h) + row * a.ldh + col, n, false), xh[c]);
        else
          decode16(load_codes16(a.ck_codes + row * a.ck_ld + col, n), fp8_scale(scale[c]), xh[c]);
      }
      if (NC > 1) load_weight16<VEC>(a.weight, a.weight_dtype, col, n, w);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        // columns that do not exist are 0, or NaN in a block whose scale is:
        // there the row's sum is NaN by those that do
        xh[c][i] *= rstd;
        dw[c][i] = fmaf(g[c][i], xh[c][i], dw[c][i]);
        g[c][i] *= w[i];
        sum = fmaf(g[c][i], xh[c][i], sum);
      }
    }
    const float mean = cta_sum(sum, red[turn], warps) / static_cast<float>(a.H);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = column(c);
      const int n = clamp16(a.H - col);
#pragma unroll
      for (int i = 0; i < 16; ++i) g[c][i] = rstd * fmaf(-xh[c][i], mean, g[c][i]);
      if (a.dh) {
        float d[16];
        unpack<T>(VEC ? staged(s, c, S::kT)
                      : load16<T, false>(static_cast<const T*>(a.dh) + row * a.lddh + col, n, false), d);
#pragma unroll
        for (int i = 0; i < 16; ++i) g[c][i] += d[i];
      }
      store16<T, VEC>(static_cast<T*>(a.dx) + row * a.lddx + col, n, wide, pack<T>(g[c]));
    }
    s = s + 1 == kBufs ? 0 : s + 1;
  }
  if (VEC) copy_async_wait<0>();
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t col = column(c);
    const int n = clamp16(a.H - col);
    float* p = a.partial + blockIdx.x * a.H + col;
    if (n == 16 && a.H % 4 == 0) {   // every CTA's row of partial sums starts on 16 bytes
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<float4*>(p + i) = make_float4(dw[c][i], dw[c][i + 1], dw[c][i + 2], dw[c][i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < n) p[i] = dw[c][i];
    }
  }
}

// dw = the sum of the G rows of partial sums, in a fixed order: a CTA takes 32
// columns, warp w adds rows w, w + 8, ..., and the 8 sums meet in order.
__global__ void __launch_bounds__(256) norm_dw_kernel(const float* partial, int G, int64_t H, float* dw) {
  __shared__ float part[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  grid_launch_dependents();
  grid_dependency_wait();
  float s = 0.0f;
  if (col < H) {
#pragma unroll 8
    for (int g = warp; g < G; g += 8) s += partial[g * H + col];
  }
  part[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < H) {
    s = part[0][lane];
#pragma unroll
    for (int w = 1; w < 8; ++w) s += part[w][lane];
    dw[col] = s;
  }
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
  return launch_dependent(vec ? norm_kernel<T, NC, true> : norm_kernel<T, NC, false>,
                          dim3(static_cast<unsigned>(a.M)), threads, 0, st, a, vec == kVec32);
}

// Shared memory that a CTA's ring of rows may take: two CTAs per SM, else one.
constexpr size_t kRingTwo = 112 * 1024, kRingOne = 226 * 1024;
constexpr int kMaxThreads = 512;

// The ring's depth for a stage of this size (0: no ring) and its bytes.
int ring_depth(size_t stage, bool vec) { return !vec ? 0 : 4 * stage <= kRingTwo ? 4 : 2 * stage <= kRingOne ? 2 : 0; }

template <typename T, int NC, bool H, typename F>
auto with_backward_kernel(int depth, F&& f) {
  return depth == 4   ? f(norm_backward_kernel<T, NC, 4, H>)
         : depth == 2 ? f(norm_backward_kernel<T, NC, 2, H>)
                      : f(norm_backward_kernel<T, NC, 0, H>);
}

template <typename T, int NC, bool H>
cudaError_t launch_norm_backward_t(const NormBackwardArgs& a, int threads, int vec, int grid, cudaStream_t st) {
  const size_t stage = BackwardStage<T, NC, H>::bytes(threads);
  const int depth = ring_depth(stage, vec != kVecNone);
  return with_backward_kernel<T, NC, H>(depth, [&](auto k) {
    return launch_dependent(k, dim3(grid), threads, depth * stage, st, a, vec == kVec32);
  });
}

template <typename T, int NC, bool H>
cudaError_t prepare_backward_t() {
  cudaError_t e = cudaSuccess;
  for (int depth : {2, 4})
    if (e == cudaSuccess)
      e = with_backward_kernel<T, NC, H>(depth, [&](auto k) {
        const size_t most = depth * BackwardStage<T, NC, H>::bytes(kMaxThreads);
        const size_t room = depth == 4 ? kRingTwo : kRingOne;
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(most < room ? most : room));
      });
  return e;
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, int dtype, int vec, int sms, cudaStream_t st) {
  (void)sms;
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

// CTAs of the backward pass: as many as stay resident (3, 2 or 1 per SM by
// their threads), no more than rows, and no more than rows of partial sums.
int norm_backward_ctas(int64_t M, int64_t H, int sms) {
  int threads, nc;
  norm_shape(H, &threads, &nc);
  const int per_sm = threads <= 128 ? 3 : threads <= 256 ? 2 : 1;
  int64_t most = static_cast<int64_t>(per_sm) * sms;
  if (most > kNormMaxPartials) most = kNormMaxPartials;
  return static_cast<int>(M < most ? M : most);
}

cudaError_t launch_norm_backward(const NormBackwardArgs& a, int dtype, int vec, int grid, cudaStream_t st) {
  int threads, nc;
  norm_shape(a.H, &threads, &nc);
  const auto launch = [&](auto t, auto held) {
    using T = decltype(t);
    constexpr bool H = decltype(held)::value;
    return nc == 1   ? launch_norm_backward_t<T, 1, H>(a, threads, vec, grid, st)
           : nc == 2 ? launch_norm_backward_t<T, 2, H>(a, threads, vec, grid, st)
                     : launch_norm_backward_t<T, 4, H>(a, threads, vec, grid, st);
  };
  if (grid > 0) {
    const cudaError_t e = with_dtype(dtype, [&](auto t) {
      return a.h ? launch(t, std::true_type{}) : launch(t, std::false_type{});
    });
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(norm_dw_kernel, dim3(static_cast<unsigned>((a.H + 31) / 32)), 256, 0, st,
                          static_cast<const float*>(a.partial), grid, a.H, a.dw);
}

}  // namespace taco
