// C [M, N] = A [M, K] B [N, K]^T of two FP8 block tensors, on the block-scaled
// tensor-core instructions (tcgen05 kind::mxf8f6f4):
//
//   C[m][n] = sum over blocks k of  2^(sa[m][k] - 127) 2^(sb[n][k] - 127)
//             * sum over the 128 columns of block k of  a[m][j] b[n][j]
//
// The instruction multiplies each 32-column product by the two E8M0 scales as
// it accumulates, in fp32 in tensor memory; a scale of a 128-column block
// serves four of them. Nothing is decoded on the CUDA cores. Rows and columns
// beyond the tensors read as zero codes (the tensor copies fill them in) with
// scale 1.
//
// CTA = 8 warps, one output tile of 128 x 128:
//   warp 0     TMA producer: stages of 128 columns, [128 rows x 128 bytes] of
//              A and of B, 128-byte swizzle;
//   warp 1     owns the tensor memory; one lane copies the scales to tensor
//              memory, issues the MMAs and commits each stage;
//   warp 2     scales: every 4 stages (512 columns) one 32-bit word per row of
//              A and B, byte j the scale of stage j, in the order that
//              tcgen05.cp 32x128b spreads over the tensor memory;
//   warps 4-7  epilogue: lane = row, tensor memory to registers to C.
// Every wait is bounded in time with a CTA-wide abort flag.

#include "fp8_block.cuh"
#include "tcgen05.cuh"

namespace taco {

namespace {

__device__ unsigned int g_fp8_matmul_fault;

constexpr int kThreads = 256;
constexpr int kTileM = 128, kTileN = 128;
constexpr int kStages = 6;
constexpr int kChunk = 4;                               // stages per word of scales
constexpr int kScaleBufs = 3;
constexpr uint32_t kStageBytes = (kTileM + kTileN) * kFp8Block;
constexpr uint32_t kScaleBytes = (kTileM + kTileN) * 4;
constexpr uint32_t kSmemStages = 0;
constexpr uint32_t kSmemScales = kStages * kStageBytes;
constexpr uint32_t kSmemBars = kSmemScales + kScaleBufs * kScaleBytes;
constexpr uint32_t kFull = kSmemBars, kEmpty = kFull + 8 * kStages;
constexpr uint32_t kSFull = kEmpty + 8 * kStages, kSEmpty = kSFull + 8 * kScaleBufs;
constexpr uint32_t kDone = kSEmpty + 8 * kScaleBufs, kSlot = kDone + 8, kAbort = kSlot + 4;
constexpr uint32_t kSmemBytes = kAbort + 4 + 1024;
constexpr uint32_t kTmemCols = 256;
// Scale words of three chunks in tensor memory, so that a copy never meets an
// MMA that still reads the words it replaces: when stage i's operands have
// landed, the MMAs of stage i - kStages are done, and those of the chunk three
// before the one that stage i begins ended with stage i - 9.
constexpr int kTmemScaleBufs = 3;
static_assert(4 * kTmemScaleBufs - 3 >= kStages, "scale words replaced too early");
constexpr uint32_t kColScales = kTileN;

// Instruction descriptor of kind::mxf8f6f4 with E4M3 operands, K-major, E8M0
// scales: N >> 3 at bits 17-22, scale type at bit 23, M >> 7 at bits 27-28;
// the byte of the scale word at bits 29-30 (A) and 4-5 (B).
constexpr uint32_t mx_desc(uint32_t m, uint32_t n) {
  return ((n >> 3) << 17) | (1u << 23) | ((m >> 7) << 27);
}
constexpr uint32_t kDesc = mx_desc(kTileM, kTileN);
__device__ __forceinline__ void mma_mx(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%5], [%6], p;\n}"
      :: "r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb) : "memory");
}
// 32 rows of 16 bytes to 4 tensor-memory columns, repeated for the four
// 32-lane quarters.
__device__ __forceinline__ void tmem_copy_scales(uint32_t taddr, uint32_t saddr) {
  const uint64_t desc = umma_desc(saddr, 0, 128);   // no swizzle, 8 rows of 16 bytes per group
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" :: "r"(taddr), "l"(desc) : "memory");
}
__device__ __forceinline__ bool wait_here(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag) {
  return wait_or_abort(bar, parity, abort_flag, &g_fp8_matmul_fault, kFaultFp8MatmulWait);
}

struct MatmulMaps {
  CUtensorMap a, b;
};

// The scale word of one row for chunk q (bytes beyond the last block are
// whatever the row's padding holds and are never used).
__device__ __forceinline__ uint32_t scale_word(const uint8_t* s, int64_t ld, int64_t row, int64_t rows,
                                               int tile, int64_t q) {
  if (row >= rows) return 0x7f7f7f7fu;
  return *reinterpret_cast<const uint32_t*>(s + (tile == 1 ? row : row / kFp8Block) * ld + 4 * q);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
matmul_kernel(const __grid_constant__ MatmulMaps maps, MatmulArgs a) {
  extern __shared__ unsigned char smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  volatile uint32_t* abort_flag =
      reinterpret_cast<volatile uint32_t*>(smem_raw + (base - smem_u32(smem_raw)) + kAbort);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t tiles_n = (a.N + kTileN - 1) / kTileN;
  const int64_t m0 = blockIdx.x / tiles_n * kTileM, n0 = blockIdx.x % tiles_n * kTileN;
  const int kb = static_cast<int>((a.K + kFp8Block - 1) / kFp8Block);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(base + kFull + 8 * s, 1);
      mbar_init(base + kEmpty + 8 * s, 1);
    }
    for (int s = 0; s < kScaleBufs; ++s) {
      mbar_init(base + kSFull + 8 * s, 1);
      mbar_init(base + kSEmpty + 8 * s, 1);
    }
    mbar_init(base + kDone, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(base + kSlot, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = lds_u32(base + kSlot);
  grid_launch_dependents();
  grid_dependency_wait();

  if (warp == 0) {
    if (lane == 0) {
      prefetch_map(&maps.a);
      prefetch_map(&maps.b);
      uint64_t policy;
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
      int i = 0;
      for (; i < kb; ++i) {
        const int s = i % kStages;
        if (!wait_here(base + kEmpty + 8 * s, ((i / kStages) & 1u) ^ 1u, abort_flag)) break;
        const uint32_t st = base + kSmemStages + s * kStageBytes;
        mbar_arrive_expect_tx(base + kFull + 8 * s, kStageBytes);
        tma_load_2d(st, &maps.a, i * kFp8Block, static_cast<int>(m0), base + kFull + 8 * s, policy);
        tma_load_2d(st + kTileM * kFp8Block, &maps.b, i * kFp8Block, static_cast<int>(n0),
                    base + kFull + 8 * s, policy);
      }
      if (i < kb)   // copies still in flight land before the CTA exits
        for (int j = i > kStages ? i - kStages : 0; j < i; ++j)
          mbar_wait(base + kFull + 8 * (j % kStages), (j / kStages) & 1u);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      bool ok = true;
      for (int i = 0; i < kb && ok; ++i) {
        const int s = i % kStages, q = i / kChunk, j = i % kChunk, sb = q % kScaleBufs;
        ok = wait_here(base + kFull + 8 * s, (i / kStages) & 1u, abort_flag);
        if (ok && j == 0) ok = wait_here(base + kSFull + 8 * sb, (q / kScaleBufs) & 1u, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sfa = tmem + kColScales + 8 * (q % kTmemScaleBufs), sfb = sfa + 4;
        if (j == 0) {
          const uint32_t sc = base + kSmemScales + sb * kScaleBytes;
          tmem_copy_scales(sfa, sc);
          tmem_copy_scales(sfb, sc + 4 * kTileM);
          mma_commit(base + kSEmpty + 8 * sb);
        }
        const uint32_t st = base + kSmemStages + s * kStageBytes;
        const uint32_t idesc = kDesc | (static_cast<uint32_t>(j) << 29) | (static_cast<uint32_t>(j) << 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_mx(tmem, umma_desc(st + 32 * kk, kSwizzle128, 1024),
                 umma_desc(st + kTileM * kFp8Block + 32 * kk, kSwizzle128, 1024), idesc, sfa,
                 sfb, (i | kk) != 0);
        mma_commit(base + kEmpty + 8 * s);
      }
      mma_commit(base + kDone);
      mbar_wait(base + kDone, 0);   // nothing in flight when the tensor memory is freed
    }
    __syncwarp();
  } else if (warp == 2) {
    const int chunks = (kb + kChunk - 1) / kChunk;
    bool ok = true;
    for (int q = 0; q < chunks && ok; ++q) {
      const int sb = q % kScaleBufs;
      ok = wait_here(base + kSEmpty + 8 * sb, ((q / kScaleBufs) & 1u) ^ 1u, abort_flag);
      ok = __all_sync(kFullMask, ok);
      if (!ok) break;
      const uint32_t sc = base + kSmemScales + sb * kScaleBytes;
#pragma unroll
      for (int r = 0; r < kTileM; r += 32)
        asm volatile("st.shared.u32 [%0], %1;" :: "r"(sc + lane * 16 + r / 8),
                     "r"(scale_word(a.sa, a.lda_s, m0 + r + lane, a.M, a.tile_a, q)) : "memory");
#pragma unroll
      for (int r = 0; r < kTileN; r += 32)
        asm volatile("st.shared.u32 [%0], %1;" :: "r"(sc + 4 * kTileM + lane * 16 + r / 8),
                     "r"(scale_word(a.sb, a.ldb_s, n0 + r + lane, a.N, a.tile_b, q)) : "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(base + kSFull + 8 * sb);
    }
  } else if (warp >= 4) {
    const int quad = warp & 3;
    const int64_t m = m0 + quad * 32 + lane;
    const bool got = wait_here(base + kDone, 0, abort_flag) && *abort_flag == 0u;
    tc_fence_after();
    const bool all = __all_sync(kFullMask, got);
    if (all)
      for (int c = 0; c < kTileN; c += 16) {
        float v[16];
        tmem_ld16(tmem + (static_cast<uint32_t>(quad * 32) << 16) + c, v);
        tmem_wait_ld();
        reg_fence16(v);
        if (m < a.M)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int64_t n = n0 + c + i;
            if (n < a.N) {
              float r = v[i];
              if (a.add) r += to_f32(static_cast<const T*>(a.add)[m * a.ldadd + n]);
              static_cast<T*>(a.out)[m * a.ldo + n] = from_f32<T>(r);
            }
          }
      }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

bool encode_codes(EncodeTiled encode, CUtensorMap* map, const uint8_t* p, int64_t rows, int64_t cols,
                  int64_t ld, int box_rows) {
  const cuuint64_t dim[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t stride[1] = {static_cast<cuuint64_t>(ld)};
  const cuuint32_t box[2] = {kFp8Block, static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t unit[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(p), dim, stride, box, unit,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t prepare_matmul() {
  cudaError_t e = cudaSuccess;
  for (const void* k : {reinterpret_cast<const void*>(matmul_kernel<__nv_bfloat16>),
                        reinterpret_cast<const void*>(matmul_kernel<__half>),
                        reinterpret_cast<const void*>(matmul_kernel<float>)})
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes));
  return e;
}

cudaError_t launch_matmul(const MatmulArgs& a, int dtype, int sms, cudaStream_t st) {
  (void)sms;
  EncodeTiled encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
  MatmulMaps maps;
  if (!encode_codes(encode, &maps.a, a.a, a.M, a.K, a.lda, kTileM) ||
      !encode_codes(encode, &maps.b, a.b, a.N, a.K, a.ldb, kTileN))
    return cudaErrorInvalidValue;
  const int64_t tiles = ((a.M + kTileM - 1) / kTileM) * ((a.N + kTileN - 1) / kTileN);
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    return launch_dependent(matmul_kernel<T>, dim3(static_cast<unsigned>(tiles)), kThreads, kSmemBytes, st, maps, a);
  });
}

cudaError_t matmul_fault(unsigned int* bits, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(bits, g_fp8_matmul_fault, sizeof(unsigned int));
  if (e == cudaSuccess && clear) {
    const unsigned int zero = 0;
    e = cudaMemcpyToSymbol(g_fp8_matmul_fault, &zero, sizeof(unsigned int));
  }
  return e;
}

}  // namespace taco
