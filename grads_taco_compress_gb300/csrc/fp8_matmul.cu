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
// Two kernels: pairs of CTAs on 256-row tiles (matmul_pair_kernel) and, for few
// rows of A, the roles of A and B exchanged and K split over a cluster
// (matmul_few_kernel). Both have 8 warps:
//   warp 0     TMA producer: blocks of 128 columns of K, rows of 128 bytes in
//              the 128-byte swizzle;
//   warp 1     owns the tensor memory; one lane copies the scales to tensor
//              memory, issues the MMAs and commits each stage;
//   warp 2     (and 3, in pairs) scales: every chunk of 4 blocks (512 columns)
//              one 32-bit word per row of A and B, byte j the scale of block j,
//              in the order that tcgen05.cp 32x128b spreads over the tensor
//              memory;
//   warps 4-7  epilogue: lane = row, tensor memory to registers to C.
// Every wait is bounded in time with a CTA-wide abort flag.
//
// Measured (twice the measured bf16 rate of a library product is 3.94 PFLOP/s):
// 16384 x 4096 x 3584 to bf16 136 us, 3.53 PFLOP/s, tensor pipe 80% active, and
// 157 us (3.06 PFLOP/s) in a second-long loop under the power limit; the MMAs
// without copies 120 us, the copies without MMAs 89 us: both go through shared
// memory, 32 KB in and 32 KB or more out a block of 128 columns. 1600 x 4096 x
// 8190 to f32 with add 54 us, 2.0 PFLOP/s, pipe 48%: a tile 128 columns wide
// moves a third more bytes a product, and 224 tiles are 2.95 waves of pairs.
// Few rows: 8 x 4096 x 4096 6.5 us over weights that come from memory, whose 16.8
// MB would take 2.5, and 5.5 us where they are in L2 from the call before; 1 x
// 16384 x 4096 13.6 us, 4.9 TB/s.

#include "fp8_block.cuh"
#include "tcgen05.cuh"

namespace taco {

namespace {

__device__ unsigned int g_fp8_matmul_fault;

constexpr int kThreads = 256;
constexpr int kChunk = 4;   // blocks of 128 columns per word of scales

// Instruction descriptor of kind::mxf8f6f4 with E4M3 operands, K-major, E8M0
// scales: N >> 3 at bits 17-22, scale type at bit 23, M >> 7 at bits 27-28;
// the byte of the scale word at bits 29-30 (A) and 4-5 (B).
constexpr uint32_t mx_desc(uint32_t m, uint32_t n) {
  return ((n >> 3) << 17) | (1u << 23) | ((m >> 7) << 27);
}
constexpr uint32_t kDescPair256 = mx_desc(256, 256), kDescPair128 = mx_desc(256, 128);
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
// The same on a barrier that the other CTA of a pair arrives at.
__device__ __forceinline__ bool wait_pair(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag) {
  return wait_or_abort<true>(bar, parity, abort_flag, &g_fp8_matmul_fault, kFaultFp8MatmulWait);
}

struct MatmulMaps {
  CUtensorMap a, b;
};

// 16 bytes of outputs from fp32.
template <typename T>
__device__ __forceinline__ uint4 pack16(const float* v) {
  if constexpr (std::is_same<T, float>::value) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  } else if constexpr (std::is_same<T, __half>::value) {
    __half2 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    return *reinterpret_cast<const uint4*>(h);
  } else {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
  }
}
template <typename T>
__device__ __forceinline__ T load_staged(uint32_t addr) {
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(lds_u32(addr));
  } else {
    uint16_t r;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(addr));
    T v;
    memcpy(&v, &r, 2);
    return v;
  }
}
// v += the `left` (or COLS) elements of a row of `add`; vec: rows of it start on
// 16 bytes (and p on as many as COLS elements take, at most 16).
template <typename T, int COLS>
__device__ __forceinline__ void add_row(float* v, const T* p, int64_t left, bool vec) {
  constexpr int kPer = COLS * static_cast<int>(sizeof(T)) < 16 ? COLS : 16 / static_cast<int>(sizeof(T));
  if (vec && left >= COLS) {
#pragma unroll
    for (int i = 0; i < COLS; i += kPer) {
      alignas(16) T q[kPer];
      if constexpr (kPer * sizeof(T) == 16)
        *reinterpret_cast<uint4*>(q) = *reinterpret_cast<const uint4*>(p + i);
      else
        *reinterpret_cast<uint2*>(q) = *reinterpret_cast<const uint2*>(p + i);
#pragma unroll
      for (int e = 0; e < kPer; ++e) v[i + e] += to_f32(q[e]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < COLS; ++i)
      if (i < left) v[i] += to_f32(p[i]);
  }
}

// 4 consecutive outputs, of which `left` exist.
template <typename T>
__device__ __forceinline__ void store_row4(T* p, const float* v, int64_t left, bool vec) {
  if (vec && left >= 4) {
    alignas(16) T q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = from_f32<T>(v[i]);
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(q);
    else
      *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(q);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) p[i] = from_f32<T>(v[i]);
  }
}

// One lane of a converged warp, always the same. The warps that issue copies
// and MMAs run their loops with all lanes, so that counters, addresses and
// descriptors stay in uniform registers, and only the instruction itself is
// left to this lane: with the whole loop in one lane the operands of every MMA
// went through vector registers and the issue, not the tensor cores, set the
// pace (1000 cycles a stage at either tile width).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(kFullMask, v, 0); }

// The scale words of one row for chunks 4 g .. 4 g + 3 (16 blocks). Bytes
// beyond the row's last block are whatever lies there and are never used. vec:
// the rows of scales start on 16 bytes.
struct ScaleRows {
  const uint8_t* p;
  int64_t ld, rows;
  int tile, chunks;
  bool vec;
  __device__ __forceinline__ uint4 at(int64_t row, int g) const {
    if (row >= rows) return make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
    const uint8_t* s = p + (tile == 1 ? row : row / kFp8Block) * ld + 16 * g;
    if (vec) return *reinterpret_cast<const uint4*>(s);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(s);
    const int n = chunks - 4 * g;
    return make_uint4(w[0], n > 1 ? w[1] : 0u, n > 2 ? w[2] : 0u, n > 3 ? w[3] : 0u);
  }
};
__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
__device__ __forceinline__ void sts_words(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  sts128(addr, make_uint4(a, b, c, d));
}

// ------------------------------------------------------------ CTA pairs ----
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of `addr` in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// An arrival on the barrier `bar` (this CTA's address) of the even CTA of the
// pair, behind everything that the thread has written or seen written. From the
// odd CTA it is a release at cluster scope, which the barrier's waiter acquires
// at that scope (wait_pair); such a release takes about a microsecond, and
// longer where the thread has loads in flight.
__device__ __forceinline__ void arrive_even(uint32_t bar, uint32_t even_bar, uint32_t rank) {
  if (rank == 0)
    mbar_arrive(bar);
  else
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(even_bar) : "memory");
}
// The same for accumulators that this warp has read. No memory is announced, and
// the fence of the tensor-memory loads (tc_fence_before) orders them before any
// execution-ordering operation, so the arrival needs no release, whose latency
// would lie between the tiles (16384 x 4096 x 3584: 136 us, 142 with a release;
// f32, 8192 x 4096 x 8192: 213 and 224).
__device__ __forceinline__ void arrive_even_read(uint32_t even_bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" :: "r"(even_bar) : "memory");
}
__device__ __forceinline__ void tma_load_2d_plain(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar) : "memory");
}
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int c0, int c1) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];"
               :: "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1) : "memory");
}
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];"
      :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar) : "memory");
}
__device__ __forceinline__ void mma_mx_pair(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale [%0], %1, %2, %3, [%5], [%6], p;\n}"
      :: "r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb) : "memory");
}
__device__ __forceinline__ void tmem_copy_scales_pair(uint32_t taddr, uint32_t saddr) {
  const uint64_t desc = umma_desc(saddr, 0, 128);
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" :: "r"(taddr), "l"(desc) : "memory");
}
// One arrival on the barrier at this offset in both CTAs once every tcgen05
// operation this thread has issued so far has completed.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
      :: "r"(bar), "h"(static_cast<uint16_t>(3)) : "memory");
}
// The same on this CTA's barrier alone.
__device__ __forceinline__ void commit_here(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(bar) : "memory");
}
// How long the odd CTA of a pair that gives up waits for copies that it has
// issued: thousands of times what one takes.
constexpr unsigned long long kDrainNs = 10ull * 1000ull * 1000ull;
// 32 consecutive fp32 columns of this thread's lane, without the wait.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  tmem_ld16(taddr, v);
  tmem_ld16(taddr + 16, v + 16);
}
__device__ __forceinline__ void tmem_ready32(float (&v)[32]) {
  tmem_wait_ld();
  reg_fence16(v);
  reg_fence16(v + 16);
}

// Output tile t of the persistent grid: bands of 8 row tiles, all column
// tiles of a band before the next, so that the tiles in flight at one time
// share rows of A and of B in L2.
constexpr int64_t kBand = 8;
struct TileMap {
  int64_t tiles_m, tiles_n;
  __device__ __forceinline__ void at(int64_t t, int64_t& mt, int64_t& nt) const {
    const int64_t per = kBand * tiles_n, band = t / per, in = t - band * per;
    const int64_t left = tiles_m - band * kBand, size = left < kBand ? left : kBand;
    nt = in / size;
    mt = band * kBand + (in - nt * size);
  }
};

// Chunks whose scale words may wait in shared memory: two groups of 4, one of
// either warp that brings them. A warp stalls for the latency of its loads and
// of the release to the other CTA once a group, and the other group (16 blocks)
// covers it (a release a chunk, the next loads in front of it, took 1% more for
// 16384 x 4096 x 3584 and 4% for f32, 8192 x 4096 x 8192).
constexpr int kScaleBufs = 8;

template <int TN>
struct Pair {
  // A stage is two blocks of K: with one, the issuing warp's barrier traffic
  // (140 ns a stage with nothing else to do) is longer than the MMAs at TN = 128.
  static constexpr int kStages = 3;
  static constexpr uint32_t kA = 128 * kFp8Block, kB = TN / 2 * kFp8Block, kBlock = kA + kB, kStage = 2 * kBlock;
  static constexpr uint32_t kScale = (128 + TN) * 4;       // scale words of one chunk
  static constexpr uint32_t stages = 0;
  // Staging of the outputs, boxes of 32 rows x 128 bytes: one for each of the 4
  // epilogue warps, and at TN = 128 (f32) all 4 of a warp's rows, which `add`
  // is copied to while the sums are formed.
  static constexpr uint32_t kBoxes = TN == 128 ? 4 : 1;
  static constexpr uint32_t staging = kStages * kStage;
  static constexpr uint32_t scales = staging + 4 * kBoxes * 4096;
  static constexpr uint32_t full = scales + kScaleBufs * kScale;
  static constexpr uint32_t empty = full + 8 * kStages;
  // scale words of a chunk: in shared memory; copied to tensor memory; read by
  // the last MMA of the chunk, whose set of scale columns is free
  static constexpr uint32_t sfull = empty + 8 * kStages;
  static constexpr uint32_t sempty = sfull + 8 * kScaleBufs;
  static constexpr uint32_t sdone = sempty + 8 * kScaleBufs;
  static constexpr uint32_t tfull = sdone + 16;
  static constexpr uint32_t tempty = tfull + 16;
  static constexpr uint32_t added = tempty + 16;              // `add` has landed in a warp's staging
  static constexpr uint32_t done = added + 32;
  static constexpr uint32_t slot = done + 8;
  static constexpr uint32_t abort_flag = slot + 4;
  static constexpr uint32_t bytes = abort_flag + 4 + 1024;
  static_assert(bytes <= 232448, "shared memory per CTA");
  // Tensor memory: two accumulators of TN columns and two sets of scale words
  // (4 columns of A's, TN / 32 of B's). At TN = 256 the accumulators share 32
  // columns (224 - 255), which the epilogue reads first.
  static constexpr uint32_t kAcc1 = TN == 256 ? 224 : TN;
  static constexpr uint32_t kColScales = TN == 256 ? 480 : 2 * TN;
  static constexpr uint32_t kScaleCols = 4 + TN / 32;
  static_assert(kColScales + 2 * kScaleCols <= 512, "tensor memory");
};

// Two CTAs, one 256 x TN output tile: CTA r holds rows 128 r .. of A, the r-th
// half of B's TN rows and accumulator rows 128 r .. ; the even CTA issues the
// MMAs of both. Persistent: pair p takes tiles p, p + pairs, ...; a tile's
// epilogue overlaps the next one's MMAs. SEG: the sum over K is formed in
// segments of kSegment blocks, each started from zero in tensor memory, that
// the epilogue adds in registers: the tensor cores cut, not round, what falls
// below an accumulator's last bit, and a long sum drifts.
constexpr int kSegment = 8;

template <typename T, int TN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
matmul_pair_kernel(const __grid_constant__ MatmulMaps maps, const __grid_constant__ CUtensorMap out_map,
                   const __grid_constant__ CUtensorMap add_map, MatmulArgs a) {
  using S = Pair<TN>;
  constexpr bool kSeg = std::is_same<T, float>::value;
  static_assert(!kSeg || TN == 128, "the segments' sum is held in registers");
  extern __shared__ unsigned char smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  volatile uint32_t* abort_flag =
      reinterpret_cast<volatile uint32_t*>(smem_raw + (base - smem_u32(smem_raw)) + S::abort_flag);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const TileMap tm{(a.M + 255) / 256, (a.N + TN - 1) / TN};
  const int64_t tiles = tm.tiles_m * tm.tiles_n;
  const int kb = static_cast<int>((a.K + kFp8Block - 1) / kFp8Block);
  const int chunks = (kb + kChunk - 1) / kChunk;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(base + S::full + 8 * s, 1);
      mbar_init(base + S::empty + 8 * s, 1);
    }
    for (int s = 0; s < kScaleBufs; ++s) {
      mbar_init(base + S::sfull + 8 * s, 2);    // one scale warp of each CTA
      mbar_init(base + S::sempty + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(base + S::sdone + 8 * s, 1);
      mbar_init(base + S::tfull + 8 * s, 1);
      mbar_init(base + S::tempty + 8 * s, 8);   // 4 epilogue warps of both CTAs
    }
    for (int w = 0; w < 4; ++w) mbar_init(base + S::added + 8 * w, 1);
    mbar_init(base + S::done, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;"
                 :: "r"(base + S::slot) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the other CTA's barriers are initialised
  tc_fence_after();
  const uint32_t tmem = uniform(lds_u32(base + S::slot));
  grid_launch_dependents();
  grid_dependency_wait();

  if (warp == 0) {
    // ---------------------------------------------------- TMA producer ----
    const bool leader = elect_one();
    if (leader) {
      prefetch_map(&maps.a);
      prefetch_map(&maps.b);
    }
    // both CTAs' copies count on the even CTA's barriers
    const uint32_t full0 = uniform(in_cta(base + S::full, 0));
    uint32_t s = 0, ph = 0, issued = 0;
    bool ok = true;
    for (int64_t t = pair; t < tiles && ok; t += pairs) {
      int64_t mt, nt;
      tm.at(t, mt, nt);
      const int row_a = static_cast<int>(mt * 256 + rank * 128);
      const int row_b = static_cast<int>(nt * TN + rank * (TN / 2));
      for (int k = 0; k < kb; k += 2) {
        ok = wait_pair(base + S::empty + 8 * s, ph ^ 1u, abort_flag);
        ok = __all_sync(kFullMask, ok);
        if (!ok) break;
        const uint32_t st = base + S::stages + s * S::kStage, bar = full0 + 8 * s;
        if (leader) {
          const bool two = k + 1 < kb;
          if (rank == 0) mbar_arrive_expect_tx(base + S::full + 8 * s, two ? 2 * S::kStage : S::kStage);
          tma_load_pair(st, &maps.a, k * kFp8Block, row_a, bar);
          tma_load_pair(st + S::kA, &maps.b, k * kFp8Block, row_b, bar);
          if (two) {
            tma_load_pair(st + S::kBlock, &maps.a, (k + 1) * kFp8Block, row_a, bar);
            tma_load_pair(st + S::kBlock + S::kA, &maps.b, (k + 1) * kFp8Block, row_b, bar);
          }
        }
        ++issued;
        if (++s == S::kStages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    if (!ok && rank == 0) {   // copies still in flight land before the CTAs exit
      const uint32_t first = issued > static_cast<uint32_t>(S::kStages) ? issued - S::kStages : 0u;
      for (uint32_t j = first; j < issued; ++j) mbar_wait(base + S::full + 8 * (j % S::kStages), (j / S::kStages) & 1u);
    } else if (!ok) {   // the odd CTA's, of which it may have issued more, count where it cannot wait
      const unsigned long long t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < kDrainNs) __nanosleep(1000);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA issuer ----
    if (rank == 0) {
      const bool leader = elect_one();
      const uint64_t adesc0 = umma_desc(base + S::stages, kSwizzle128, 1024);
      const uint64_t bdesc0 = umma_desc(base + S::stages + S::kA, kSwizzle128, 1024);
      uint32_t s = 0, ph = 0, q = 0, u = 0;   // stage and its phase; scale chunks and accumulators used so far
      bool ok = true;
      for (int64_t t = pair; t < tiles && ok; t += pairs) {
        for (int k = 0; k < kb; k += 2) {
          const uint32_t j = k % kChunk, sb = q % kScaleBufs;
          const bool first = kSeg ? k % kSegment == 0 : k == 0;
          const bool last = k + 2 >= kb || (kSeg && (k + 2) % kSegment == 0);
          if (first) {
            // the accumulator is free, and so are the columns it shares
            const uint32_t before = TN == 256 ? 1u : 2u;
            if (u >= before)
              ok = wait_pair(base + S::tempty + 8 * ((u - before) & 1u), ((u - before) >> 1) & 1u, abort_flag);
          }
          if (ok && j == 0) {
            ok = wait_pair(base + S::sfull + 8 * sb, (q / kScaleBufs) & 1u, abort_flag);
            if (ok && q >= 2) ok = wait_here(base + S::sdone + 8 * (q & 1u), ((q - 2) >> 1) & 1u, abort_flag);
          }
          if (ok) ok = wait_pair(base + S::full + 8 * s, ph, abort_flag);
          ok = __all_sync(kFullMask, ok);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sfa = tmem + S::kColScales + (q & 1u) * S::kScaleCols, sfb = sfa + 4;
          const uint32_t d = tmem + (u & 1u) * S::kAcc1;
          const uint32_t idesc = (TN == 256 ? kDescPair256 : kDescPair128) | (j << 29) | (j << 4);
          const uint64_t adesc = adesc0 + s * (S::kStage >> 4), bdesc = bdesc0 + s * (S::kStage >> 4);
          const uint32_t sc = base + S::scales + sb * S::kScale;
          const bool end = j == kChunk - 2 || k + 2 >= kb;
          if (leader) {
            if (j == 0) {
              tmem_copy_scales_pair(sfa, sc);
#pragma unroll
              for (int g = 0; g < TN / 128; ++g) tmem_copy_scales_pair(sfb + 4 * g, sc + 512 * (g + 1));
              commit_pair(base + S::sempty + 8 * sb);
            }
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)   // 32 columns: 2 units of 16 bytes further on
              mma_mx_pair(d, adesc + 2 * kk, bdesc + 2 * kk, idesc, sfa, sfb, !first || kk > 0);
            if (k + 1 < kb) {
              const uint32_t next = idesc + ((1u << 29) | (1u << 4));   // the scale words' next byte
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_mx_pair(d, adesc + (S::kBlock >> 4) + 2 * kk, bdesc + (S::kBlock >> 4) + 2 * kk, next, sfa, sfb,
                            1u);
            }
            commit_pair(base + S::empty + 8 * s);
            if (end) commit_here(base + S::sdone + 8 * (q & 1u));
            if (last) commit_pair(base + S::tfull + 8 * (u & 1u));
          }
          if (end) ++q;
          if (last) ++u;
          if (++s == S::kStages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (leader) {
        commit_here(base + S::done);
        mbar_wait(base + S::done, 0);   // nothing in flight when the tensor memory is freed
      }
    }
    __syncwarp();
  } else if (warp <= 3) {
    // ---------------------------------------------------------- scales ----
    // The words of 4 chunks (a group) are read together; the two warps take
    // the pair's groups in turn and read their next one ahead of its use.
    const ScaleRows ra{a.sa, a.lda_s, a.M, a.tile_a, chunks, a.vec_sa};
    const ScaleRows rb{a.sb, a.ldb_s, a.N, a.tile_b, chunks, a.vec_sb};
    const int groups = (chunks + 3) / 4;
    uint4 na[4], nb[TN / 32];
    int64_t t = pair;      // group g of tile t, whose first chunk is number q of the pair
    int g = 0;
    uint32_t q = 0;
    const auto advance = [&]() {
      q += chunks - 4 * g < 4 ? chunks - 4 * g : 4;
      if (++g == groups) {
        g = 0;
        t += pairs;
      }
    };
    const auto fetch = [&]() {
      int64_t mt, nt;
      tm.at(t, mt, nt);
#pragma unroll
      for (int r = 0; r < 4; ++r) na[r] = ra.at(mt * 256 + rank * 128 + r * 32 + lane, g);
#pragma unroll
      for (int r = 0; r < TN / 32; ++r) nb[r] = rb.at(nt * TN + r * 32 + lane, g);
    };
    const uint32_t sfull0 = in_cta(base + S::sfull, 0);
    bool ok = true;
    if (warp == 3) advance();
    if (t < tiles) fetch();
    while (t < tiles && ok) {
      uint4 wa[4], wb[TN / 32];
#pragma unroll
      for (int r = 0; r < 4; ++r) wa[r] = na[r];
#pragma unroll
      for (int r = 0; r < TN / 32; ++r) wb[r] = nb[r];
      const uint32_t q0 = q;
      const int here = chunks - 4 * g < 4 ? chunks - 4 * g : 4;
      advance();
      if (t < tiles) advance();
      for (int j = 0; j < here && ok; ++j) {
        const uint32_t use = q0 + j;
        ok = wait_pair(base + S::sempty + 8 * (use % kScaleBufs), ((use / kScaleBufs) & 1u) ^ 1u, abort_flag);
      }
      ok = __all_sync(kFullMask, ok);
      if (!ok) break;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j >= here) break;
        const uint32_t sc = base + S::scales + ((q0 + j) % kScaleBufs) * S::kScale + lane * 16;
        sts_words(sc, word_of(wa[0], j), word_of(wa[1], j), word_of(wa[2], j), word_of(wa[3], j));
#pragma unroll
        for (int n = 0; n < TN / 128; ++n)
          sts_words(sc + 512 * (n + 1), word_of(wb[4 * n], j), word_of(wb[4 * n + 1], j), word_of(wb[4 * n + 2], j),
                    word_of(wb[4 * n + 3], j));
      }
      fence_proxy_async_smem();
      __syncwarp();
      // the group's chunks by one release, a lane each, and the next loads behind it
      if (lane < here) {
        const uint32_t at = 8 * ((q0 + lane) % kScaleBufs);
        arrive_even(base + S::sfull + at, sfull0 + at, rank);
      }
      if (t < tiles) fetch();
    }
  } else if (warp >= 4) {
    // -------------------------------------------------------- epilogue ----
    const int quad = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t staging = base + S::staging + quad * (S::kBoxes * 4096);
    const bool tma_add = kSeg && a.add && a.tma_add;
    const uint32_t tempty0 = in_cta(base + S::tempty, 0);
    constexpr int kCols = 128 / static_cast<int>(sizeof(T));   // columns of one 128-byte staging row
    if (lane == 0 && a.tma_out) prefetch_map(&out_map);
    if (lane == 0 && tma_add) prefetch_map(&add_map);
    uint32_t u = 0, adds = 0;
    bool ok = true;
    for (int64_t t = pair; t < tiles && ok; t += pairs) {
      int64_t mt, nt;
      tm.at(t, mt, nt);
      const int64_t m0 = mt * 256 + rank * 128 + quad * 32, n0 = nt * TN;
      const int boxes = m0 >= a.M ? 0 : static_cast<int>(a.N - n0 < TN ? (a.N - n0 + kCols - 1) / kCols : TN / kCols);
      if (kSeg && lane == 0) {
        bulk_wait_read<0>();   // the last tile's stores have read the staging
        if (tma_add && boxes > 0) {
          const uint32_t bar = base + S::added + 8 * quad;
          mbar_arrive_expect_tx(bar, boxes * 4096);
          for (int c = 0; c < boxes; ++c)
            tma_load_2d_plain(staging + c * 4096, &add_map, static_cast<int>(n0) + c * kCols, static_cast<int>(m0),
                              bar);
        }
      }
      __syncwarp();
      float sum[kSeg ? TN : 1];
      if constexpr (kSeg) {
        const int segments = (kb + kSegment - 1) / kSegment;
#pragma unroll
        for (int c = 0; c < TN; ++c) sum[c] = 0.0f;
        for (int g = 0; g < segments && ok; ++g, ++u) {
          ok = wait_pair(base + S::tfull + 8 * (u & 1u), (u >> 1) & 1u, abort_flag) && *abort_flag == 0u;
          ok = __all_sync(kFullMask, ok);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < TN; c += 32) {
            float v[32];
            tmem_ld32(tmem + lanes + (u & 1u) * S::kAcc1 + c, v);
            tmem_ready32(v);
#pragma unroll
            for (int i = 0; i < 32; ++i) sum[c + i] += v[i];
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive_even_read(tempty0 + 8 * (u & 1u));
        }
      } else {
        ok = wait_pair(base + S::tfull + 8 * (u & 1u), (u >> 1) & 1u, abort_flag) && *abort_flag == 0u;
        ok = __all_sync(kFullMask, ok);
      }
      if (tma_add && boxes > 0) {
        // the copy ends in bounded time whether or not the sums arrived
        const bool landed = wait_here(base + S::added + 8 * quad, adds++ & 1u, abort_flag);
        ok = __all_sync(kFullMask, landed) && ok;
      }
      if (!ok) break;
      if constexpr (!kSeg) tc_fence_after();
      const uint32_t acc = tmem + lanes + (u & 1u) * S::kAcc1;
#pragma unroll
      for (int c = 0; c < TN / kCols; ++c) {
        // the shared columns first: the last ones of accumulator 0, the first of accumulator 1
        const int chunk = (TN == 256 && (u & 1u) == 0) ? (c + TN / kCols - 1) % (TN / kCols) : c;
        float v[kCols];
        if constexpr (kSeg) {
#pragma unroll
          for (int i = 0; i < kCols; ++i) v[i] = sum[c * kCols + i];
        } else {
#pragma unroll
          for (int i = 0; i < kCols; i += 16) tmem_ld16(acc + chunk * kCols + i, v + i);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < kCols; i += 16) reg_fence16(v + i);
          if (c == (TN == 256 ? 0 : TN / kCols - 1)) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_even_read(tempty0 + 8 * (u & 1u));
          }
        }
        const int64_t m = m0 + lane, n = n0 + static_cast<int64_t>(chunk) * kCols;
        // staging: 32 rows of 128 bytes, 16-byte pieces permuted by row & 7
        const uint32_t box = staging + (kSeg ? c * 4096 : 0), row = box + lane * 128;
        if (tma_add) {
          if constexpr (kSeg)
#pragma unroll
            for (int p = 0; p < 8; ++p) {
              const uint4 w = lds128(row + 16 * (p ^ (lane & 7)));
              v[4 * p] += __uint_as_float(w.x);
              v[4 * p + 1] += __uint_as_float(w.y);
              v[4 * p + 2] += __uint_as_float(w.z);
              v[4 * p + 3] += __uint_as_float(w.w);
            }
        } else if (a.add && m < a.M) {
          add_row<T, kCols>(v, static_cast<const T*>(a.add) + m * a.ldadd + n, a.N - n, a.vec_add);
        }
        if (!kSeg) {
          if (lane == 0) bulk_wait_read<0>();   // the last store has read it
          __syncwarp();
        }
#pragma unroll
        for (int p = 0; p < 8; ++p) sts128(row + 16 * (p ^ (lane & 7)), pack16<T>(v + p * (kCols / 8)));
        // a tensor copy to memory ends on 16 bytes and takes what lies behind the row
        // with it, so rows that end elsewhere are finished by plain stores
        if (a.tma_out && (n + kCols <= a.N || ((a.N - n) * static_cast<int>(sizeof(T))) % 16 == 0)) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && m0 < a.M && n < a.N) {
            tma_store_2d(&out_map, box, static_cast<int>(n), static_cast<int>(m0));
            bulk_commit();
          }
        } else {
          __syncwarp();
          for (int r = 0; r < 32; ++r) {
            if (m0 + r >= a.M) break;
            T* p = static_cast<T*>(a.out) + (m0 + r) * a.ldo + n;
#pragma unroll
            for (int e = lane; e < kCols; e += 32)
              if (n + e < a.N)
                p[e] = load_staged<T>(box + r * 128 + 16 * (((e * static_cast<int>(sizeof(T))) >> 4) ^ (r & 7)) +
                                      ((e * sizeof(T)) & 15));
          }
          if (kSeg) fence_proxy_async_smem();   // the next tile's `add` is copied over what was read here
          __syncwarp();
        }
      }
      if constexpr (!kSeg) ++u;
    }
    if (lane == 0) bulk_wait_read<0>();   // every store has read the staging
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // the other CTA is done with this one's barriers and shared memory
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" :: "r"(tmem) : "memory");
  }
}

// -------------------------------------------------------------- few rows ----
// C with few rows of A ("tokens"): the 128 rows of one MMA are rows of B
// (weights), TT tokens its columns, and the blocks of K are split over the CTAs
// of a cluster, each of which reads its own part of the weights once. The
// partial sums meet through distributed shared memory: every CTA adds the
// parts of its tokens in the order of the splits and writes them.
constexpr int kMaxSplits = 8;   // the portable cluster size

template <int TT>
struct Few {
  static constexpr uint32_t kW = 128 * kFp8Block, kX = TT * kFp8Block, kStage = kW + kX;
  static constexpr int kStages = TT <= 16 ? 10 : TT == 32 ? 9 : TT == 64 ? 7 : 6;
  static constexpr uint32_t kScale = 1024;                 // words of 128 weight rows and 128 token rows
  static constexpr uint32_t stages = 0;                    // and then the partial sums, [token][128] fp32
  static constexpr uint32_t scales = kStages * kStage;
  static constexpr uint32_t full = scales + 2 * kScale;
  static constexpr uint32_t empty = full + 8 * kStages;
  static constexpr uint32_t sfull = empty + 8 * kStages;
  static constexpr uint32_t sempty = sfull + 16;
  static constexpr uint32_t tfull = sempty + 16;
  static constexpr uint32_t tempty = tfull + 16;
  static constexpr uint32_t done = tempty + 16;
  static constexpr uint32_t slot = done + 8;
  static constexpr uint32_t abort_flag = slot + 4;
  static constexpr uint32_t bytes = abort_flag + 4 + 1024;
  static_assert(bytes <= 232448 && kStages * kStage >= TT * 128 * 4, "shared memory per CTA");
  static constexpr uint32_t kTmemCols = TT <= 16 ? 64 : TT == 32 ? 128 : TT == 64 ? 256 : 512;
  static constexpr uint32_t kColScales = 2 * TT;
  static_assert(kColScales + 16 <= kTmemCols, "tensor memory");
};

template <typename T, int TT>
__global__ void __launch_bounds__(kThreads, 1)
matmul_few_kernel(const __grid_constant__ MatmulMaps maps, MatmulArgs a, int splits) {
  using S = Few<TT>;
  constexpr bool kSeg = std::is_same<T, float>::value;
  constexpr uint32_t kDesc = ((TT >> 3) << 17) | (1u << 23) | (1u << 27);   // mx_desc(128, TT)
  extern __shared__ unsigned char smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  volatile uint32_t* abort_flag =
      reinterpret_cast<volatile uint32_t*>(smem_raw + (base - smem_u32(smem_raw)) + S::abort_flag);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int64_t n0 = static_cast<int64_t>(blockIdx.x / splits) * 128;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * TT;
  const int kb = static_cast<int>((a.K + kFp8Block - 1) / kFp8Block);
  const int k0 = static_cast<int>(static_cast<int64_t>(kb) * rank / splits);
  const int k1 = static_cast<int>(static_cast<int64_t>(kb) * (rank + 1) / splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(base + S::full + 8 * s, 1);
      mbar_init(base + S::empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(base + S::sfull + 8 * s, 1);
      mbar_init(base + S::sempty + 8 * s, 1);
      mbar_init(base + S::tfull + 8 * s, 1);
      mbar_init(base + S::tempty + 8 * s, 4);
    }
    mbar_init(base + S::done, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(base + S::slot, S::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(lds_u32(base + S::slot));
  grid_launch_dependents();
  if (warp == 0 && lane == 0)   // while the preceding kernel drains: prefetches into L2 return nothing
    for (int k = k0; k < k1 && k < k0 + S::kStages; ++k) tma_prefetch_2d(&maps.b, k * kFp8Block, static_cast<int>(n0));
  __syncwarp();
  grid_dependency_wait();

  bool failed = false;
  if (warp == 0) {
    const bool leader = elect_one();
    if (leader) {
      prefetch_map(&maps.a);
      prefetch_map(&maps.b);
    }
    int i = 0;
    bool ok = true;
    for (int k = k0; k < k1; ++k, ++i) {
      const int s = i % S::kStages;
      ok = wait_here(base + S::empty + 8 * s, ((i / S::kStages) & 1u) ^ 1u, abort_flag);
      ok = __all_sync(kFullMask, ok);
      if (!ok) break;
      const uint32_t st = base + S::stages + s * S::kStage, bar = base + S::full + 8 * s;
      if (leader) {
        mbar_arrive_expect_tx(bar, S::kStage);
        tma_load_2d_plain(st, &maps.b, k * kFp8Block, static_cast<int>(n0), bar);
        tma_load_2d_plain(st + S::kW, &maps.a, k * kFp8Block, static_cast<int>(m0), bar);
      }
    }
    if (!ok)   // copies still in flight land before the CTA goes on
      for (int j = i > S::kStages ? i - S::kStages : 0; j < i; ++j)
        mbar_wait(base + S::full + 8 * (j % S::kStages), (j / S::kStages) & 1u);
    __syncwarp();
  } else if (warp == 1) {
    const bool leader = elect_one();
    const uint64_t wdesc0 = umma_desc(base + S::stages, kSwizzle128, 1024);
    const uint64_t xdesc0 = umma_desc(base + S::stages + S::kW, kSwizzle128, 1024);
    uint32_t i = 0, q = 0, u = 0;
    bool ok = true;
    for (int k = k0; k < k1; ++k, ++i) {
      const uint32_t s = i % S::kStages, sb = q & 1u, j = k % kChunk;
      const bool first = kSeg ? i % kSegment == 0 : i == 0;
      const bool last = k + 1 == k1 || (kSeg && (i + 1) % kSegment == 0);
      const bool begin = j == 0 || i == 0, end = j == kChunk - 1 || k + 1 == k1;
      if (first && u >= 2) ok = wait_here(base + S::tempty + 8 * (u & 1u), ((u - 2) >> 1) & 1u, abort_flag);
      if (ok && begin) ok = wait_here(base + S::sfull + 8 * sb, (q >> 1) & 1u, abort_flag);
      if (ok) ok = wait_here(base + S::full + 8 * s, (i / S::kStages) & 1u, abort_flag);
      ok = __all_sync(kFullMask, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t sfw = tmem + S::kColScales + 8 * sb, sfx = sfw + 4;
      const uint32_t sc = base + S::scales + sb * S::kScale;
      const uint64_t wdesc = wdesc0 + s * (S::kStage >> 4), xdesc = xdesc0 + s * (S::kStage >> 4);
      const uint32_t idesc = kDesc | (j << 29) | (j << 4);
      if (leader) {
        if (begin) {
          tmem_copy_scales(sfw, sc);
          tmem_copy_scales(sfx, sc + 512);
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_mx(tmem + (u & 1u) * TT, wdesc + 2 * kk, xdesc + 2 * kk, idesc, sfw, sfx, !first || kk > 0);
        mma_commit(base + S::empty + 8 * s);
        if (end) mma_commit(base + S::sempty + 8 * sb);
        if (last) mma_commit(base + S::tfull + 8 * (u & 1u));
      }
      if (end) ++q;
      if (last) ++u;
    }
    if (leader) {
      mma_commit(base + S::done);
      mbar_wait(base + S::done, 0);   // nothing in flight when the stages and the tensor memory are reused
    }
    __syncwarp();
  } else if (warp == 2) {
    const int chunks = (kb + kChunk - 1) / kChunk;
    const ScaleRows rw{a.sb, a.ldb_s, a.N, a.tile_b, chunks, a.vec_sb};
    const ScaleRows rx{a.sa, a.lda_s, a.M, a.tile_a, chunks, a.vec_sa};
    const uint4 one = make_uint4(0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu, 0x7f7f7f7fu);
    uint4 nw[4], nx[4];
    const auto fetch = [&](int g) {
#pragma unroll
      for (int r = 0; r < 4; ++r) nw[r] = rw.at(n0 + r * 32 + lane, g);
#pragma unroll
      for (int r = 0; r < 4; ++r) nx[r] = r * 32 < TT ? rx.at(m0 + r * 32 + lane, g) : one;
    };
    const int c0 = k0 / kChunk, c1 = (k1 + kChunk - 1) / kChunk;   // chunks of this split
    uint32_t q = 0;
    bool ok = true;
    fetch(c0 / 4);
    for (int g = c0 / 4; 4 * g < c1 && ok; ++g) {
      uint4 ww[4], wx[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        ww[r] = nw[r];
        wx[r] = nx[r];
      }
      if (4 * (g + 1) < c1) fetch(g + 1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (4 * g + j < c0 || 4 * g + j >= c1) continue;
        const uint32_t sb = q & 1u;
        ok = wait_here(base + S::sempty + 8 * sb, ((q >> 1) & 1u) ^ 1u, abort_flag);
        ok = __all_sync(kFullMask, ok);
        if (!ok) break;
        const uint32_t sc = base + S::scales + sb * S::kScale + lane * 16;
        sts_words(sc, word_of(ww[0], j), word_of(ww[1], j), word_of(ww[2], j), word_of(ww[3], j));
        sts_words(sc + 512, word_of(wx[0], j), word_of(wx[1], j), word_of(wx[2], j), word_of(wx[3], j));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(base + S::sfull + 8 * sb);
        ++q;
      }
    }
  } else if (warp >= 4) {
    const int quad = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const int segments = kSeg ? (k1 - k0 + kSegment - 1) / kSegment : 1;
    float sum[TT];
    for (int u = 0; u < segments; ++u) {
      bool ok = wait_here(base + S::tfull + 8 * (u & 1), (u >> 1) & 1u, abort_flag) && *abort_flag == 0u;
      ok = __all_sync(kFullMask, ok);
      if (!ok) {
        failed = true;
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < TT; c += 16) {
        float v[16];
        tmem_ld16(tmem + lanes + (u & 1) * TT + c, v);
        tmem_wait_ld();
        reg_fence16(v);
#pragma unroll
        for (int i = 0; i < 16; ++i) sum[c + i] = u == 0 ? v[i] : sum[c + i] + v[i];
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(base + S::tempty + 8 * (u & 1));
    }
    // every MMA of this CTA has read its stages: they take the partial sums
    if (!failed) {
#pragma unroll
      for (int c = 0; c < TT; ++c)
        asm volatile("st.shared.f32 [%0], %1;" :: "r"(base + S::stages + 4 * (c * 128 + quad * 32 + lane)), "f"(sum[c])
                     : "memory");
    }
  }
  __syncwarp();
  cluster_sync();   // every split's sums are written
  if (*abort_flag == 0u) {
    // a warp takes a token at a time, 4 columns a lane, all splits' parts in flight
    const int64_t n = n0 + 4 * lane, left = a.N - n;
    const int rows = static_cast<int>(a.M - m0 < TT ? a.M - m0 : TT);
    uint32_t from[kMaxSplits];
#pragma unroll
    for (int r = 0; r < kMaxSplits; ++r) from[r] = in_cta(base + S::stages + 16 * lane, r < splits ? r : 0);
#pragma unroll 2
    for (int c = rank + splits * warp; c < rows; c += splits * (kThreads / 32)) {
      float4 v[kMaxSplits];
#pragma unroll
      for (int r = 0; r < kMaxSplits; ++r)
        if (r < splits)
          asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                       : "=f"(v[r].x), "=f"(v[r].y), "=f"(v[r].z), "=f"(v[r].w) : "r"(from[r] + 512 * c));
      float s[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int r = 1; r < kMaxSplits; ++r)
        if (r < splits) {
          s[0] += v[r].x;
          s[1] += v[r].y;
          s[2] += v[r].z;
          s[3] += v[r].w;
        }
      if (a.add) add_row<T, 4>(s, static_cast<const T*>(a.add) + (m0 + c) * a.ldadd + n, left, a.vec_add);
      store_row4<T>(static_cast<T*>(a.out) + (m0 + c) * a.ldo + n, s, left, a.tma_out);
    }
  }
  tc_fence_before();
  cluster_sync();   // no CTA leaves while another reads its sums
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
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

// [32 rows x 128 bytes] boxes of a matrix of the output's shape and type.
template <typename T>
bool encode_out(EncodeTiled encode, CUtensorMap* map, const MatmulArgs& a, const void* p, int64_t ld) {
  const cuuint64_t dim[2] = {static_cast<cuuint64_t>(a.N), static_cast<cuuint64_t>(a.M)};
  const cuuint64_t stride[1] = {static_cast<cuuint64_t>(ld) * sizeof(T)};
  const cuuint32_t box[2] = {128 / sizeof(T), 32};
  const cuuint32_t unit[2] = {1, 1};
  const CUtensorMapDataType type = std::is_same<T, float>::value    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                   : std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                    : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return encode(map, type, 2, const_cast<void*>(p), dim, stride, box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// Launch of `gx` x `gy` CTAs in clusters of `splits`.
cudaLaunchConfig_t few_config(int splits, unsigned gx, unsigned gy, size_t smem, cudaStream_t st,
                              cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(gx, gy);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

cudaError_t prepare_matmul(int* clusters) {
  cudaError_t e = cudaSuccess;
  const auto set = [&](auto k, uint32_t bytes) {
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(reinterpret_cast<const void*>(k), cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(bytes));
  };
  set(matmul_pair_kernel<__nv_bfloat16, 256>, Pair<256>::bytes);
  set(matmul_pair_kernel<__half, 256>, Pair<256>::bytes);
  set(matmul_pair_kernel<__nv_bfloat16, 128>, Pair<128>::bytes);
  set(matmul_pair_kernel<__half, 128>, Pair<128>::bytes);
  set(matmul_pair_kernel<float, 128>, Pair<128>::bytes);
  const auto few = [&](auto t) {
    using T = decltype(t);
    set(matmul_few_kernel<T, 16>, Few<16>::bytes);
    set(matmul_few_kernel<T, 32>, Few<32>::bytes);
    set(matmul_few_kernel<T, 64>, Few<64>::bytes);
    set(matmul_few_kernel<T, 128>, Few<128>::bytes);
  };
  few(__nv_bfloat16{});
  few(__half{});
  few(float{});
  // one CTA per SM in every form: the count is the same for all of them
  for (int splits = 1; splits <= kMaxSplits && e == cudaSuccess; ++splits) {
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = few_config(splits, splits, 1, Few<128>::bytes, nullptr, attr);
    e = cudaOccupancyMaxActiveClusters(&clusters[splits], matmul_few_kernel<__nv_bfloat16, 128>, &cfg);
  }
  return e;
}

// One 256 x TN tile per CTA pair, at most one pair per two SMs.
template <typename T, int TN>
cudaError_t launch_pair(EncodeTiled encode, const MatmulArgs& a, int sms, cudaStream_t st) {
  MatmulMaps maps;
  if (!encode_codes(encode, &maps.a, a.a, a.M, a.K, a.lda, 128) ||
      !encode_codes(encode, &maps.b, a.b, a.N, a.K, a.ldb, TN / 2))
    return cudaErrorInvalidValue;
  CUtensorMap out = maps.a, add = maps.a;
  if (a.tma_out && !encode_out<T>(encode, &out, a, a.out, a.ldo)) return cudaErrorInvalidValue;
  if (a.add && a.tma_add && !encode_out<T>(encode, &add, a, a.add, a.ldadd)) return cudaErrorInvalidValue;
  const int64_t tiles = ((a.M + 255) / 256) * ((a.N + TN - 1) / TN);
  const int64_t pairs = tiles < sms / 2 ? tiles : sms / 2;
  return launch_dependent(matmul_pair_kernel<T, TN>, dim3(static_cast<unsigned>(2 * pairs)), kThreads,
                          Pair<TN>::bytes, st, maps, out, add, a);
}

template <typename T, int TT>
cudaError_t launch_few(EncodeTiled encode, const MatmulArgs& a, int splits, cudaStream_t st) {
  MatmulMaps maps;
  if (!encode_codes(encode, &maps.a, a.a, a.M, a.K, a.lda, TT) ||
      !encode_codes(encode, &maps.b, a.b, a.N, a.K, a.ldb, 128))
    return cudaErrorInvalidValue;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = few_config(splits, static_cast<unsigned>((a.N + 127) / 128 * splits),
                                            static_cast<unsigned>((a.M + TT - 1) / TT), Few<TT>::bytes, st, attr);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, matmul_few_kernel<T, TT>, maps, a, splits);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// Which kernel. Up to 64 rows: K split over clusters, as many splits as let all
// clusters run at once (clusters[s]: how many clusters of s CTAs do). Above, a
// block of 128 columns of K takes either kernel about 0.25 us, and the cluster's
// barriers and sums cost it about 4 us more than a pair's epilogue: the split
// pays where it takes kFewSaves blocks off each CTA. N = K = 4096, bf16: 128
// rows (24 blocks less) 7.8 us split, 8.9 in pairs; 256 rows (16 less) 10.3 and
// 9.4; 256 rows at K = 16384 (64 less) 23.8 and 32.9. Pairs take tiles 128
// columns wide where that is one wave (256 rows: 9.4 us, 14.0 at 256 wide),
// else 256 wide (1024 rows: 15.7 us, 18.4 at 128 wide); f32 always 128, whose
// sum its epilogue can hold.
constexpr int kFewSaves = 24;
cudaError_t launch_matmul(const MatmulArgs& a, int dtype, int sms, const int* clusters, cudaStream_t st) {
  EncodeTiled encode = tensor_map_encoder();
  if (!encode) return cudaErrorNotSupported;
  return with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const int64_t kb = (a.K + kFp8Block - 1) / kFp8Block;
    const int64_t tiles = ((a.N + 127) / 128) * ((a.M + 127) / 128);
    int s = 1;
    while (s < kMaxSplits && s < kb && tiles <= clusters[s + 1]) ++s;
    if (a.M <= 16) return launch_few<T, 16>(encode, a, s, st);
    if (a.M <= 32) return launch_few<T, 32>(encode, a, s, st);
    if (a.M <= 64) return launch_few<T, 64>(encode, a, s, st);
    if (kb - (kb + s - 1) / s >= kFewSaves) return launch_few<T, 128>(encode, a, s, st);
    if constexpr (std::is_same<T, float>::value) {
      return launch_pair<T, 128>(encode, a, sms, st);
    } else {
      const int64_t narrow = ((a.M + 255) / 256) * ((a.N + 127) / 128);
      return narrow <= sms / 2 ? launch_pair<T, 128>(encode, a, sms, st) : launch_pair<T, 256>(encode, a, sms, st);
    }
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
