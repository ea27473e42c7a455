/*
 * taco.h - C ABI of the GB300 (sm_103a) TACO fused compression operator.
 *
 * The operator is the one described for tensor-parallel intermediate tensors
 * in "TACO: Efficient Communication Compression of Intermediate Tensors for
 * Scalable Tensor-Parallel LLM Training" (gist.science Portuguese summary,
 * §2.B.1 "Adaptive Scale-Hadamard transform", §2.B.2 "Dual-Scale
 * quantization", §2.B.3 "fused operator" and "two-shot AllReduce"):
 *
 *   compress, per block of n contiguous elements of a row (n = 64, 128, 256):
 *     E      = mean of x^2 over the block            (raw second moment)
 *     alpha  = sqrt(E* / E)      (1 when E == 0)      (pre-rotation scale),
 *              rounded to fp32 and kept in [2^-126, 2^126], where alpha and
 *              1/alpha are both normal fp32 numbers (a block whose energy is
 *              further than 2^252 from E* is rescaled only part of the way)
 *     y      = (H_n / sqrt(n)) (alpha x)              (Sylvester Hadamard)
 *     s      = max(1, max|y| / 448)                   (post-rotation scale)
 *     q      = E4M3(y / s)   round-to-nearest-even, saturating at +-448
 *   decompress-reduce, over P shards compressed with the same n:
 *     x_hat  = bf16( sum_p (1/alpha_p) (H_n / sqrt(n)) (s_p dec(q_p)) )
 *
 * Conventions of every entry point:
 *   - All buffers are device memory owned by the caller. The library never
 *     allocates, frees or synchronises; work is enqueued on `stream`
 *     (a cudaStream_t; NULL is the legacy default stream) of the device that
 *     is current on the calling thread.
 *   - Arguments are checked on the host before anything is enqueued. On any
 *     error nothing is launched and nothing is written.
 *   - A launch failure is reported as TACO_ERR_CUDA (from cudaGetLastError).
 *   - bf16 tensors are row-major [N, h] with h % n == 0; a block is n
 *     contiguous elements of one row, block b = row * (h/n) + column / n.
 */
#ifndef TACO_H_
#define TACO_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum taco_status {
  TACO_OK = 0,
  TACO_ERR_NULL = 1,       /* a required pointer is NULL                       */
  TACO_ERR_SHAPE = 2,      /* N < 0, h <= 0, h % block != 0, or N*h too large  */
  TACO_ERR_BLOCK = 3,      /* block is not 64, 128 or 256                      */
  TACO_ERR_ALIGN = 4,      /* a tensor or bundle pointer is not 16-byte aligned */
  TACO_ERR_ARG = 5,        /* target energy not in (0, 2^120], P out of
                              [1, TACO_MAX_SHARDS], unknown variant            */
  TACO_ERR_CUDA = 6,       /* a CUDA call or launch failed                     */
  TACO_ERR_WORKSPACE = 7   /* workspace NULL or smaller than taco_workspace_bytes */
} taco_status;

/* Dual-scale variants. DUAL is the operator above. ABSMAX replaces the
 * overflow guard by s = max|y| / 448 (1 for an all-zero block); alpha then
 * cancels from the codes. STATIC gives every block of the tensor the same
 * data-independent s = fp32(sqrt(block * E*) / 448): after the energy
 * rescale the rotated block has squared norm block * E*, so no |y| exceeds
 * sqrt(block * E*) and no code saturates (a per-tensor scale in the sense of
 * the euno.news rewrite, Methodology). ABSMAX and STATIC are kept for error
 * studies. */
enum { TACO_VARIANT_DUAL = 0, TACO_VARIANT_ABSMAX = 1, TACO_VARIANT_STATIC = 2 };

#define TACO_MAX_SHARDS 16
#define TACO_Q_MAX 448.0f
#define TACO_ABI_VERSION 1

/* Per-tensor header written by the compress kernel (one per shard).
 * s_max = max over blocks of s (0 for an empty tensor); n_clamped = number of
 * blocks with s > 1. This is the per-tensor part of the dual scale: the
 * "per-tensor scale adapted to the dynamic range" of the euno.news rewrite
 * ("Adaptive Scale-Hadamard Transform" in its Methodology), kept as a
 * summary, not applied to the codes. */
typedef struct taco_header {
  int64_t N;
  int64_t h;
  int32_t block;
  int32_t variant;
  float target_energy;
  float q_max;
  float s_max;
  uint32_t n_clamped;
} taco_header; /* 40 bytes */

/* ---- Shard layout -------------------------------------------------------
 * One compressed tensor ("shard") is one contiguous byte range:
 *   [codes:  N*h bytes, E4M3, row-major][pad to 256]
 *   [scales: N*(h/n) pairs of fp32 (alpha, s), block order][pad to 256]
 * The two scales of a block are adjacent because every reader needs both
 * (TACO pt summary §2.B.2: reconstruction uses alpha_k and s_k together).
 * A bundle is P shards back to back, shard p at p * taco_shard_bytes(...);
 * it is the receive buffer of the ReduceScatter half of the two-shot
 * AllReduce (TACO pt summary, §2.B.3). Both parts start 256-byte aligned
 * relative to the shard start. Return 0 for invalid arguments. */
size_t taco_shard_bytes(int64_t N, int64_t h, int block);
size_t taco_shard_scales_offset(int64_t N, int64_t h, int block);

/* Bytes of device workspace that compress needs for P shards (16 per
 * shard). The workspace holds, per shard, an arrival counter and the running
 * maximum and count used to write the per-tensor header in the same launch;
 * the first shard's slot also holds the counter from which the tensor-core
 * compress hands out tiles of every shard. It must be zero-filled before
 * its first use; each call leaves it zero-filled again. Calls that share a
 * workspace must not overlap on the GPU (use one workspace per stream). */
size_t taco_workspace_bytes(int P);

/* ---- taco_compress ------------------------------------------------------
 * Compress one bf16 tensor x [N, h] (device, 16-byte aligned) into one
 * shard at `shard_out` (device, 16-byte aligned, taco_shard_bytes(N,h,block)
 * bytes) and its header at `header_out` (device, 8-byte aligned).
 *   block          n, one of 64, 128, 256
 *   target_energy  E* in (0, 2^120], the per-element energy of every
 *                  rescaled block (TACO pt summary §2.B.1: each block is
 *                  rescaled to one common energy level); 4096 puts the
 *                  rotated RMS at 64 code units
 *   variant        TACO_VARIANT_DUAL, TACO_VARIANT_ABSMAX or TACO_VARIANT_STATIC
 *   workspace      device memory of taco_workspace_bytes(1) bytes, 16-byte
 *                  aligned, zero before its first use. The pages specify no
 *                  API; this argument is this library's addition to the plain
 *                  compress(x, block, E*) signature, because the per-tensor
 *                  header is written in the same launch (the CTA that
 *                  arrives last reads counters that every CTA updates) and
 *                  the library itself never allocates.
 * Every finite bf16 input is accepted, subnormals and values near the bf16
 * maximum included; no finite input gives a NaN code.
 * N == 0 is valid: no code is written and the header reports s_max = 0. */
taco_status taco_compress(const void* x_bf16, int64_t N, int64_t h, int block,
                          float target_energy, int variant, void* shard_out,
                          taco_header* header_out, void* workspace,
                          size_t workspace_bytes, void* stream);

/* ---- taco_compress_shards -----------------------------------------------
 * The same for P tensors x [P, N, h] (contiguous) in one launch: shard p of
 * the bundle at `bundle_out` (P * taco_shard_bytes bytes) and header p of
 * `headers_out` [P]. 1 <= P <= TACO_MAX_SHARDS. These are the P chunks one
 * rank compresses before the ReduceScatter (TACO pt summary §2.B.3).
 * taco_compress and taco_compress_shards run the tensor-core kernel of
 * taco_compress_shards_mma (below) when a shard holds at most 2^31 - 256
 * blocks, and the CUDA-core kernel of taco_compress_shards_fwht beyond that:
 * the outputs meet the same parity bar either way. */
taco_status taco_compress_shards(const void* x_bf16, int P, int64_t N, int64_t h,
                                 int block, float target_energy, int variant,
                                 void* bundle_out, taco_header* headers_out,
                                 void* workspace, size_t workspace_bytes,
                                 void* stream);

/* ---- taco_compress_shards_fwht ---------------------------------------------
 * taco_compress_shards with the whole rotation as a CUDA-core fast
 * Walsh-Hadamard transform (log2 n butterfly levels in registers and warp
 * shuffles; TACO pt summary §2.B.1 rotates each block by the orthonormal
 * Hadamard matrix): same arguments, layout, headers, workspace and errors,
 * no limit on blocks per shard beyond the shape checks. The energy is summed
 * from x. A code can differ from the tensor-core kernel's by one E4M3 step
 * where the fp32 rotated value differs in its last bits. */
taco_status taco_compress_shards_fwht(const void* x_bf16, int P, int64_t N, int64_t h,
                                      int block, float target_energy, int variant,
                                      void* bundle_out, taco_header* headers_out,
                                      void* workspace, size_t workspace_bytes,
                                      void* stream);

/* ---- taco_compress_shards_mma ----------------------------------------------
 * taco_compress_shards with the Hadamard rotation on the tensor cores
 * (tcgen05, sm_100 family): same arguments, layout, headers, workspace and
 * errors. H_n = H_{n/64} (x) H_64 (Sylvester, TACO pt summary §2.B.1), so
 * every 64-element chunk of a block is multiplied by H_64 as one row of a
 * [128 x 64] x [64 x 64] bf16 product accumulated in fp32, and the
 * log2(n/64) remaining butterfly levels run in registers. The block energy
 * is taken from the rotated block (sum t^2 = n sum x^2). The outputs meet the
 * same parity bar as taco_compress_shards_fwht; a code can differ from that
 * kernel's by one E4M3 step where the fp32 rotated value differs in its last
 * bits. A block whose largest rotated magnitude lies outside [2^-40, 2^56]
 * takes a slower path: its energy is summed again from the rotated values
 * scaled by a power of two, or, for blocks of bf16 subnormals only and
 * blocks near the bf16 maximum whose rotation overflows fp32, the block is
 * redone from x. Extra limit: at most 2^31 - 256 blocks per shard (the tensor
 * copies address rows with 32-bit coordinates), else TACO_ERR_SHAPE.
 * N == 0 writes the headers as taco_compress_shards does. */
taco_status taco_compress_shards_mma(const void* x_bf16, int P, int64_t N, int64_t h,
                                     int block, float target_energy, int variant,
                                     void* bundle_out, taco_header* headers_out,
                                     void* workspace, size_t workspace_bytes,
                                     void* stream);

/* ---- taco_compress_shards_noalloc -----------------------------------------
 * The paper has no counterpart to this entry point: it exists for callers
 * that cannot allocate device memory when they compress (a communication
 * library's progress thread or collective callback, where cudaMalloc may
 * synchronise the device or deadlock against work in flight; a runtime
 * whose memory belongs to an external pool). It is taco_compress_shards
 * without the workspace argument: the counters and running totals live in
 * a static device array of the library (TACO_NOALLOC_MAX_SHARDS * 16 = 128
 * bytes), which every GPU that loads the library holds until the process
 * exits. The caller still passes x, the bundle and the headers.
 *   - P > TACO_NOALLOC_MAX_SHARDS returns TACO_ERR_WORKSPACE (the request does
 *     not fit the static scratch); other errors as taco_compress_shards, and a
 *     rejected call enqueues nothing.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture.
 *   - Each call clears the counters it uses with cudaMemsetAsync on `stream`
 *     and then launches the compress kernel; it allocates nothing.
 *   - All calls share the one array, so calls that overlap on the GPU (other
 *     streams, other threads) race on it: order them. */
#define TACO_NOALLOC_MAX_SHARDS 8
taco_status taco_compress_shards_noalloc(const void* x_bf16, int P, int64_t N, int64_t h,
                                         int block, float target_energy, int variant,
                                         void* bundle_out, taco_header* headers_out,
                                         void* stream);

/* ---- taco_decompress_reduce ---------------------------------------------
 * Reconstruct and sum P shards of one bundle (device, 16-byte aligned, the
 * layout above, all compressed from [N, h] tensors with the same block)
 * into bf16 out [N, h] (device, 16-byte aligned). The P reconstructions are
 * summed in fp32 in the rotated domain and rotated back once (the rotation is
 * linear and shared by all shards), then rounded to bf16 once. This is the
 * reconstruction of TACO pt summary §2.B.2 fused with the reduce of the
 * ReduceScatter step of §2.B.3. 1 <= P <= TACO_MAX_SHARDS. N == 0 is valid
 * and launches nothing. `out` must not overlap the bundle. */
taco_status taco_decompress_reduce(const void* bundle, int P, int64_t N, int64_t h,
                                   int block, void* out_bf16, void* stream);

/* ---- taco_decompress_reduce_mma[_ptrs] ------------------------------------
 * taco_decompress_reduce[_ptrs] with the inverse rotation on the tensor
 * cores (tcgen05, E4M3 operands): same arguments, layout and errors, for
 * block 64 or 128 (block 256 returns TACO_ERR_BLOCK). By linearity
 * x_hat = sum_p (s_p / (alpha_p sqrt(n))) H_n q_p (TACO pt summary §2.B.2,
 * reduce of §2.B.3); each 64-code chunk of each shard is multiplied by H_64
 * as it arrives, exactly in fp32, the scaled sum over shards and the
 * remaining butterfly levels run in registers, one bf16 rounding at the end.
 * The output meets the reconstruction bar of taco_decompress_reduce; the two
 * entries sum in different orders, so single bf16 results may differ by one
 * unit in the last place. At most 2^31 - 256 blocks per shard. */
taco_status taco_decompress_reduce_mma(const void* bundle, int P, int64_t N, int64_t h,
                                       int block, void* out_bf16, void* stream);
taco_status taco_decompress_reduce_mma_ptrs(const void* const* shards, int P, int64_t N,
                                            int64_t h, int block, void* out_bf16, void* stream);

/* ---- INT8 fallback format -------------------------------------------------
 * TACO pt summary §5 ("Agnóstico de Hardware"): the framework degrades to
 * INT8 on hardware without FP8 support. The pages define no INT8 format
 * beyond the uniform steps of §2.A; these entries take the plainest reading:
 * every step of the operator as above, with the code of a rotated value y
 * being q = round-half-to-even(y / s) as a signed byte (two's complement,
 * never -128) and Q_max = 127 in place of 448 in the scale rules (DUAL:
 * s = max(1, max|y| / 127); ABSMAX: s = max|y| / 127; STATIC:
 * s = sqrt(block * E*) / 127). The headers report q_max = 127. Same shard
 * layout, arguments, workspace and errors as taco_compress_shards_mma /
 * taco_decompress_reduce; the rotation runs on the tensor cores. A bundle
 * must be decompressed with the entry of its format. */
taco_status taco_compress_shards_int8(const void* x_bf16, int P, int64_t N, int64_t h,
                                      int block, float target_energy, int variant,
                                      void* bundle_out, taco_header* headers_out,
                                      void* workspace, size_t workspace_bytes,
                                      void* stream);
taco_status taco_decompress_reduce_int8(const void* bundle, int P, int64_t N, int64_t h,
                                        int block, void* out_bf16, void* stream);
/* The AllGather side and the step between the two halves of the two-shot
 * AllReduce in the INT8 format: taco_reduce_recompress_ptrs and
 * taco_decompress_shards_ptrs with INT8 codes in and out (q_max 127 in the
 * written header). */
taco_status taco_reduce_recompress_int8_ptrs(const void* const* shards, int P, int64_t N,
                                             int64_t h, int block, float target_energy,
                                             int variant, void* shard_out,
                                             taco_header* header_out, void* out_bf16,
                                             void* workspace, size_t workspace_bytes,
                                             void* stream);
taco_status taco_decompress_shards_int8_ptrs(const void* const* shards, int P, int64_t N,
                                             int64_t h, int block, void* out_bf16, void* stream);

/* ---- taco_reduce_recompress_batched_ptrs --------------------------------
 * Y independent reduce-recompress operations in one launch: the step between
 * the ReduceScatter and the AllGather (TACO pt summary §2.B.3) for Y
 * destinations at once. Reduction y sums shards[y*P .. y*P+P-1] (host array
 * of Y*P device pointers, 1 <= Y*P <= TACO_MAX_SHARDS) and writes shard y of
 * `shards_out` (Y consecutive shards of taco_shard_bytes, device, 16-byte
 * aligned) and headers_out[y]; the workspace holds Y shard workspaces
 * (taco_workspace_bytes(Y)). code_format: TACO_FORMAT_E4M3 or
 * TACO_FORMAT_INT8 (codes in and out). No bf16 side output. Otherwise as
 * taco_reduce_recompress_ptrs. */
enum { TACO_FORMAT_E4M3 = 0, TACO_FORMAT_INT8 = 1 };
taco_status taco_reduce_recompress_batched_ptrs(const void* const* shards, int Y, int P, int64_t N,
                                                int64_t h, int block, float target_energy,
                                                int variant, int code_format, void* shards_out,
                                                taco_header* headers_out, void* workspace,
                                                size_t workspace_bytes, void* stream);

/* ---- taco_decompress_reduce_ptrs ----------------------------------------
 * As taco_decompress_reduce, with the P shards in P separate buffers
 * (`shards[p]` a device pointer to one shard, 16-byte aligned; `shards` itself
 * is a host array of P pointers, read before the call returns). This is the
 * form a receive step that lands each peer's chunk in its own buffer uses. */
taco_status taco_decompress_reduce_ptrs(const void* const* shards, int P, int64_t N,
                                        int64_t h, int block, void* out_bf16,
                                        void* stream);

/* ---- taco_decompress_shards ---------------------------------------------
 * Reconstruct each of the P shards of `bundle` on its own (no sum) into
 * out_bf16 [P][N][h]: shard p to rows p*N .. p*N+N-1. This is the receive
 * side of the AllGather half of the two-shot AllReduce (TACO pt summary
 * §2.B.3), where every rank expands the P reduced chunks into the full
 * tensor; the reconstruction is that of §2.B.2, the same arithmetic as
 * taco_decompress_reduce with P = 1 (bit-identical output). One launch.
 * N == 0 launches nothing. */
taco_status taco_decompress_shards(const void* bundle, int P, int64_t N, int64_t h, int block,
                                   void* out_bf16, void* stream);

/* The same with the shards in separate buffers (host array of P pointers). */
taco_status taco_decompress_shards_ptrs(const void* const* shards, int P, int64_t N, int64_t h,
                                        int block, void* out_bf16, void* stream);

/* ---- taco_reduce_recompress ---------------------------------------------
 * The reduced chunk compressed again for the AllGather half of the two-shot
 * AllReduce (TACO pt summary §2.B.3: compression around ReduceScatter +
 * AllGather), fused with the reduce: the P shards of `bundle` (as for
 * taco_decompress_reduce) are summed and the sum x_hat is compressed into
 * one shard at `shard_out` with its header at `header_out`, with the same
 * block, target energy and variant rules as taco_compress. x_hat is
 * compressed as computed, without rounding it to bf16 first. Because the
 * rotation is shared and orthogonal, this needs no Hadamard transform on the
 * device: the rotated sum is already at hand. If `out_bf16` is not NULL the
 * bf16 sum [N, h] is written there as well (bit-identical to
 * taco_decompress_reduce). `workspace`: at least taco_workspace_bytes(1)
 * zero-filled bytes, as for compress. No output may overlap an input. */
taco_status taco_reduce_recompress(const void* bundle, int P, int64_t N, int64_t h, int block,
                                   float target_energy, int variant, void* shard_out,
                                   taco_header* header_out, void* out_bf16, void* workspace,
                                   size_t workspace_bytes, void* stream);

/* The same with the P shards in separate buffers (`shards`: host array of P
 * device pointers, read before the call returns). */
taco_status taco_reduce_recompress_ptrs(const void* const* shards, int P, int64_t N, int64_t h,
                                        int block, float target_energy, int variant,
                                        void* shard_out, taco_header* header_out, void* out_bf16,
                                        void* workspace, size_t workspace_bytes, void* stream);

/* ---- E4M3 codec ----------------------------------------------------------
 * Elementwise conversions with the instructions the operator's kernels use
 * (TACO pt summary §2.A: FP8 E4M3 instead of INT8). `in` and `out` are device
 * arrays of n elements; n == 0 launches nothing.
 *   taco_e4m3_encode_f32: fp32 -> E4M3 code, round to nearest even, |v| > 448
 *                         and +-inf saturate to +-448, NaN -> 0x7F.
 *   taco_e4m3_decode_f32: E4M3 code -> its exact fp32 value (0x7F/0xFF: NaN). */
taco_status taco_e4m3_encode_f32(const float* in, uint8_t* out, int64_t n, void* stream);
taco_status taco_e4m3_decode_f32(const uint8_t* in, float* out, int64_t n, void* stream);

/* ---- FP8 block tensors ------------------------------------------------------
 * What a tensor-parallel layer computes between its compressed all-reduces,
 * in 8 bits: the TACO pages compress the tensors that such layers exchange
 * (pt summary, section 1) and leave the layers themselves to the training
 * framework; these entry points are this library's own.
 *
 * A matrix [rows, cols] is held as E4M3 codes and E8M0 scale bytes (byte b
 * stands for 2^(b - 127), 255 for NaN), one scale per row and 128 columns
 * (tile_rows 1) or per 128 x 128 tile (tile_rows 128, for weights):
 *   value[r][c] = E4M3(codes[r][c]) * 2^(scales[r / tile_rows][c / 128] - 127).
 * Quantising a block with largest magnitude m takes the smallest power of two
 * s >= m / 448, s >= 2^-126 (1 for an all-zero block), and rounds value / s to
 * nearest even. A block that holds an infinity or a NaN gets the scale byte
 * 255, so that all its values, and every sum they enter, are NaN; its codes
 * are unspecified. Values below half a code step of a block with s = 2^-126
 * round to zero like any others.
 *
 * Conventions: rows of codes start at multiples of 16 bytes (codes 16-byte
 * aligned, ld_codes % 16 == 0), rows of scales at multiples of 4 (scales
 * 4-byte aligned, ld_scales % 4 == 0). ld_codes >= cols, and ld_scales >=
 * ceil(cols / 128). Bytes between the end of a row and the next row are
 * never written; a product reads scales by whole aligned words (of 4 bytes,
 * or of 16 where rows of scales start on 16), so it may read up to 15 bytes
 * behind a row's last scale, and makes no use of them. rows == 0 is valid
 * everywhere; cols >= 1.
 *
 * Plain matrices are bf16, f16 or f32 (dtype) with contiguous columns and ld
 * elements between rows (ld >= cols), aligned to their element; rows that all
 * start on 16 bytes are read and written faster. No output may overlap an
 * input or another output except where an entry says so. Statuses:
 * TACO_ERR_NULL, TACO_ERR_SHAPE (sizes, strides or two descriptors that
 * disagree), TACO_ERR_BLOCK (tile_rows), TACO_ERR_ALIGN, TACO_ERR_ARG (dtype,
 * eps), TACO_ERR_WORKSPACE, TACO_ERR_CUDA. */
enum { TACO_DTYPE_BF16 = 0, TACO_DTYPE_F16 = 1, TACO_DTYPE_F32 = 2 };

typedef struct taco_fp8_tensor {
  uint8_t* codes;
  uint8_t* scales;
  int64_t ld_codes;  /* bytes between rows of codes  */
  int64_t ld_scales; /* bytes between rows of scales */
  int64_t rows;
  int64_t cols;
  int32_t tile_rows; /* 1 or 128 */
} taco_fp8_tensor;

/* x [M, K] -> its FP8 blocks in `rows_out` [M, K], its transpose's in
 * `cols_out` [K, M] (blocks of 128 of x's rows: the operand of a product that
 * sums over them), or both from one read of x (either may be NULL, not both).
 * The outputs' tile_rows are equal where both are given; with 128 the two
 * hold the same codes and scales, transposed. */
taco_status taco_fp8_quantize(const void* x, int dtype, int64_t M, int64_t K, int64_t ld,
                              const taco_fp8_tensor* rows_out, const taco_fp8_tensor* cols_out,
                              void* stream);
/* The same from an FP8 block tensor: a checkpoint quantised along its columns
 * becomes the operand of the weight gradient, which sums over its rows. */
taco_status taco_fp8_requantize(const taco_fp8_tensor* x, const taco_fp8_tensor* rows_out,
                                const taco_fp8_tensor* cols_out, void* stream);

/* Root-mean-square norm of h = x + residual, rows of H (1 <= H <= 32768):
 *   h    = x + residual rounded to dtype   (h = x where residual is NULL)
 *   rstd = (mean over the row of h^2 + eps)^(-1/2)          (fp32 sums)
 *   y    = h * rstd * weight               quantised to `y` [M, H], tile_rows 1
 * residual, h_out: both NULL or neither; h_out may be x or residual itself
 * (same pointer and stride). weight [H] has the type weight_dtype. rstd [M]
 * (f32) and `checkpoint` [M, H] (h in FP8 blocks, tile_rows 1, for the
 * backward pass) may be NULL. eps >= 0. */
taco_status taco_rms_norm_fp8(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                              const void* weight, int weight_dtype, int dtype, int64_t M, int64_t H,
                              float eps, void* h_out, int64_t ldh, float* rstd,
                              const taco_fp8_tensor* y, const taco_fp8_tensor* checkpoint,
                              void* stream);

/* Its gradient, the quantisation of y taken as the identity. With xh = h *
 * rstd, g = dy * weight, c = mean over the row of g * xh:
 *   dx = rstd * (g - xh * c) + dh     the gradient of x and of the residual
 *   dw = sum over the rows of dy * xh (f32 [H])
 * h is read from `checkpoint`, or from h itself where that is not NULL
 * (exactly one of the two). dh is the gradient that reached h_out by other
 * ways (NULL: none). dy, h, dh and dx have the type dtype; dx may be dy, h or
 * dh itself. The row sums of dw are formed in a fixed order. `workspace`
 * (f32 partial sums, 16-byte aligned) need not be zeroed. M == 0 zeroes dw. */
size_t taco_rms_norm_workspace_bytes(int64_t M, int64_t H);
taco_status taco_rms_norm_fp8_backward(const void* dy, int64_t lddy,
                                       const taco_fp8_tensor* checkpoint, const void* h, int64_t ldh,
                                       const void* weight, int weight_dtype, const float* rstd,
                                       const void* dh, int64_t lddh, int dtype, int64_t M, int64_t H,
                                       void* dx, int64_t lddx, float* dw, void* workspace,
                                       size_t workspace_bytes, void* stream);

/* Gated activation y = silu(gate) * up, silu(g) = g / (1 + exp(-g)), of
 * matrices [M, F], quantised to `y` (tile_rows 1); gate and up are also
 * quantised as they are to checkpoint_gate and checkpoint_up (tile_rows 1,
 * both or neither NULL). */
taco_status taco_swiglu_fp8(const void* gate, int64_t ldg, const void* up, int64_t ldu, int dtype,
                            int64_t M, int64_t F, const taco_fp8_tensor* y,
                            const taco_fp8_tensor* checkpoint_gate,
                            const taco_fp8_tensor* checkpoint_up, void* stream);
/* Its gradient at the checkpointed gate and up, s = 1 / (1 + exp(-gate)):
 *   dgate = dy * up * s * (1 + gate * (1 - s)),  dup = dy * gate * s.
 * dup or dgate may be dy itself. */
taco_status taco_swiglu_fp8_backward(const void* dy, int64_t lddy,
                                     const taco_fp8_tensor* checkpoint_gate,
                                     const taco_fp8_tensor* checkpoint_up, int dtype, int64_t M,
                                     int64_t F, void* dgate, int64_t lddg, void* dup, int64_t lddu,
                                     void* stream);

/* out [M, N] = a [M, K] * b [N, K]^T (+ add), on the block-scaled tensor
 * cores: products of codes times both scales, summed in fp32, `add` (NULL:
 * none; out's type) added in fp32, rounded once to dtype. a and b may have
 * either tile_rows. add may be out itself (the running sum of a weight
 * gradient). A linear layer y = x W^T takes a = x, b = W; its input gradient
 * a = dy, b = W^T quantised; its weight gradient a = dy^T, b = x^T, both
 * quantised along the tokens. M, N and K at most 2^31 - 256. */
taco_status taco_matmul_fp8(const taco_fp8_tensor* a, const taco_fp8_tensor* b, const void* add,
                            int64_t ldadd, void* out, int64_t ldo, int dtype, void* stream);

/* The same product with a layer's epilogue, before anything is rounded:
 *   pre = a b^T + bias,   y = act(pre) + residual
 * Sums are fp32, those of outputs in 16 and 8 bits (and of the checkpoint beside
 * them) as the tensor cores leave them, which cut where fp32 rounds: off by
 * (K / 32 + 32) 2^-23 of their products' magnitudes at most. f32 outputs are sums of
 * segments of 1024 columns.
 * bias [N] (bias_dtype), residual [M, N] (dtype) and `checkpoint` may be NULL.
 * y goes to `out` (dtype), or quantised to y_fp8 (tile_rows 1; out and residual
 * NULL then, dtype unused): exactly one of the two. `checkpoint` (tile_rows 1)
 * keeps pre in 8 bits for the backward pass. residual may be out itself.
 * Activations: GELU x Phi(x); GELU_TANH x (1 + tanh(sqrt(2 / pi) (x + 0.044715
 * x^3))) / 2; SILU x / (1 + exp(-x)); RELU max(x, 0), of a NaN NaN. */
enum { TACO_ACT_NONE = 0, TACO_ACT_GELU = 1, TACO_ACT_GELU_TANH = 2, TACO_ACT_SILU = 3, TACO_ACT_RELU = 4 };
taco_status taco_linear_fp8(const taco_fp8_tensor* a, const taco_fp8_tensor* b, const void* bias,
                            int bias_dtype, int activation, const void* residual, int64_t ldr,
                            void* out, int64_t ldo, int dtype, const taco_fp8_tensor* y_fp8,
                            const taco_fp8_tensor* checkpoint, void* stream);

/* Its gradient at pre, d = dy * act'(pre), quantised once from fp32 as the two
 * products that follow read it: its rows [M, N] to rows_out (dx = d b), its
 * transpose [N, M] to cols_out (db = d^T a), and db [N] (f32), the sum of d's
 * rows in a fixed order; any of the three may be NULL, not all. pre is read from
 * `checkpoint` (tile_rows 1); without an activation d is dy, and checkpoint is
 * NULL. Outputs have tile_rows 1. RELU's slope at 0 is 0. `workspace`
 * (taco_linear_backward_workspace_bytes bytes, 16-byte aligned, not zeroed) may
 * be NULL where db is, or where M <= 128. M == 0 zeroes db. */
size_t taco_linear_backward_workspace_bytes(int64_t M, int64_t N);
taco_status taco_linear_fp8_backward(const void* dy, int64_t lddy, int dtype, int64_t M, int64_t N,
                                     const taco_fp8_tensor* checkpoint, int activation,
                                     const taco_fp8_tensor* rows_out, const taco_fp8_tensor* cols_out,
                                     float* db, void* workspace, size_t workspace_bytes, void* stream);

/* ---- Many tensors at once ---------------------------------------------------
 * What a training step does with a model's gradients: their norm, and an AdamW
 * step. A call takes a host array of `count` tensors (0 .. 2^20, read before
 * the call returns), contiguous on the device, of n elements each (n == 0 is
 * valid; 2^40 elements in all). Tensors that start on 16 bytes are read and
 * written faster. What a call writes shares no byte with anything else that it
 * is given. One launch takes up to 400 tensors of one combination of types
 * (AdamW) or 1300 of any (norm); others follow in the same stream. */
typedef struct taco_grad_tensor {
  const void* data;
  int64_t n;
  int32_t dtype;
} taco_grad_tensor;

/* out[0] = the square root of the sum of the squares of all elements, out[1] =
 * the factor that clips it: max_norm / out[0] where out[0] > max_norm, else 1,
 * and NaN where out[0] is infinite or NaN (taco_adamw then changes nothing).
 * Squares are formed in fp32 and summed in it 32 at a time at most, those sums in
 * fp64, all in a fixed order. Every finite value counts, whatever its magnitude:
 * out[0] is infinite only where the norm itself lies beyond fp32.
 * max_norm >= 0, infinity included. `workspace`: taco_grad_norm_workspace_bytes
 * bytes, 8-byte aligned, need not be zeroed. */
size_t taco_grad_norm_workspace_bytes(int64_t count);
taco_status taco_grad_norm(const taco_grad_tensor* tensors, int64_t count, double max_norm, float* out,
                           void* workspace, size_t workspace_bytes, void* stream);

/* A parameter with its gradient and states. States in 32 bits: m and v are f32
 * [n], the first and the second moment, and both scales are NULL. In 8 bits: m
 * and v are E4M3 codes [n] (16-byte aligned) of the first moment and of the
 * square ROOT of the second, with one E8M0 scale byte per 128 elements in
 * m_scales and v_scales [ceil(n / 128)]: FP8 block tensors [1, n], tile_rows 1.
 * All start at zero. master (f32 [n], NULL: none) holds a 16-bit parameter's
 * exact value, of which `param` is then the rounded copy. grad_dtype is
 * param_dtype or TACO_DTYPE_F32. */
typedef struct taco_adamw_tensor {
  void* param;
  const void* grad;
  float* master;
  void* m;
  void* v;
  uint8_t* m_scales;
  uint8_t* v_scales;
  int64_t n;
  float weight_decay;
  int32_t param_dtype;
  int32_t grad_dtype;
} taco_adamw_tensor;

/* One AdamW step of all tensors, in place, in fp32. With t = counter[0] + 1,
 * g = grad_scale * grad and x the parameter (or its master):
 *   m = beta1 m + (1 - beta1) g        v = beta2 v + (1 - beta2) g^2
 *   x = x (1 - lr weight_decay) - lr / (1 - beta1^t) m / (sqrt(v / (1 - beta2^t)) + eps)
 * counter (device, int32 [2], zero at first) holds the steps done and a word
 * of the call's own; the call counts one more, as its last act. lr_dev and
 * grad_scale (device, f32; NULL: lr, and 1) are read when the step runs, so a
 * captured call can be replayed with another rate and scale, and takes the next
 * step each time. A grad_scale that is infinite or NaN leaves everything as it
 * was, the counter too.
 * Parameters with a master are rounded to nearest. States in 8 bits, and 16-bit
 * parameters without a master, are rounded to floor(|x| / s + u) s, s the step
 * of the type at x (of E4M3 under the block's scale, chosen as everywhere), by
 * thresholds u = ((i 0xC13FA9A9 + t 0x9E3779B1) mod 2^32) / 2^32 of the element
 * i of a tensor, which take all values in [0, 1) evenly over the steps: changes
 * far below s are kept on average (a 16-bit parameter that this takes beyond its
 * type's largest value becomes infinite). The root of a second moment that is not zero
 * gets no zero code. A block with an infinity or a NaN becomes NaN.
 * v is an f32 number with either form of the states: what lies below 2^-149 is zero,
 * and what lies below 2^-126 a multiple of that. Where (1 - beta2) g^2 is so small,
 * an eps that is not well above |g| is all that the quotient has to go by.
 * 0 <= beta1, beta2 < 1; eps at least 2^-126 (the smallest normal f32). Calls on the
 * same tensors or counter must be in order on one stream. */
taco_status taco_adamw(const taco_adamw_tensor* tensors, int64_t count, double lr, const float* lr_dev,
                       double beta1, double beta2, double eps, const float* grad_scale, int32_t* counter,
                       void* stream);

/* ---- Device faults ---------------------------------------------------------
 * The kernels wait on shared-memory barriers for their bulk copies; each wait
 * gives up after one second of wall-clock time, sets a bit in a device-side
 * fault word of the library, lets the copies still in flight land (again
 * bounded) and returns, so that a fault never hangs the GPU. Bits:
 *   TACO_FAULT_COMPRESS_WAIT, TACO_FAULT_DECOMPRESS_WAIT, TACO_FAULT_SELFTEST_WAIT,
 *   TACO_FAULT_COMPRESS_MMA_WAIT (taco_compress_shards_mma: a wait on a copy,
 *   an MMA or the epilogue gave up; the CTA drains its MMAs and copies and
 *   frees its tensor memory before it returns), TACO_FAULT_DECOMPRESS_MMA_WAIT
 *   (the same for taco_decompress_reduce_mma), TACO_FAULT_FP8_MATMUL_WAIT (the
 *   same for taco_matmul_fp8).
 * taco_get_fault reads (and with clear != 0 resets) the word of the current
 * device; it synchronises with the device. */
#define TACO_FAULT_COMPRESS_WAIT 1u
#define TACO_FAULT_DECOMPRESS_WAIT 2u
#define TACO_FAULT_SELFTEST_WAIT 4u
#define TACO_FAULT_COMPRESS_MMA_WAIT 8u
#define TACO_FAULT_DECOMPRESS_MMA_WAIT 16u
#define TACO_FAULT_FP8_MATMUL_WAIT 32u
taco_status taco_get_fault(uint32_t* bits, int clear);

/* Self-test of that time-out path: one warp waits on a barrier that nothing
 * completes, for limit_ns (1 .. 2e9) nanoseconds, then writes 1 to
 * *status_dev (a device word) and sets TACO_FAULT_SELFTEST_WAIT; 0 would
 * mean the wait completed, which it cannot. */
taco_status taco_selftest_wait_timeout(uint64_t limit_ns, uint32_t* status_dev, void* stream);

/* Human-readable name of a status code (static storage). */
const char* taco_status_string(taco_status status);

/* TACO_ABI_VERSION of the loaded library. */
int taco_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* TACO_H_ */
