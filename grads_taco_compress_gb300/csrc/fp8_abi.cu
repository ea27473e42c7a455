// C ABI of the FP8 block tensors: argument checks and dispatch. Declarations
// and contracts are in taco.h.

#include <cmath>
#include <cstdint>
#include <mutex>

#include "taco_launch.h"

namespace taco {

namespace {

constexpr int64_t kMaxSide = (int64_t{1} << 31) - 256;   // 32-bit coordinates of the tensor copies
constexpr int64_t kMaxElements = int64_t{1} << 40;
constexpr int64_t kMaxNormColumns = 32768;               // 512 threads hold 64 columns each
constexpr int kMaxDevices = 64;
constexpr int32_t kTileRows = 128;

inline uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }
inline bool valid_dtype(int d) { return d == TACO_DTYPE_BF16 || d == TACO_DTYPE_F16 || d == TACO_DTYPE_F32; }
inline int64_t elem(int dtype) { return dtype == TACO_DTYPE_F32 ? 4 : 2; }

// A region of memory: rows of `width` bytes, `pitch` bytes apart.
struct Region {
  uintptr_t p = 0;
  int64_t rows = 0, width = 0, pitch = 0;
  uintptr_t end() const { return p + static_cast<uintptr_t>((rows - 1) * pitch + width); }
  bool empty() const { return rows <= 0 || p == 0; }
  bool same(const Region& o) const {
    return p == o.p && width == o.width && rows == o.rows && (rows == 1 || pitch == o.pitch);
  }
};
// Whether two regions may share a byte. Rows that interleave without touching
// (two halves of one wider matrix) do not.
bool overlap(const Region& a, const Region& b) {
  if (a.empty() || b.empty() || a.p >= b.end() || b.p >= a.end()) return false;
  if (a.pitch == b.pitch && a.pitch > 0) {
    const int64_t pitch = a.pitch;
    const int64_t d = static_cast<int64_t>(b.p >= a.p ? b.p - a.p : a.p - b.p) % pitch;
    const int64_t first = b.p >= a.p ? a.width : b.width, second = b.p >= a.p ? b.width : a.width;
    return !(d >= first && d + second <= pitch);
  }
  return true;
}

// Checks a plain matrix; lowers *vec to what the alignment of its rows allows.
taco_status check_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int dtype, Region* r, int* vec) {
  const int64_t es = elem(dtype);
  if (ld < cols || (rows > 0 && ld > kMaxElements / rows)) return TACO_ERR_SHAPE;
  if (rows > 0 && !p) return TACO_ERR_NULL;
  if (addr(p) % es) return TACO_ERR_ALIGN;
  *r = Region{addr(p), rows, cols * es, ld * es};
  if (vec) {
    const uintptr_t low = addr(p) | (rows > 1 ? static_cast<uintptr_t>(ld * es) : 0);
    const int level = low % 32 == 0 ? kVec32 : low % 16 == 0 ? kVec16 : kVecNone;
    if (level < *vec) *vec = level;
  }
  return TACO_OK;
}

taco_status check_fp8(const taco_fp8_tensor* t, int64_t rows, int64_t cols, bool tile128, Region* codes,
                      Region* scales) {
  if (t->tile_rows != 1 && t->tile_rows != kTileRows) return TACO_ERR_BLOCK;
  if (t->tile_rows != 1 && !tile128) return TACO_ERR_BLOCK;
  if (t->rows != rows || t->cols != cols || rows < 0 || cols < 1) return TACO_ERR_SHAPE;
  if (rows > kMaxSide || cols > kMaxSide) return TACO_ERR_SHAPE;
  const int64_t kb = (cols + 127) / 128, srows = (rows + t->tile_rows - 1) / t->tile_rows;
  if (t->ld_codes < cols || t->ld_scales < kb || t->ld_codes % 16 || t->ld_scales % 4) return TACO_ERR_SHAPE;
  if (rows > 0 && t->ld_codes > kMaxElements / rows) return TACO_ERR_SHAPE;
  if (rows > 0 && (!t->codes || !t->scales)) return TACO_ERR_NULL;
  if (addr(t->codes) % 16 || addr(t->scales) % 4) return TACO_ERR_ALIGN;
  *codes = Region{addr(t->codes), rows, cols, t->ld_codes};
  *scales = Region{addr(t->scales), srows, kb, t->ld_scales};
  return TACO_OK;
}

// Bit i of a set of inputs.
constexpr unsigned input(int i) { return 1u << i; }

// Every output apart from every input and from the other outputs; the first
// output may be one of the inputs in the set `shared`, with the same rows.
taco_status check_apart(const Region* in, int nin, const Region* out, int nout, unsigned shared = 0) {
  for (int o = 0; o < nout; ++o) {
    for (int i = 0; i < nin; ++i)
      if (overlap(out[o], in[i]) && !(o == 0 && (shared & input(i)) && out[o].same(in[i]))) return TACO_ERR_ARG;
    for (int p = 0; p < o; ++p)
      if (overlap(out[o], out[p])) return TACO_ERR_ARG;
  }
  return TACO_OK;
}

std::once_flag g_once[kMaxDevices];
struct DeviceFacts {
  int sms;
  int clusters[9];   // [s]: clusters of s CTAs of the matrix product that run at once
};
DeviceFacts g_device[kMaxDevices];
cudaError_t g_err[kMaxDevices];

// The current device's facts; sets the kernels' attributes on the first call.
cudaError_t device_facts(const DeviceFacts** out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::call_once(g_once[dev], [dev]() {
    cudaError_t err = cudaDeviceGetAttribute(&g_device[dev].sms, cudaDevAttrMultiProcessorCount, dev);
    if (err == cudaSuccess) err = prepare_norm();
    if (err == cudaSuccess) err = prepare_matmul(g_device[dev].clusters);
    g_err[dev] = err;
  });
  *out = &g_device[dev];
  return g_err[dev];
}

inline taco_status done(cudaError_t e) { return e == cudaSuccess ? TACO_OK : TACO_ERR_CUDA; }

#define TACO_TRY(expr)                        \
  do {                                        \
    const taco_status st_ = (expr);           \
    if (st_ != TACO_OK) return st_;           \
  } while (0)

taco_status quantize_common(QuantizeArgs& a, int dtype, int vec, const Region* in, int nin,
                            const taco_fp8_tensor* rows_out, const taco_fp8_tensor* cols_out, void* stream) {
  if (!rows_out && !cols_out) return TACO_ERR_NULL;
  Region out[4];
  a.tile = rows_out ? rows_out->tile_rows : cols_out->tile_rows;
  if (rows_out) {
    TACO_TRY(check_fp8(rows_out, a.M, a.K, true, &out[0], &out[1]));
    a.codes = rows_out->codes;
    a.scales = rows_out->scales;
    a.ldc = rows_out->ld_codes;
    a.lds = rows_out->ld_scales;
  }
  if (cols_out) {
    // a transpose of no rows has no columns: nothing to describe or write
    if (a.M == 0 && cols_out->rows == a.K && cols_out->cols == 0) return TACO_OK;
    TACO_TRY(check_fp8(cols_out, a.K, a.M, true, &out[2], &out[3]));
    if (cols_out->tile_rows != a.tile) return TACO_ERR_BLOCK;
    a.t_codes = cols_out->codes;
    a.t_scales = cols_out->scales;
    a.t_ldc = cols_out->ld_codes;
    a.t_lds = cols_out->ld_scales;
  }
  TACO_TRY(check_apart(in, nin, out, 4));
  if (((a.M + 127) / 128) * ((a.K + 127) / 128) > kMaxSide) return TACO_ERR_SHAPE;
  if (a.M == 0) return TACO_OK;
  return done(launch_quantize(a, dtype, vec, static_cast<cudaStream_t>(stream)));
}

}  // namespace

}  // namespace taco

using namespace taco;

extern "C" {

taco_status taco_fp8_quantize(const void* x, int dtype, int64_t M, int64_t K, int64_t ld,
                              const taco_fp8_tensor* rows_out, const taco_fp8_tensor* cols_out, void* stream) {
  if (!valid_dtype(dtype)) return TACO_ERR_ARG;
  if (M < 0 || K < 1 || M > kMaxSide || K > kMaxSide) return TACO_ERR_SHAPE;
  QuantizeArgs a{};
  Region in;
  int vec = kVec32;
  TACO_TRY(check_matrix(x, M, K, ld, dtype, &in, &vec));
  a.x = x;
  a.ldx = ld;
  a.M = M;
  a.K = K;
  return quantize_common(a, dtype, vec, &in, 1, rows_out, cols_out, stream);
}

taco_status taco_fp8_requantize(const taco_fp8_tensor* x, const taco_fp8_tensor* rows_out,
                                const taco_fp8_tensor* cols_out, void* stream) {
  if (!x) return TACO_ERR_NULL;
  Region in[2];
  TACO_TRY(check_fp8(x, x->rows, x->cols, true, &in[0], &in[1]));
  QuantizeArgs a{};
  a.x = x->codes;
  a.ldx = x->ld_codes;
  a.x_scales = x->scales;
  a.x_lds = x->ld_scales;
  a.x_tile = x->tile_rows;
  a.M = x->rows;
  a.K = x->cols;
  return quantize_common(a, TACO_DTYPE_BF16, kVec32, in, 2, rows_out, cols_out, stream);
}

taco_status taco_rms_norm_fp8(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                              int weight_dtype, int dtype, int64_t M, int64_t H, float eps, void* h_out,
                              int64_t ldh, float* rstd, const taco_fp8_tensor* y,
                              const taco_fp8_tensor* checkpoint, void* stream) {
  if (!valid_dtype(dtype) || !valid_dtype(weight_dtype)) return TACO_ERR_ARG;
  if (!(eps >= 0.0f) || std::isinf(eps)) return TACO_ERR_ARG;
  if (M < 0 || M > kMaxSide || H < 1 || H > kMaxNormColumns) return TACO_ERR_SHAPE;
  if (!y || !weight || (residual != nullptr) != (h_out != nullptr)) return TACO_ERR_NULL;
  Region in[3], out[6];
  int vec = kVec32;
  TACO_TRY(check_matrix(x, M, H, ldx, dtype, &in[0], &vec));
  TACO_TRY(check_matrix(weight, 1, H, H, weight_dtype, &in[1], &vec));
  if (residual) {
    TACO_TRY(check_matrix(residual, M, H, ldr, dtype, &in[2], &vec));
    TACO_TRY(check_matrix(h_out, M, H, ldh, dtype, &out[0], &vec));
  }
  if (rstd) TACO_TRY(check_matrix(rstd, 1, M, M, TACO_DTYPE_F32, &out[1], nullptr));
  TACO_TRY(check_fp8(y, M, H, false, &out[2], &out[3]));
  if (checkpoint) TACO_TRY(check_fp8(checkpoint, M, H, false, &out[4], &out[5]));
  // h_out may be x or residual
  TACO_TRY(check_apart(in, 3, out, 6, input(0) | input(2)));
  if (M == 0) return TACO_OK;
  NormArgs a{};
  a.x = x;
  a.residual = residual;
  a.h = h_out;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldh = ldh;
  a.weight = weight;
  a.weight_dtype = weight_dtype;
  a.eps = eps;
  a.M = M;
  a.H = H;
  a.rstd = rstd;
  a.codes = y->codes;
  a.scales = y->scales;
  a.ldc = y->ld_codes;
  a.lds = y->ld_scales;
  if (checkpoint) {
    a.ck_codes = checkpoint->codes;
    a.ck_scales = checkpoint->scales;
    a.ck_ld = checkpoint->ld_codes;
    a.ck_lds = checkpoint->ld_scales;
  }
  return done(launch_norm(a, dtype, vec, static_cast<cudaStream_t>(stream)));
}

size_t taco_rms_norm_workspace_bytes(int64_t M, int64_t H) {
  if (M < 0 || H < 1 || H > kMaxNormColumns) return 0;
  const int64_t most = norm_max_partials(H), rows = M < 1 ? 1 : M < most ? M : most;
  return static_cast<size_t>(rows) * static_cast<size_t>(H) * sizeof(float);
}

taco_status taco_rms_norm_fp8_backward(const void* dy, int64_t lddy, const taco_fp8_tensor* checkpoint,
                                       const void* h, int64_t ldh, const void* weight, int weight_dtype,
                                       const float* rstd, const void* dh, int64_t lddh, int dtype, int64_t M,
                                       int64_t H, void* dx, int64_t lddx, float* dw, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  if (!valid_dtype(dtype) || !valid_dtype(weight_dtype)) return TACO_ERR_ARG;
  if (M < 0 || M > kMaxSide || H < 1 || H > kMaxNormColumns) return TACO_ERR_SHAPE;
  if ((checkpoint != nullptr) == (h != nullptr)) return TACO_ERR_NULL;
  if (!weight || !dw || (M > 0 && !rstd)) return TACO_ERR_NULL;
  Region in[7], out[3];
  int vec = kVec32;
  TACO_TRY(check_matrix(dy, M, H, lddy, dtype, &in[0], &vec));
  if (checkpoint) TACO_TRY(check_fp8(checkpoint, M, H, false, &in[1], &in[2]));
  if (h) TACO_TRY(check_matrix(h, M, H, ldh, dtype, &in[3], &vec));
  TACO_TRY(check_matrix(weight, 1, H, H, weight_dtype, &in[4], &vec));
  if (M > 0) TACO_TRY(check_matrix(rstd, 1, M, M, TACO_DTYPE_F32, &in[5], nullptr));
  if (dh) TACO_TRY(check_matrix(dh, M, H, lddh, dtype, &in[6], &vec));
  TACO_TRY(check_matrix(dx, M, H, lddx, dtype, &out[0], &vec));
  TACO_TRY(check_matrix(dw, 1, H, H, TACO_DTYPE_F32, &out[1], nullptr));
  const size_t need = taco_rms_norm_workspace_bytes(M, H);
  if (!workspace || workspace_bytes < need) return TACO_ERR_WORKSPACE;
  if (addr(workspace) % 16) return TACO_ERR_ALIGN;
  out[2] = Region{addr(workspace), 1, static_cast<int64_t>(need), static_cast<int64_t>(need)};
  // dx may be dy, h or dh
  TACO_TRY(check_apart(in, 7, out, 3, input(0) | input(3) | input(6)));
  NormBackwardArgs a{};
  a.dy = dy;
  a.h = h;
  a.dh = dh;
  a.dx = dx;
  a.lddy = lddy;
  a.ldh = ldh;
  a.lddh = lddh;
  a.lddx = lddx;
  if (checkpoint) {
    a.ck_codes = checkpoint->codes;
    a.ck_scales = checkpoint->scales;
    a.ck_ld = checkpoint->ld_codes;
    a.ck_lds = checkpoint->ld_scales;
  }
  a.weight = weight;
  a.weight_dtype = weight_dtype;
  a.rstd = rstd;
  a.M = M;
  a.H = H;
  a.partial = static_cast<float*>(workspace);
  a.dw = dw;
  const DeviceFacts* dev = nullptr;
  if (device_facts(&dev) != cudaSuccess) return TACO_ERR_CUDA;
  const int grid = norm_backward_ctas(M, H, dev->sms);
  return done(launch_norm_backward(a, dtype, vec, grid, static_cast<cudaStream_t>(stream)));
}

taco_status taco_swiglu_fp8(const void* gate, int64_t ldg, const void* up, int64_t ldu, int dtype, int64_t M,
                            int64_t F, const taco_fp8_tensor* y, const taco_fp8_tensor* checkpoint_gate,
                            const taco_fp8_tensor* checkpoint_up, void* stream) {
  if (!valid_dtype(dtype)) return TACO_ERR_ARG;
  if (M < 0 || F < 1 || M > kMaxSide || F > kMaxSide) return TACO_ERR_SHAPE;
  if (!y || (checkpoint_gate != nullptr) != (checkpoint_up != nullptr)) return TACO_ERR_NULL;
  Region in[2], out[6];
  int vec = kVec32;
  TACO_TRY(check_matrix(gate, M, F, ldg, dtype, &in[0], &vec));
  TACO_TRY(check_matrix(up, M, F, ldu, dtype, &in[1], &vec));
  TACO_TRY(check_fp8(y, M, F, false, &out[0], &out[1]));
  if (checkpoint_gate) {
    TACO_TRY(check_fp8(checkpoint_gate, M, F, false, &out[2], &out[3]));
    TACO_TRY(check_fp8(checkpoint_up, M, F, false, &out[4], &out[5]));
  }
  TACO_TRY(check_apart(in, 2, out, 6));
  if (M == 0) return TACO_OK;
  SwigluArgs a{};
  a.gate = gate;
  a.up = up;
  a.ldg = ldg;
  a.ldu = ldu;
  a.M = M;
  a.F = F;
  a.codes = y->codes;
  a.scales = y->scales;
  a.ldc = y->ld_codes;
  a.lds = y->ld_scales;
  if (checkpoint_gate) {
    a.g_codes = checkpoint_gate->codes;
    a.g_scales = checkpoint_gate->scales;
    a.g_ld = checkpoint_gate->ld_codes;
    a.g_lds = checkpoint_gate->ld_scales;
    a.u_codes = checkpoint_up->codes;
    a.u_scales = checkpoint_up->scales;
    a.u_ld = checkpoint_up->ld_codes;
    a.u_lds = checkpoint_up->ld_scales;
  }
  return done(launch_swiglu(a, dtype, vec, static_cast<cudaStream_t>(stream)));
}

taco_status taco_swiglu_fp8_backward(const void* dy, int64_t lddy, const taco_fp8_tensor* checkpoint_gate,
                                     const taco_fp8_tensor* checkpoint_up, int dtype, int64_t M, int64_t F,
                                     void* dgate, int64_t lddg, void* dup, int64_t lddu, void* stream) {
  if (!valid_dtype(dtype)) return TACO_ERR_ARG;
  if (M < 0 || F < 1 || M > kMaxSide || F > kMaxSide) return TACO_ERR_SHAPE;
  if (!checkpoint_gate || !checkpoint_up) return TACO_ERR_NULL;
  Region in[5], out[2];
  int vec = kVec32;
  TACO_TRY(check_matrix(dy, M, F, lddy, dtype, &in[0], &vec));
  TACO_TRY(check_fp8(checkpoint_gate, M, F, false, &in[1], &in[2]));
  TACO_TRY(check_fp8(checkpoint_up, M, F, false, &in[3], &in[4]));
  TACO_TRY(check_matrix(dgate, M, F, lddg, dtype, &out[0], &vec));
  TACO_TRY(check_matrix(dup, M, F, lddu, dtype, &out[1], &vec));
  // one of the two may be dy itself; the outputs stay apart from each other
  if (overlap(out[0], out[1])) return TACO_ERR_ARG;
  TACO_TRY(check_apart(in, 5, out, 1, input(0)));
  TACO_TRY(check_apart(in, 5, out + 1, 1, input(0)));
  if (M == 0) return TACO_OK;
  SwigluBackwardArgs a{};
  a.dy = dy;
  a.lddy = lddy;
  a.M = M;
  a.F = F;
  a.g_codes = checkpoint_gate->codes;
  a.g_scales = checkpoint_gate->scales;
  a.g_ld = checkpoint_gate->ld_codes;
  a.g_lds = checkpoint_gate->ld_scales;
  a.u_codes = checkpoint_up->codes;
  a.u_scales = checkpoint_up->scales;
  a.u_ld = checkpoint_up->ld_codes;
  a.u_lds = checkpoint_up->ld_scales;
  a.dgate = dgate;
  a.dup = dup;
  a.lddg = lddg;
  a.lddu = lddu;
  return done(launch_swiglu_backward(a, dtype, vec, static_cast<cudaStream_t>(stream)));
}

taco_status taco_matmul_fp8(const taco_fp8_tensor* a, const taco_fp8_tensor* b, const void* add, int64_t ldadd,
                            void* out, int64_t ldo, int dtype, void* stream) {
  if (!a || !b) return TACO_ERR_NULL;
  if (!valid_dtype(dtype)) return TACO_ERR_ARG;
  if (a->cols != b->cols) return TACO_ERR_SHAPE;
  Region in[5], o;
  TACO_TRY(check_fp8(a, a->rows, a->cols, true, &in[0], &in[1]));
  TACO_TRY(check_fp8(b, b->rows, b->cols, true, &in[2], &in[3]));
  const int64_t M = a->rows, N = b->rows;
  int vec_add = kVec32, vec_out = kVec32;
  if (add) TACO_TRY(check_matrix(add, M, N, ldadd, dtype, &in[4], &vec_add));
  if (N > 0) TACO_TRY(check_matrix(out, M, N, ldo, dtype, &o, &vec_out));
  TACO_TRY(check_apart(in, 5, &o, 1, input(4)));   // out may be add
  if (M == 0 || N == 0) return TACO_OK;
  if (((M + 127) / 128) * ((N + 127) / 128) > kMaxSide) return TACO_ERR_SHAPE;
  MatmulArgs m{};
  m.a = a->codes;
  m.b = b->codes;
  m.lda = a->ld_codes;
  m.ldb = b->ld_codes;
  m.sa = a->scales;
  m.sb = b->scales;
  m.lda_s = a->ld_scales;
  m.ldb_s = b->ld_scales;
  m.tile_a = a->tile_rows;
  m.tile_b = b->tile_rows;
  m.M = M;
  m.N = N;
  m.K = a->cols;
  m.add = add;
  m.ldadd = ldadd;
  m.out = out;
  m.ldo = ldo;
  m.vec_sa = addr(a->scales) % 16 == 0 && a->ld_scales % 16 == 0;
  m.vec_sb = addr(b->scales) % 16 == 0 && b->ld_scales % 16 == 0;
  m.vec_add = vec_add != kVecNone;
  m.tma_add = vec_add != kVecNone && (ldadd * elem(dtype)) % 16 == 0;
  // a tensor map wants a row stride of 16 bytes even where there is one row
  m.tma_out = vec_out != kVecNone && (ldo * elem(dtype)) % 16 == 0;
  const DeviceFacts* dev = nullptr;
  if (device_facts(&dev) != cudaSuccess) return TACO_ERR_CUDA;
  return done(launch_matmul(m, dtype, dev->sms, dev->clusters, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
