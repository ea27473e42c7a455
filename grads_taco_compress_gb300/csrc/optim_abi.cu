// C ABI of the calls over many tensors (AdamW step, gradient norm): argument
// checks, grouping into launches. Declarations and contracts are in taco.h.

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <limits>
#include <memory>

#include "taco_launch.h"

namespace taco {

namespace {

constexpr int64_t kMaxElements = int64_t{1} << 40;   // of all tensors of a call together
constexpr int64_t kMaxTensors = int64_t{1} << 20;
constexpr int64_t kChunk = 4096;                     // elements, kOptimChunk of the kernels

inline uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }
inline bool valid_dtype(int d) { return d == TACO_DTYPE_BF16 || d == TACO_DTYPE_F16 || d == TACO_DTYPE_F32; }
inline int64_t elem(int dtype) { return dtype == TACO_DTYPE_F32 ? 4 : 2; }
inline taco_status done(cudaError_t e) { return e == cudaSuccess ? TACO_OK : TACO_ERR_CUDA; }

cudaError_t multiprocessors(int* sms) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  return e != cudaSuccess ? e : cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
}

// Host memory that the C entries need; nothing here throws.
struct Free {
  void operator()(void* p) const { std::free(p); }
};
template <typename T>
std::unique_ptr<T[], Free> host_array(int64_t n) {
  return std::unique_ptr<T[], Free>(static_cast<T*>(std::malloc(static_cast<size_t>(n ? n : 1) * sizeof(T))));
}

struct Span {
  uintptr_t begin, end;
  bool written;
};
void add_span(Span* s, int64_t* n, const void* p, int64_t bytes, bool written) {
  if (p && bytes > 0) s[(*n)++] = Span{addr(p), addr(p) + static_cast<uintptr_t>(bytes), written};
}
// Whether what is written shares no byte with anything else.
bool apart(Span* s, int64_t n) {
  std::sort(s, s + n, [](const Span& a, const Span& b) { return a.begin < b.begin; });
  uintptr_t any = 0, written = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (s[i].begin < written || (s[i].written && s[i].begin < any)) return false;
    any = std::max(any, s[i].end);
    if (s[i].written) written = std::max(written, s[i].end);
  }
  return true;
}

taco_status check(const taco_adamw_tensor& t) {
  if (!valid_dtype(t.param_dtype) || !valid_dtype(t.grad_dtype)) return TACO_ERR_ARG;
  if (t.grad_dtype != t.param_dtype && t.grad_dtype != TACO_DTYPE_F32) return TACO_ERR_ARG;
  if (t.master && t.param_dtype == TACO_DTYPE_F32) return TACO_ERR_ARG;
  if (!std::isfinite(t.weight_decay)) return TACO_ERR_ARG;
  if (t.n < 0 || t.n > kMaxElements) return TACO_ERR_SHAPE;
  if (t.n == 0) return TACO_OK;
  if (!t.param || !t.grad || !t.m || !t.v) return TACO_ERR_NULL;
  if ((t.m_scales != nullptr) != (t.v_scales != nullptr)) return TACO_ERR_NULL;
  const uintptr_t state = t.m_scales ? 16 : 4;
  if (addr(t.param) % elem(t.param_dtype) || addr(t.grad) % elem(t.grad_dtype) || addr(t.master) % 4 ||
      addr(t.m) % state || addr(t.v) % state)
    return TACO_ERR_ALIGN;
  return TACO_OK;
}
// Which launch a tensor belongs to: types, form of the states, alignment.
uintptr_t low_bits(const taco_adamw_tensor& t) {
  const uintptr_t states = t.m_scales ? 0 : addr(t.m) | addr(t.v);
  return addr(t.param) | addr(t.grad) | addr(t.master) | states;
}
constexpr int kKinds = 24;
int kind_of(const taco_adamw_tensor& t) {
  return ((t.param_dtype * 2 + (t.grad_dtype == TACO_DTYPE_F32)) * 2 + (t.m_scales != nullptr)) * 2 +
         (low_bits(t) % 16 == 0);
}

}  // namespace

}  // namespace taco

using namespace taco;

extern "C" {

taco_status taco_adamw(const taco_adamw_tensor* tensors, int64_t count, double lr, const float* lr_dev, double beta1,
                       double beta2, double eps, const float* grad_scale, int32_t* counter, void* stream) {
  if (count < 0 || count > kMaxTensors) return TACO_ERR_SHAPE;
  if ((count > 0 && !tensors) || !counter) return TACO_ERR_NULL;
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0)) return TACO_ERR_ARG;
  const float eps32 = static_cast<float>(eps);
  if (!(eps32 >= std::numeric_limits<float>::min()) || std::isinf(eps32)) return TACO_ERR_ARG;
  if (!lr_dev && !std::isfinite(static_cast<float>(lr))) return TACO_ERR_ARG;
  if (addr(counter) % 4 || addr(lr_dev) % 4 || addr(grad_scale) % 4) return TACO_ERR_ALIGN;
  int64_t total = 0, members[kKinds] = {};
  for (int64_t i = 0; i < count; ++i) {
    const taco_status st = check(tensors[i]);
    if (st != TACO_OK) return st;
    total += tensors[i].n;
    if (total > kMaxElements) return TACO_ERR_SHAPE;
    if (tensors[i].n) ++members[kind_of(tensors[i])];
  }
  const auto spans = host_array<Span>(7 * count + 3);
  if (!spans) return TACO_ERR_CUDA;
  int64_t n = 0;
  add_span(spans.get(), &n, counter, 8, true);
  add_span(spans.get(), &n, lr_dev, 4, false);
  add_span(spans.get(), &n, grad_scale, 4, false);
  for (int64_t i = 0; i < count; ++i) {
    const taco_adamw_tensor& t = tensors[i];
    const int64_t state = t.m_scales ? t.n : 4 * t.n, blocks = t.m_scales && t.n ? (t.n + 127) / 128 : 0;
    add_span(spans.get(), &n, t.param, t.n * elem(t.param_dtype), true);
    add_span(spans.get(), &n, t.grad, t.n * elem(t.grad_dtype), false);
    add_span(spans.get(), &n, t.master, 4 * t.n, true);
    add_span(spans.get(), &n, t.m, state, true);
    add_span(spans.get(), &n, t.v, state, true);
    add_span(spans.get(), &n, t.m_scales, blocks, true);
    add_span(spans.get(), &n, t.v_scales, blocks, true);
  }
  if (!apart(spans.get(), n)) return TACO_ERR_ARG;

  AdamwArgs a{};
  a.b1 = static_cast<float>(beta1);
  a.one_b1 = static_cast<float>(1.0 - beta1);
  a.b2 = static_cast<float>(beta2);
  a.one_b2 = static_cast<float>(1.0 - beta2);
  a.log_b1 = static_cast<float>(std::log(beta1));
  a.log_b2 = static_cast<float>(std::log(beta2));
  a.eps = eps32;
  a.lr = static_cast<float>(lr);
  a.lr_dev = lr_dev;
  a.factor = grad_scale;
  a.counter = counter;
  int sms = 0;
  if (multiprocessors(&sms) != cudaSuccess) return TACO_ERR_CUDA;
  const auto st = static_cast<cudaStream_t>(stream);
  int64_t launches = 0;
  for (const int64_t m : members) launches += (m + kAdamwMany - 1) / kAdamwMany;
  if (launches == 0) {   // no element: the step counts all the same
    a.last = true;
    return done(launch_adamw(a, nullptr, 0, TACO_DTYPE_F32, TACO_DTYPE_F32, false, true, sms, st));
  }
  AdamwEntry entries[kAdamwMany];
  for (int kind = 0; kind < kKinds; ++kind) {
    int64_t left = members[kind];
    int filled = 0;
    a.chunks = 0;
    for (int64_t i = 0; left > 0; ++i) {
      const taco_adamw_tensor& t = tensors[i];
      if (t.n == 0 || kind_of(t) != kind) continue;
      entries[filled++] = AdamwEntry{t.param,    t.grad,     t.master, t.m, t.v, t.m_scales, t.v_scales, t.n,
                                     a.chunks, t.weight_decay, low_bits(t) % 32 == 0};
      a.chunks += static_cast<uint32_t>((t.n + kChunk - 1) / kChunk);
      if (--left && filled < kAdamwMany) continue;
      a.last = --launches == 0;
      if (launch_adamw(a, entries, filled, t.param_dtype, t.grad_dtype, t.m_scales != nullptr, kind & 1, sms, st) !=
          cudaSuccess)
        return TACO_ERR_CUDA;
      filled = 0;
      a.chunks = 0;
    }
  }
  return TACO_OK;
}

size_t taco_grad_norm_workspace_bytes(int64_t count) {
  if (count < 0 || count > kMaxTensors) return 0;
  const int64_t launches = count ? (count + kNormMany - 1) / kNormMany : 1;
  return static_cast<size_t>(launches) * kNormCtas * sizeof(double);
}

taco_status taco_grad_norm(const taco_grad_tensor* tensors, int64_t count, double max_norm, float* out,
                           void* workspace, size_t workspace_bytes, void* stream) {
  if (count < 0 || count > kMaxTensors) return TACO_ERR_SHAPE;
  if ((count > 0 && !tensors) || !out) return TACO_ERR_NULL;
  if (!(max_norm >= 0.0)) return TACO_ERR_ARG;
  const size_t need = taco_grad_norm_workspace_bytes(count);
  if (!workspace || workspace_bytes < need) return TACO_ERR_WORKSPACE;
  if (addr(workspace) % 8 || addr(out) % 4) return TACO_ERR_ALIGN;
  const auto spans = host_array<Span>(count + 2);
  if (!spans) return TACO_ERR_CUDA;
  int64_t n = 0, total = 0, present = 0;
  add_span(spans.get(), &n, out, 8, true);
  add_span(spans.get(), &n, workspace, static_cast<int64_t>(need), true);
  for (int64_t i = 0; i < count; ++i) {
    const taco_grad_tensor& t = tensors[i];
    if (!valid_dtype(t.dtype)) return TACO_ERR_ARG;
    if (t.n < 0 || t.n > kMaxElements || (total += t.n) > kMaxElements) return TACO_ERR_SHAPE;
    if (t.n == 0) continue;
    if (!t.data) return TACO_ERR_NULL;
    if (addr(t.data) % elem(t.dtype)) return TACO_ERR_ALIGN;
    add_span(spans.get(), &n, t.data, t.n * elem(t.dtype), false);
    ++present;
  }
  if (!apart(spans.get(), n)) return TACO_ERR_ARG;
  int sms = 0;
  if (multiprocessors(&sms) != cudaSuccess) return TACO_ERR_CUDA;
  const auto st = static_cast<cudaStream_t>(stream);
  double* partial = static_cast<double*>(workspace);
  int sums = 0;
  GradEntry entries[kNormMany];
  for (int64_t i = 0; present > 0;) {
    int filled = 0;
    uint32_t chunks = 0;
    for (; filled < kNormMany && present > 0; ++i) {
      const taco_grad_tensor& t = tensors[i];
      if (t.n == 0) continue;
      entries[filled++] = GradEntry{t.data, t.n, chunks, static_cast<int16_t>(t.dtype), addr(t.data) % 16 == 0,
                                    addr(t.data) % 32 == 0};
      const int64_t chunk = kNormChunkBytes / elem(t.dtype);
      chunks += static_cast<uint32_t>((t.n + chunk - 1) / chunk);
      --present;
    }
    int ctas = 0;
    if (launch_grad_squares(entries, filled, chunks, sms, partial + sums, &ctas, st) != cudaSuccess)
      return TACO_ERR_CUDA;
    sums += ctas;
  }
  return done(launch_grad_norm(partial, sums, static_cast<float>(max_norm), out, st));
}

}  // extern "C"
