// Compiled argument marshalling of the FP8 block-tensor entry points (fp8.py).
//
// These calls take and return several tensors each and run for a few
// microseconds on small inputs, where building the arguments in Python took
// longer than the launch (20 us for the norm of 4 rows, 3.3 us of them in the
// library). As in binding.py, nothing computes here: tensors are checked and
// described, outputs allocated through torch, and the library of taco.h is
// called on the current stream.
//
// Every function returns what its Python entry point does (None for what there
// is not), or the int status of a library call that failed; wrong arguments
// raise ValueError.

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <exception>
#include <initializer_list>
#include <optional>
#include <stdexcept>
#include <string>

#include <ATen/ATen.h>
#include <ATen/EmptyTensor.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "taco.h"

namespace {

constexpr int64_t kBlock = 128;

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

int64_t up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }

bool given(PyObject* o) { return o && o != Py_None; }

bool flag(PyObject* o, const char* what) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    refuse(std::string(what) + " must be true or false");
  }
  return v != 0;
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse(std::string(what) + " must be a tensor");
  return THPVariable_Unpack(o);
}

int dtype_of(at::ScalarType t) {
  return t == at::kBFloat16 ? TACO_DTYPE_BF16 : t == at::kHalf ? TACO_DTYPE_F16 : t == at::kFloat ? TACO_DTYPE_F32 : -1;
}

struct Matrix {
  void* p = nullptr;
  int64_t rows = 0, cols = 0, ld = 0;
  int dtype = 0;
};

Matrix matrix(const at::Tensor& t, const char* what) {
  Matrix m;
  m.dtype = dtype_of(t.scalar_type());
  if (!t.is_cuda() || m.dtype < 0 || t.dim() != 2)
    refuse(std::string(what) + " must be a 2-D bf16, f16 or f32 CUDA tensor");
  m.rows = t.size(0);
  m.cols = t.size(1);
  if (m.cols > 1 && t.stride(1) != 1) refuse(std::string(what) + " must have contiguous columns");
  m.ld = m.rows > 1 ? t.stride(0) : (m.cols > 1 ? m.cols : 1);
  m.p = t.data_ptr();
  return m;
}

// A matrix of the shape and type of another.
Matrix like(const at::Tensor& t, const char* what, int64_t rows, int64_t cols, int dtype) {
  const Matrix m = matrix(t, what);
  if (m.rows != rows || m.cols != cols)
    refuse(std::string(what) + " must have shape (" + std::to_string(rows) + ", " + std::to_string(cols) + ")");
  if (m.dtype != dtype) refuse(std::string(what) + " has another type than the call's");
  return m;
}

void* vector(const at::Tensor& t, const char* what, int64_t n, bool f32) {
  if (!t.is_cuda() || dtype_of(t.scalar_type()) < 0 || t.dim() != 1 || t.size(0) != n || !t.is_contiguous() ||
      (f32 && t.scalar_type() != at::kFloat))
    refuse(std::string(what) + " must be a contiguous " + (f32 ? "f32 " : "") + "CUDA tensor [" + std::to_string(n) +
           "]");
  return t.data_ptr();
}

// Checks an FP8 block tensor (a plane of it where it has three dimensions) and
// describes it. The scales of a single row have the same shape in both tilings:
// one_row_tile then.
taco_fp8_tensor describe(const at::Tensor& codes, const at::Tensor& scales, const char* what, int one_row_tile = 1,
                         int dims = 2, int64_t plane = 0) {
  if (codes.dim() != dims || scales.dim() != dims || codes.scalar_type() != at::kByte ||
      scales.scalar_type() != at::kByte)
    refuse(std::string(what) + " must be " + std::to_string(dims) + "-D uint8 codes and scales");
  if (!codes.is_cuda() || !scales.is_cuda()) refuse(std::string(what) + " must be CUDA tensors");
  const int r = dims - 2, c = dims - 1;
  taco_fp8_tensor t{};
  t.rows = codes.size(r);
  t.cols = codes.size(c);
  const int64_t srows = scales.size(r), kb = scales.size(c);
  t.tile_rows = srows != t.rows ? kBlock : t.rows == 1 ? one_row_tile : 1;
  if (srows != (t.rows + t.tile_rows - 1) / t.tile_rows || kb != (t.cols + kBlock - 1) / kBlock)
    refuse(std::string(what) + ": the scales' shape does not fit the codes'");
  if ((t.cols > 1 && codes.stride(c) != 1) || (kb > 1 && scales.stride(c) != 1))
    refuse(std::string(what) + " must have contiguous columns");
  t.ld_codes = t.rows > 1 ? codes.stride(r) : up(t.cols, 16);
  t.ld_scales = srows > 1 ? scales.stride(r) : up(kb, 4);
  t.codes = static_cast<uint8_t*>(codes.data_ptr()) + (dims == 3 ? plane * codes.stride(0) : 0);
  t.scales = static_cast<uint8_t*>(scales.data_ptr()) + (dims == 3 ? plane * scales.stride(0) : 0);
  return t;
}

// The two tensors of an Fp8Tensor (a Python tuple).
struct Pair {
  at::Tensor codes, scales;
};
Pair pair_of(PyObject* o, const char* what) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 2) refuse(std::string(what) + " must be an Fp8Tensor");
  return {tensor(PyTuple_GET_ITEM(o, 0), what), tensor(PyTuple_GET_ITEM(o, 1), what)};
}

// A new tensor on the current device (the call's: see OnStream), straight from
// torch's caching allocator: the dispatcher on the way to it costs as much again.
at::Tensor empty_strided(at::IntArrayRef shape, at::IntArrayRef strides, at::ScalarType type) {
  return at::detail::empty_strided_generic(shape, strides, c10::cuda::CUDACachingAllocator::get(),
                                           c10::DispatchKeySet(c10::DispatchKey::CUDA), type);
}
at::Tensor empty_matrix(int64_t rows, int64_t cols, at::ScalarType type) {
  return empty_strided({rows, cols}, {cols > 1 ? cols : 1, 1}, type);
}
at::Tensor empty_vector(int64_t n, at::ScalarType type) { return empty_strided({n}, {1}, type); }
void lay_out(const at::Tensor& t, at::IntArrayRef shape, at::IntArrayRef strides, int64_t offset) {
  t.unsafeGetTensorImpl()->set_sizes_and_strides(shape, strides, offset);
}
// A tensor in the allocation of another, from the byte `at` (a multiple of its element) on.
at::Tensor part(const at::Tensor& whole, int64_t at, at::IntArrayRef shape, at::IntArrayRef strides,
                at::ScalarType type) {
  const caffe2::TypeMeta meta = c10::scalarTypeToTypeMeta(type);
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(whole.storage()),
                                                          whole.key_set(), meta);
  lay_out(t, shape, strides, at / static_cast<int64_t>(meta.itemsize()));
  return t;
}
// Codes and scales of a new FP8 block tensor, rows of either on 16 bytes (which a
// product reads fastest), in one allocation: they live and die together, and an
// allocation costs more than the rest of such a call's arguments. A norm's
// checkpoint has its rstd there too, which the backward pass reads with it.
Pair new_fp8(at::IntArrayRef shape, int64_t tile, at::Tensor* rstd = nullptr) {
  const int64_t cols = shape.back(), rows = shape[shape.size() - 2], planes = shape.size() == 3 ? shape[0] : 1;
  const int64_t kb = (cols + kBlock - 1) / kBlock, srows = (rows + tile - 1) / tile;
  const int64_t ld = up(cols, 16), lds = up(kb, 16), at = up(planes * rows * ld, 256);
  const int64_t end = at + planes * srows * lds;  // a multiple of 16
  const at::Tensor codes = empty_vector(end + (rstd ? 4 * rows : 0), at::kByte);
  if (rstd) *rstd = part(codes, end, {rows}, {1}, at::kFloat);
  if (shape.size() == 3) {
    lay_out(codes, {planes, rows, cols}, {rows * ld, ld, 1}, 0);
    return {codes, part(codes, at, {planes, srows, kb}, {srows * lds, lds, 1}, at::kByte)};
  }
  lay_out(codes, {rows, cols}, {ld, 1}, 0);
  return {codes, part(codes, at, {srows, kb}, {lds, 1}, at::kByte)};
}

// The device of `t` and the stream of the call (the current one, or the one
// whose handle is given) made current for its length: what the call allocates
// belongs to that stream, so that memory freed after the call (a workspace
// above all) is not handed out on another one while the kernels still use it.
class OnStream {
 public:
  OnStream(PyObject* handle, const at::Tensor& t) : device_(t.device()) {
    if (!given(handle)) return;
    void* p = PyLong_AsVoidPtr(handle);
    if (!p && PyErr_Occurred()) {
      PyErr_Clear();
      refuse("stream must be a CUDA stream");
    }
    stream_.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(p), t.device().index()));
  }
  void* handle() const { return c10::cuda::getCurrentCUDAStream().stream(); }

 private:
  c10::cuda::OptionalCUDAGuard device_;
  c10::cuda::OptionalCUDAStreamGuard stream_;
};

// fp8.py's Fp8Tensor and RmsNormOutput (named tuples), given by it once.
PyTypeObject *fp8_type = nullptr, *norm_type = nullptr;

PyObject* none() {
  Py_INCREF(Py_None);
  return Py_None;
}
PyObject* object(const at::Tensor& t) { return THPVariable_Wrap(t); }

// A tuple, or one of the types above, of `items`, whose references it takes.
PyObject* tuple(PyTypeObject* type, std::initializer_list<PyObject*> items) {
  PyObject* t = type->tp_alloc(type, static_cast<Py_ssize_t>(items.size()));
  Py_ssize_t n = 0;
  bool whole = t != nullptr;
  for (PyObject* o : items) {
    whole = whole && o;
    if (t)
      PyTuple_SET_ITEM(t, n++, o);
    else
      Py_XDECREF(o);
  }
  if (whole) return t;
  Py_XDECREF(t);
  return nullptr;
}
PyObject* object(const std::optional<Pair>& p) {
  return p ? tuple(fp8_type, {object(p->codes), object(p->scales)}) : none();
}

template <typename F>
taco_status call(F&& f) {
  taco_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  return st;
}

// The CUDA tensors among the arguments, those in an Fp8Tensor included, all on
// one device: the call's kernels run on the first's and take the others'
// addresses as they are. (What is no CUDA tensor is refused where it is read.)
void on_one_device(PyObject* const* v, Py_ssize_t n) {
  std::optional<c10::Device> device;
  const auto check = [&](PyObject* o) {
    if (!THPVariable_Check(o)) return;
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) return;
    if (!device) device = t.device();
    if (*device != t.device())
      refuse("the tensors of a call must be on one device, not on " + device->str() + " and " + t.device().str());
  };
  for (Py_ssize_t i = 0; i < n; ++i) {
    if (PyTuple_Check(v[i]))
      for (Py_ssize_t j = 0; j < PyTuple_GET_SIZE(v[i]); ++j) check(PyTuple_GET_ITEM(v[i], j));
    else
      check(v[i]);
  }
}

// Runs `body` on `count` positional arguments; C++ exceptions become Python's.
template <typename F>
PyObject* guarded(PyObject* const* v, Py_ssize_t got, Py_ssize_t count, F&& body) {
  if (got != count) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", count, got);
    return nullptr;
  }
  try {
    at::AutoDispatchBelowADInplaceOrView guard;
    on_one_device(v, got);
    return body();
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// quantize(x, rows, cols, tile, out, out_t, stream) -> rows, transpose
PyObject* quantize(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(v, n, 7, [&]() -> PyObject* {
    const bool rows = flag(v[1], "rows"), cols = flag(v[2], "cols");
    const long tile = PyLong_AsLong(v[3]);
    if (PyErr_Occurred()) PyErr_Clear();
    if (tile != 1 && tile != kBlock) refuse("tile must be 1 or 128");
    std::optional<Pair> source;
    Matrix m;
    int64_t M, K;
    taco_fp8_tensor from{};
    at::Tensor x;
    if (PyTuple_Check(v[0])) {
      source = pair_of(v[0], "x");
      from = describe(source->codes, source->scales, "x");
      M = from.rows;
      K = from.cols;
      x = source->codes;
    } else {
      x = tensor(v[0], "x");
      m = matrix(x, "x");
      M = m.rows;
      K = m.cols;
    }
    const OnStream on(v[6], x);
    std::optional<Pair> out, out_t;
    if (rows) out = given(v[4]) ? pair_of(v[4], "out") : new_fp8({M, K}, tile);
    if (cols) out_t = given(v[5]) ? pair_of(v[5], "out_t") : new_fp8({K, M}, tile);
    taco_fp8_tensor a{}, b{};
    if (out) a = describe(out->codes, out->scales, "out", tile);
    if (out_t) b = describe(out_t->codes, out_t->scales, "out_t", tile);
    void* stream = on.handle();
    const taco_status st = call([&] {
      return source ? taco_fp8_requantize(&from, out ? &a : nullptr, out_t ? &b : nullptr, stream)
                    : taco_fp8_quantize(m.p, m.dtype, M, K, m.ld, out ? &a : nullptr, out_t ? &b : nullptr, stream);
    });
    if (st != TACO_OK) return PyLong_FromLong(st);
    return tuple(&PyTuple_Type, {object(out), object(out_t)});
  });
}

// rms_norm(x, weight, residual, eps, checkpoint, out, h, rstd, stream)
//   -> y, h, rstd, checkpoint
PyObject* rms_norm(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(v, n, 9, [&]() -> PyObject* {
    const at::Tensor& x = tensor(v[0], "x");
    const Matrix m = matrix(x, "x");
    const bool keep = PyTuple_Check(v[4]) || flag(v[4], "checkpoint");
    const OnStream on(v[8], x);
    const at::Tensor& weight = tensor(v[1], "weight");
    void* w = vector(weight, "weight", m.cols, false);
    const double eps = PyFloat_AsDouble(v[3]);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      refuse("eps must be a number");
    }
    // A new rstd lies with the new tensor that lives as long: the checkpoint, else h.
    at::Tensor h = x, rstd;
    if (given(v[7])) rstd = tensor(v[7], "rstd");
    std::optional<Pair> ck;
    if (PyTuple_Check(v[4]))
      ck = pair_of(v[4], "checkpoint");
    else if (keep)
      ck = new_fp8({m.rows, m.cols}, 1, rstd.defined() ? nullptr : &rstd);
    Matrix r, ho;
    if (given(v[2])) {
      r = like(tensor(v[2], "residual"), "residual", m.rows, m.cols, m.dtype);
      if (given(v[6])) {
        h = tensor(v[6], "h");
      } else {
        const int64_t end = up(m.rows * m.cols * x.element_size(), 16);
        const at::Tensor whole = empty_vector(end + (rstd.defined() ? 0 : 4 * m.rows), at::kByte);
        h = part(whole, 0, {m.rows, m.cols}, {m.cols > 1 ? m.cols : 1, 1}, x.scalar_type());
        if (!rstd.defined()) rstd = part(whole, end, {m.rows}, {1}, at::kFloat);
      }
      ho = like(h, "h", m.rows, m.cols, m.dtype);
    } else if (given(v[6])) {
      refuse("h is an output of the residual's addition: pass residual too");
    }
    if (!rstd.defined()) rstd = empty_vector(m.rows, at::kFloat);
    void* rs = vector(rstd, "rstd", m.rows, true);
    const Pair y = given(v[5]) ? pair_of(v[5], "out") : new_fp8({m.rows, m.cols}, 1);
    const taco_fp8_tensor yd = describe(y.codes, y.scales, "out");
    taco_fp8_tensor cd{};
    if (ck) cd = describe(ck->codes, ck->scales, "checkpoint");
    void* stream = on.handle();
    const taco_status st = call([&] {
      return taco_rms_norm_fp8(m.p, m.ld, r.p, r.ld, w, dtype_of(weight.scalar_type()), m.dtype, m.rows, m.cols,
                               static_cast<float>(eps), ho.p, ho.ld, static_cast<float*>(rs), &yd, ck ? &cd : nullptr,
                               stream);
    });
    if (st != TACO_OK) return PyLong_FromLong(st);
    return tuple(norm_type, {object(std::optional<Pair>(y)), object(h), object(rstd), object(ck)});
  });
}

// rms_norm_backward(dy, saved, weight, rstd, dh, dx, dw, workspace, stream) -> dx, dw
PyObject* rms_norm_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(v, n, 9, [&]() -> PyObject* {
    const at::Tensor& dy = tensor(v[0], "dy");
    const Matrix m = matrix(dy, "dy");
    const OnStream on(v[8], dy);
    std::optional<Pair> ck;
    taco_fp8_tensor cd{};
    Matrix h, dh;
    if (PyTuple_Check(v[1])) {
      ck = pair_of(v[1], "checkpoint");
      cd = describe(ck->codes, ck->scales, "checkpoint");
    } else {
      h = like(tensor(v[1], "h"), "h", m.rows, m.cols, m.dtype);
    }
    const at::Tensor& weight = tensor(v[2], "weight");
    void* w = vector(weight, "weight", m.cols, false);
    void* rstd = vector(tensor(v[3], "rstd"), "rstd", m.rows, true);
    if (given(v[4])) dh = like(tensor(v[4], "dh"), "dh", m.rows, m.cols, m.dtype);
    const at::Tensor dx =
        given(v[5]) ? tensor(v[5], "dx") : empty_matrix(m.rows, m.cols, dy.scalar_type());
    const Matrix out = like(dx, "dx", m.rows, m.cols, m.dtype);
    const at::Tensor dw = given(v[6]) ? tensor(v[6], "dw") : empty_vector(m.cols, at::kFloat);
    void* dwp = vector(dw, "dw", m.cols, true);
    at::Tensor ws;
    if (given(v[7])) {
      ws = tensor(v[7], "workspace");
      if (!ws.is_cuda() || !ws.is_contiguous()) refuse("workspace must be a contiguous CUDA tensor");
    } else {
      ws = empty_vector(static_cast<int64_t>(taco_rms_norm_workspace_bytes(m.rows, m.cols)), at::kByte);
    }
    void* stream = on.handle();
    const taco_status st = call([&] {
      return taco_rms_norm_fp8_backward(m.p, m.ld, ck ? &cd : nullptr, h.p, h.ld, w, dtype_of(weight.scalar_type()),
                                        static_cast<const float*>(rstd), dh.p, dh.ld, m.dtype, m.rows, m.cols, out.p,
                                        out.ld, static_cast<float*>(dwp), ws.data_ptr(), ws.nbytes(), stream);
    });
    if (st != TACO_OK) return PyLong_FromLong(st);
    return tuple(&PyTuple_Type, {object(dx), object(dw)});
  });
}

// swiglu(gate_up, checkpoint, out, stream) -> y, checkpoint
PyObject* swiglu(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(v, n, 4, [&]() -> PyObject* {
    const at::Tensor& x = tensor(v[0], "gate_up");
    const Matrix m = matrix(x, "gate_up");
    if (m.cols < 2 || m.cols % 2) refuse("gate_up must have an even number of columns");
    const int64_t F = m.cols / 2;
    const bool keep = PyTuple_Check(v[1]) || flag(v[1], "checkpoint");
    const OnStream on(v[3], x);
    const Pair y = given(v[2]) ? pair_of(v[2], "out") : new_fp8({m.rows, F}, 1);
    const taco_fp8_tensor yd = describe(y.codes, y.scales, "out");
    std::optional<Pair> ck;
    if (PyTuple_Check(v[1]))
      ck = pair_of(v[1], "checkpoint");
    else if (keep)
      ck = new_fp8({2, m.rows, F}, 1);
    taco_fp8_tensor g{}, u{};
    if (ck) {
      if (ck->codes.dim() != 3 || ck->codes.size(0) != 2 || ck->scales.dim() != 3 || ck->scales.size(0) != 2)
        refuse("the checkpoint of a gated activation is [2, M, F]: gate, up");
      g = describe(ck->codes, ck->scales, "checkpoint", 1, 3, 0);
      u = describe(ck->codes, ck->scales, "checkpoint", 1, 3, 1);
    }
    const char* p = static_cast<const char*>(m.p);
    void* stream = on.handle();
    const taco_status st = call([&] {
      return taco_swiglu_fp8(p, m.ld, p ? p + F * x.element_size() : p, m.ld, m.dtype, m.rows, F, &yd,
                             ck ? &g : nullptr, ck ? &u : nullptr, stream);
    });
    if (st != TACO_OK) return PyLong_FromLong(st);
    return tuple(&PyTuple_Type, {object(std::optional<Pair>(y)), object(ck)});
  });
}

// swiglu_backward(dy, checkpoint, out, stream) -> d gate_up
PyObject* swiglu_backward(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(v, n, 4, [&]() -> PyObject* {
    const at::Tensor& dy = tensor(v[0], "dy");
    const Matrix m = matrix(dy, "dy");
    const OnStream on(v[3], dy);
    const Pair ck = pair_of(v[1], "checkpoint");
    if (ck.codes.dim() != 3 || ck.codes.size(0) != 2 || ck.scales.dim() != 3 || ck.scales.size(0) != 2)
      refuse("the checkpoint of a gated activation is [2, M, F]: gate, up");
    const taco_fp8_tensor g = describe(ck.codes, ck.scales, "checkpoint", 1, 3, 0);
    const taco_fp8_tensor u = describe(ck.codes, ck.scales, "checkpoint", 1, 3, 1);
    const at::Tensor out =
        given(v[2]) ? tensor(v[2], "out") : empty_matrix(m.rows, 2 * m.cols, dy.scalar_type());
    const Matrix o = like(out, "out", m.rows, 2 * m.cols, m.dtype);
    char* p = static_cast<char*>(o.p);
    void* stream = on.handle();
    const taco_status st = call([&] {
      return taco_swiglu_fp8_backward(m.p, m.ld, &g, &u, m.dtype, m.rows, m.cols, p, o.ld,
                                      p ? p + m.cols * dy.element_size() : p, o.ld, stream);
    });
    if (st != TACO_OK) return PyLong_FromLong(st);
    return object(out);
  });
}

// matmul(a, b, out, out_dtype, add, stream) -> out
PyObject* matmul(PyObject*, PyObject* const* v, Py_ssize_t n) {
  return guarded(v, n, 6, [&]() -> PyObject* {
    const Pair a = pair_of(v[0], "a"), b = pair_of(v[1], "b");
    const taco_fp8_tensor ad = describe(a.codes, a.scales, "a"), bd = describe(b.codes, b.scales, "b");
    const OnStream on(v[5], a.codes);
    at::Tensor out;
    Matrix add;
    if (given(v[2])) {
      out = tensor(v[2], "out");
    } else {
      if (!THPDtype_Check(v[3])) refuse("out_dtype must be a torch.dtype");
      out = empty_matrix(ad.rows, bd.rows, reinterpret_cast<THPDtype*>(v[3])->scalar_type);
    }
    const Matrix o = matrix(out, "out");
    if (o.rows != ad.rows || o.cols != bd.rows) refuse("out must have the rows of a and of b");
    if (given(v[4])) add = like(tensor(v[4], "add"), "add", o.rows, o.cols, o.dtype);
    void* stream = on.handle();
    const taco_status st = call([&] { return taco_matmul_fp8(&ad, &bd, add.p, add.ld, o.p, o.ld, o.dtype, stream); });
    if (st != TACO_OK) return PyLong_FromLong(st);
    return object(out);
  });
}

// types(Fp8Tensor, RmsNormOutput)
PyObject* types(PyObject*, PyObject* const* v, Py_ssize_t n) {
  for (Py_ssize_t i = 0; i < n; ++i)
    if (!PyType_Check(v[i]) || !PyType_IsSubtype(reinterpret_cast<PyTypeObject*>(v[i]), &PyTuple_Type)) n = -1;
  if (n != 2) {
    PyErr_SetString(PyExc_TypeError, "types(Fp8Tensor, RmsNormOutput): two subclasses of tuple");
    return nullptr;
  }
  Py_INCREF(v[0]);
  Py_INCREF(v[1]);
  fp8_type = reinterpret_cast<PyTypeObject*>(v[0]);
  norm_type = reinterpret_cast<PyTypeObject*>(v[1]);
  return none();
}

#define TACO_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {TACO_METHOD(types), TACO_METHOD(quantize), TACO_METHOD(rms_norm),
                          TACO_METHOD(rms_norm_backward),
                          TACO_METHOD(swiglu), TACO_METHOD(swiglu_backward), TACO_METHOD(matmul),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fp8_binding", "Argument marshalling of the FP8 entry points.", -1,
                       kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp8_binding() { return PyModule_Create(&kModule); }
