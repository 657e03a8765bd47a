// The Python faces of the batch verification operators (fp4.py, verify.py,
// pages.py): checks of tensors, outputs' memory and the calls of the C ABI in
// one step.
//
// A call's kernels take 2 to 15 us, and what a face does in Python (30 to 40
// questions to tensors, an allocation, a foreign call) took 5 to 12 us of it
// (a fork, a cut and room: 30 of 44); here these are plain C++.
#include <Python.h>

#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstring>
#include <new>
#include <optional>
#include <string>
#include <utility>
#include <vector>

#include "dflash.h"

namespace {

struct Refusal {  // a ValueError
  std::string what;
};
struct Raised {};  // a Python error is set

void need(bool cond, const char* what) {
  if (!cond) throw Refusal{what};
}

// f() with its C++ exceptions as Python's.
template <typename F>
PyObject* faced(F&& f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refusal& r) {
    PyErr_SetString(PyExc_ValueError, r.what.c_str());
    return nullptr;
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// f() while other Python threads run: outputs' memory and the launches, which may wait for room in the GPU's queue.
// What f reads of Python's objects is read before.
template <typename F>
auto apart(F&& f) {
  struct Released {
    PyThreadState* const state = PyEval_SaveThread();
    ~Released() { PyEval_RestoreThread(state); }
  } released;
  return f();
}
// A new reference until it is taken out.
struct Hold {
  PyObject* o;
  ~Hold() { Py_XDECREF(o); }
  PyObject* take() { return std::exchange(o, nullptr); }
};

// An error of the library, raised by the package's own check.
void check(dflash_status code, const char* what) {
  if (code == DFLASH_OK) return;
  PyObject* lib = PyImport_ImportModule("block_diffusion_speculative_hidden_gb300._lib");
  if (lib != nullptr) {
    PyObject* r = PyObject_CallMethod(lib, "check", "is", static_cast<int>(code), what);
    Py_XDECREF(r);
    Py_DECREF(lib);
    if (r != nullptr) PyErr_SetString(PyExc_RuntimeError, what);
  }
  throw Raised{};
}

bool is_tensor(PyObject* o) { return THPVariable_Check(o); }
const at::Tensor& tensor(PyObject* o, const char* what) {
  need(is_tensor(o), what);
  return THPVariable_Unpack(o);
}
int index_of(const at::Tensor& t) { return t.is_cuda() ? static_cast<int>(t.get_device()) : -1; }
int elem_of(at::ScalarType t) {
  return t == at::kFloat ? DFLASH_ELEM_F32 : t == at::kBFloat16 ? DFLASH_ELEM_BF16 : t == at::kHalf ? DFLASH_ELEM_F16 : -1;
}

// The address of an optional contiguous int32 tensor of n entries.
int32_t* ints(PyObject* o, int64_t n, int dev, const char* what) {
  if (o == Py_None) return nullptr;
  if (is_tensor(o)) {
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() == at::kInt && t.numel() == n && t.is_contiguous() && index_of(t) == dev)
      return static_cast<int32_t*>(t.data_ptr());
  }
  throw Refusal{std::string(what) + ": contiguous int32 of " + std::to_string(n) + " entries on the others' device"};
}

// Device dev is the current one here, and its current stream the call's.
struct On {
  explicit On(int dev) : guard((need(dev >= 0, "tensors must be on a CUDA device"), static_cast<c10::DeviceIndex>(dev))) {
    stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  }
  c10::cuda::CUDAGuard guard;
  dflash_stream stream;
};

at::Tensor room(at::IntArrayRef sizes, at::ScalarType type, at::Device device) {
  return at::empty(sizes, at::TensorOptions().dtype(type).device(device));
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }
PyObject* same(PyObject* o) {
  Py_INCREF(o);
  return o;
}

void arguments(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    throw Raised{};
  }
}

// ------------------------------------------------------------------ 4-bit matrices

struct Matrix {
  PyObject_HEAD
  at::Tensor codes, scales;             // codes alone holds both where scales is not defined
  std::optional<at::Tensor> scale;
  int64_t rows, cols;
  int format, dev;
  const void *codes_at, *scales_at;
  const float* scale_at;
};
PyTypeObject* matrix_type;

int format_of(PyObject* o) {
  if (PyUnicode_Check(o)) {
    if (PyUnicode_CompareWithASCIIString(o, "mx") == 0) return DFLASH_FP4_MX;
    if (PyUnicode_CompareWithASCIIString(o, "nv") == 0) return DFLASH_FP4_NV;
  }
  throw Refusal{"fmt: mx or nv"};
}
// Columns are counted in 32 bits by the library's calls.
void need_cols(int64_t cols) { need(cols <= INT32_MAX, "cols: too many columns"); }
int64_t scale_bytes(int64_t rows, int64_t cols, int format) {
  return (rows + 127) / 128 * ((cols + 255) / 256) * (format == DFLASH_FP4_NV ? 2048 : 1024);
}
std::optional<at::Tensor> scale_of(PyObject* o, int format, int dev) {
  if (o == Py_None) return std::nullopt;
  constexpr const char* kWhat = "scale: fp32 of one entry on the codes' device, with the nv format";
  const at::Tensor& t = tensor(o, kWhat);
  need(format == DFLASH_FP4_NV && t.scalar_type() == at::kFloat && t.numel() == 1 && index_of(t) == dev, kWhat);
  return t;
}
void set_scale(Matrix* m, const std::optional<at::Tensor>& scale) {
  m->scale = scale;
  m->scale_at = scale ? static_cast<const float*>(scale->data_ptr()) : nullptr;
}

Matrix* new_matrix() {
  auto* m = reinterpret_cast<Matrix*>(matrix_type->tp_alloc(matrix_type, 0));
  if (m == nullptr) throw Raised{};
  new (&m->codes) at::Tensor();
  new (&m->scales) at::Tensor();
  new (&m->scale) std::optional<at::Tensor>();
  return m;
}
void free_matrix(PyObject* o) {
  auto* m = reinterpret_cast<Matrix*>(o);
  m->codes.~Tensor();
  m->scales.~Tensor();
  m->scale.~optional();
  PyTypeObject* const type = Py_TYPE(o);
  type->tp_free(o);
  Py_DECREF(type);
}
Matrix* matrix(PyObject* o, const char* what) {
  need(Py_TYPE(o) == matrix_type, what);
  return reinterpret_cast<Matrix*>(o);
}

// matrix(codes, scales, fmt, scale)
PyObject* make_matrix(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return faced([&]() -> PyObject* {
    arguments(n, 4);
    const int format = format_of(a[2]);
    constexpr const char* kCodes = "codes: contiguous uint8 [rows, cols / 2]";
    const at::Tensor& codes = tensor(a[0], kCodes);
    need(codes.dim() == 2 && codes.scalar_type() == at::kByte && codes.is_contiguous(), kCodes);
    const int64_t rows = codes.size(0), cols = 2 * codes.size(1);
    need(cols % 32 == 0, "cols: a multiple of 32");
    need_cols(cols);
    const int dev = index_of(codes);
    constexpr const char* kScales = "scales: contiguous uint8 tiles of all rows, on the codes' device";
    const at::Tensor& scales = tensor(a[1], kScales);
    need(scales.scalar_type() == at::kByte && scales.is_contiguous() && index_of(scales) == dev &&
             scales.numel() == scale_bytes(rows, cols, format),
         kScales);
    const std::optional<at::Tensor> scale = scale_of(a[3], format, dev);
    Matrix* const m = new_matrix();
    m->codes = codes;
    m->scales = scales;
    m->rows = rows;
    m->cols = cols;
    m->format = format;
    m->dev = dev;
    m->codes_at = codes.data_ptr();
    m->scales_at = scales.data_ptr();
    set_scale(m, scale);
    return reinterpret_cast<PyObject*>(m);
  });
}

// A matrix without memory, which take_room then gives it, in one piece.
Matrix* shaped(int64_t rows, int64_t cols, int format, int dev) {
  Matrix* const m = new_matrix();
  m->rows = rows;
  m->cols = cols;
  m->format = format;
  m->dev = dev;
  return m;
}
void take_room(Matrix* m, at::Device device) {
  const int64_t at = (m->rows * m->cols / 2 + 15) / 16 * 16;
  m->codes = room({at + scale_bytes(m->rows, m->cols, m->format)}, at::kByte, device);
  m->codes_at = m->codes.data_ptr();
  m->scales_at = static_cast<const uint8_t*>(m->codes_at) + at;
}
// The views of one piece, when they are first asked for.
void split(Matrix* m) {
  if (m->scales.defined()) return;
  const int64_t bytes = m->rows * m->cols / 2;
  const at::Tensor both = m->codes;
  m->scales = both.narrow(0, (bytes + 15) / 16 * 16, scale_bytes(m->rows, m->cols, m->format));
  m->codes = both.narrow(0, 0, bytes).view({m->rows, m->cols / 2});
}

PyObject* matrix_codes(PyObject* o, void*) {
  return faced([&] {
    auto* m = reinterpret_cast<Matrix*>(o);
    split(m);
    return wrap(m->codes);
  });
}
PyObject* matrix_scales(PyObject* o, void*) {
  return faced([&] {
    auto* m = reinterpret_cast<Matrix*>(o);
    split(m);
    return wrap(m->scales);
  });
}
PyObject* matrix_scale(PyObject* o, void*) {
  return faced([&] {
    auto* m = reinterpret_cast<Matrix*>(o);
    return m->scale ? wrap(*m->scale) : same(Py_None);
  });
}
PyObject* matrix_rows(PyObject* o, void*) { return PyLong_FromLongLong(reinterpret_cast<Matrix*>(o)->rows); }
PyObject* matrix_cols(PyObject* o, void*) { return PyLong_FromLongLong(reinterpret_cast<Matrix*>(o)->cols); }
PyObject* matrix_dev(PyObject* o, void*) { return PyLong_FromLong(reinterpret_cast<Matrix*>(o)->dev); }
PyObject* matrix_fmt(PyObject* o, void*) {
  return PyUnicode_FromString(reinterpret_cast<Matrix*>(o)->format == DFLASH_FP4_NV ? "nv" : "mx");
}
PyObject* matrix_at(PyObject* o, void*) {
  auto* m = reinterpret_cast<Matrix*>(o);
  const auto n = [](const void* p) { return static_cast<unsigned long long>(reinterpret_cast<uintptr_t>(p)); };
  if (m->scale_at == nullptr) return Py_BuildValue("KKO", n(m->codes_at), n(m->scales_at), Py_None);
  return Py_BuildValue("KKK", n(m->codes_at), n(m->scales_at), n(m->scale_at));
}
PyGetSetDef matrix_members[] = {{"codes", matrix_codes, nullptr, nullptr, nullptr},
                                {"scales", matrix_scales, nullptr, nullptr, nullptr},
                                {"scale", matrix_scale, nullptr, nullptr, nullptr},
                                {"rows", matrix_rows, nullptr, nullptr, nullptr},
                                {"cols", matrix_cols, nullptr, nullptr, nullptr},
                                {"dev", matrix_dev, nullptr, nullptr, nullptr},
                                {"fmt", matrix_fmt, nullptr, nullptr, nullptr},
                                {"at", matrix_at, nullptr, nullptr, nullptr},
                                {nullptr, nullptr, nullptr, nullptr, nullptr}};

// matrix_room(rows, cols, fmt, scale, like): on the device of `like`
PyObject* make_matrix_room(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return faced([&]() -> PyObject* {
    arguments(n, 5);
    const int64_t rows = PyLong_AsLongLong(a[0]), cols = PyLong_AsLongLong(a[1]);
    if (PyErr_Occurred() != nullptr) throw Raised{};
    const int format = format_of(a[2]);
    const at::Tensor& like = tensor(a[4], "like: a tensor");
    need(rows > 0 && cols > 0 && cols % 32 == 0, "at least one row, cols a multiple of 32");
    need_cols(cols);
    const std::optional<at::Tensor> scale = scale_of(a[3], format, index_of(like));
    Matrix* const m = shaped(rows, cols, format, index_of(like));
    Hold hold{reinterpret_cast<PyObject*>(m)};
    const at::Device device = like.device();
    apart([&] { take_room(m, device); });
    set_scale(m, scale);
    return hold.take();
  });
}

// quantize(x, fmt, scale, out): the matrix
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return faced([&]() -> PyObject* {
    arguments(n, 4);
    constexpr const char* kX = "x: fp32, bf16 or fp16 [rows, cols]";
    const at::Tensor& x = tensor(a[0], kX);
    const On on(index_of(x));
    const int elem = elem_of(x.scalar_type()), format = format_of(a[1]);
    need(elem >= 0 && x.dim() == 2, kX);
    const int64_t rows = x.size(0), cols = x.size(1);
    need(rows > 0 && cols > 0 && cols % 32 == 0, "x: at least one row, cols a multiple of 32");
    need(x.stride(1) == 1, "x: the entries of a row must be contiguous");
    need_cols(cols);
    const std::optional<at::Tensor> scale = scale_of(a[2], format, index_of(x));
    const bool fresh = a[3] == Py_None;
    Matrix* m;
    if (fresh) {
      m = shaped(rows, cols, format, index_of(x));
    } else {
      constexpr const char* kOut = "out: the shape of x, fmt, its device";
      m = matrix(a[3], kOut);
      need(m->rows == rows && m->cols == cols && m->format == format && m->dev == index_of(x), kOut);
      Py_INCREF(m);
    }
    Hold hold{reinterpret_cast<PyObject*>(m)};
    const float* const scale_at = scale ? static_cast<const float*>(scale->data_ptr()) : nullptr;
    const void* const x_at = x.data_ptr();
    const int64_t ld = rows > 1 ? x.stride(0) : cols;
    const at::Device device = x.device();
    check(apart([&] {
            if (fresh) take_room(m, device);
            return dflash_quantize_fp4(x_at, elem, ld, rows, static_cast<int>(cols), format, scale_at,
                                       const_cast<void*>(m->codes_at), const_cast<void*>(m->scales_at), on.stream);
          }),
          "dflash_quantize_fp4");
    set_scale(m, scale);  // (of the codes that m holds now)
    return hold.take();
  });
}

// A contiguous output [rows, cols]: the caller's, or one to be taken on the matrix's device.
struct RowsOut {
  RowsOut(PyObject* out, PyObject* dtype, int64_t rows, int64_t cols, const Matrix* m, const char* what)
      : rows(rows), cols(cols), device(m->codes.device()) {
    if (out == Py_None) {
      need(THPDtype_Check(dtype) && elem_of(reinterpret_cast<THPDtype*>(dtype)->scalar_type) >= 0,
           "dtype: fp32, bf16 or fp16");
      type = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
      return;
    }
    t = tensor(out, what);
    need(t.dim() == 2 && t.size(0) == rows && t.size(1) == cols && elem_of(t.scalar_type()) >= 0 && t.is_contiguous() &&
             index_of(t) == m->dev,
         what);
    type = t.scalar_type();
  }
  void* take() {
    if (!t.defined()) t = room({rows, cols}, type, device);
    return t.data_ptr();
  }
  int64_t rows, cols;
  at::Device device;
  at::ScalarType type;
  at::Tensor t;
};

// dequantize(t, dtype, out)
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return faced([&]() -> PyObject* {
    arguments(n, 3);
    const Matrix* m = matrix(a[0], "t: a matrix of 4-bit floats");
    const On on(m->dev);
    RowsOut out(a[2], a[1], m->rows, m->cols, m, "out: contiguous fp32, bf16 or fp16 [rows, cols] on the codes' device");
    const float* const scale = m->scale_at;
    check(apart([&] {
            return dflash_dequantize_fp4(m->codes_at, m->scales_at, m->format, scale, m->rows, static_cast<int>(m->cols),
                                         out.take(), elem_of(out.type), on.stream);
          }),
          "dflash_dequantize_fp4");
    return a[2] == Py_None ? wrap(out.t) : same(a[2]);
  });
}

// gemm(W, X, dtype, out, status)
PyObject* gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return faced([&]() -> PyObject* {
    arguments(n, 5);
    const Matrix *w = matrix(a[0], "W: a matrix of 4-bit floats"), *x = matrix(a[1], "X: a matrix of 4-bit floats");
    const On on(w->dev);
    need(x->cols == w->cols && x->format == w->format && x->dev == w->dev, "X: the columns, format and device of W");
    need(x->rows <= INT32_MAX && w->rows <= INT32_MAX, "too many rows");
    RowsOut out(a[3], a[2], x->rows, w->rows, w,
                "out: contiguous fp32, bf16 or fp16 [rows of X, rows of W] on the device of W");
    int* const status = ints(a[4], 1, w->dev, "status");
    const float *const w_scale = w->scale_at, *const x_scale = x->scale_at;
    check(apart([&] {
            return dflash_gemm_fp4(w->codes_at, w->scales_at, w_scale, static_cast<int>(w->rows), x->codes_at, x->scales_at,
                                   x_scale, static_cast<int>(x->rows), static_cast<int>(w->cols), w->format, out.take(),
                                   elem_of(out.type), status, on.stream);
          }),
          "dflash_gemm_fp4");
    return a[3] == Py_None ? wrap(out.t) : same(a[3]);
  });
}

// ------------------------------------------------------------------ verification

// Elements between rows of [B, rows, V] with contiguous, evenly spaced rows.
int64_t row_stride(const at::Tensor& t, const char* what) {
  const int64_t B = t.size(0), rows = t.size(1), V = t.size(2), sb = t.stride(0), st = t.stride(1);
  if (t.stride(2) != 1 && V != 1) throw Refusal{std::string(what) + ": the entries of a row must be contiguous"};
  if (rows == 1) return B > 1 ? sb : V;
  if (B != 1 && sb != rows * st) throw Refusal{std::string(what) + ": rows must be evenly spaced"};
  return st;
}

// verify(tokens, target, u_accept, u_sample, draft, n_draft, out, n_out, status): (out, n_out)
PyObject* verify(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return faced([&]() -> PyObject* {
    arguments(n, 9);
    constexpr const char* kTarget = "target: fp32, bf16 or fp16 [B, K + 1, V]";
    const at::Tensor& target = tensor(a[1], kTarget);
    const int dev = index_of(target);
    const On on(dev);
    const int te = elem_of(target.scalar_type());
    need(target.dim() == 3 && te >= 0, kTarget);
    const int64_t B = target.size(0), K = target.size(1) - 1, V = target.size(2);
    need(B > 0 && K > 0 && V > 0, "target: at least one sequence, two rows and one entry");
    need(B <= INT32_MAX && K <= INT32_MAX && V <= INT32_MAX, "target: too large");
    const auto plain = [&](PyObject* o, at::ScalarType type, bool block, const char* what) -> void* {
      const at::Tensor& t = tensor(o, what);
      need(t.dim() == (block ? 2 : 1) && t.size(0) == B && (!block || t.size(1) == K) && t.scalar_type() == type &&
               t.is_contiguous() && index_of(t) == dev,
           what);
      return t.data_ptr();
    };
    const auto* tokens =
        static_cast<const int32_t*>(plain(a[0], at::kInt, true, "tokens: contiguous int32 [B, K] on the target's device"));
    const auto* ua =
        static_cast<const float*>(plain(a[2], at::kFloat, true, "u_accept: contiguous fp32 [B, K] on the target's device"));
    const auto* us =
        static_cast<const float*>(plain(a[3], at::kFloat, false, "u_sample: contiguous fp32 [B] on the target's device"));
    const void* draft = nullptr;
    int de = 0;
    int64_t ld_d = 0;
    if (a[4] != Py_None) {
      constexpr const char* kDraft = "draft: fp32, bf16 or fp16 [B, K, V] on the target's device";
      const at::Tensor& d = tensor(a[4], kDraft);
      de = elem_of(d.scalar_type());
      need(d.dim() == 3 && d.size(0) == B && d.size(1) == K && d.size(2) == V && de >= 0 && index_of(d) == dev, kDraft);
      draft = d.data_ptr();
      ld_d = row_stride(d, "draft");
    }
    const int64_t ld_t = row_stride(target, "target");
    const int32_t* n_draft = ints(a[5], B, dev, "n_draft");
    int32_t *out_at = ints(a[6], B * (K + 1), dev, "out"), *n_at = ints(a[7], B, dev, "n_out");
    int32_t* status = ints(a[8], 1, dev, "status");
    const void* const target_at = target.data_ptr();
    const at::Device device = target.device();
    at::Tensor out, count;
    check(apart([&] {
            if (out_at == nullptr) {
              out = room({B, K + 1}, at::kInt, device);
              out_at = static_cast<int32_t*>(out.data_ptr());
            }
            if (n_at == nullptr) {
              count = room({B}, at::kInt, device);
              n_at = static_cast<int32_t*>(count.data_ptr());
            }
            return dflash_verify_tokens(tokens, n_draft, target_at, te, ld_t, draft, de, ld_d, ua, us,
                                        static_cast<int>(B), static_cast<int>(K), static_cast<int>(V), out_at, n_at, status,
                                        on.stream);
          }),
          "dflash_verify_tokens");
    PyObject* r = PyTuple_New(2);
    if (r == nullptr) throw Raised{};
    PyTuple_SET_ITEM(r, 0, out.defined() ? wrap(out) : same(a[6]));
    PyTuple_SET_ITEM(r, 1, count.defined() ? wrap(count) : same(a[7]));
    return r;
  });
}

// ------------------------------------------------------------------ pages

struct Pool {
  PyObject_HEAD
  PyObject* tensors[5];  // k, v (a tensor or a tuple of tensors each), page_table, seq_len, refs
  std::vector<void*> layers;
  dflash_page_pool pool;
  int dev;
  size_t workspace;
};
PyTypeObject* pool_type;

void free_pool(PyObject* o) {
  auto* p = reinterpret_cast<Pool*>(o);
  for (PyObject* t : p->tensors) Py_XDECREF(t);
  p->layers.~vector();
  PyTypeObject* const type = Py_TYPE(o);
  type->tp_free(o);
  Py_DECREF(type);
}

// The layers' addresses behind those in `at`: of one tensor [n_layers, n_pages, ...] or a tuple, each contiguous, of the
// given shape, type and device.
void add_layers(PyObject* o, at::IntArrayRef shape, at::ScalarType type, int dev, std::vector<void*>& at) {
  if (is_tensor(o)) {
    const at::Tensor& t = THPVariable_Unpack(o);
    need(t.dim() == 5 && t.sizes().slice(1) == shape && t.scalar_type() == type && index_of(t) == dev && t.size(0) >= 1,
         "k, v: layers of [n_pages, n_kv_heads, 16, head_dim], all alike");
    int64_t step = 1;  // (strides of dimensions of one entry say nothing)
    for (int64_t d = 4; d >= 1; step *= t.size(d), --d)
      need(t.stride(d) == step || t.size(d) == 1 || t.numel() == 0, "k, v: each layer must be contiguous");
    for (int64_t i = 0; i < t.size(0); ++i)
      at.push_back(static_cast<uint8_t*>(t.data_ptr()) + i * t.stride(0) * static_cast<int64_t>(t.element_size()));
    return;
  }
  constexpr const char* kWhat = "k, v: contiguous layers of [n_pages, n_kv_heads, 16, head_dim], all alike";
  for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(o); ++i) {
    const at::Tensor& t = tensor(PyTuple_GET_ITEM(o, i), kWhat);
    need(t.sizes() == shape && t.scalar_type() == type && index_of(t) == dev && t.is_contiguous(), kWhat);
    at.push_back(t.data_ptr());
  }
}

// pool(k, v, page_table, seq_len, refs)
PyObject* make_pool(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return faced([&]() -> PyObject* {
    arguments(n, 5);
    auto* p = reinterpret_cast<Pool*>(pool_type->tp_alloc(pool_type, 0));
    if (p == nullptr) throw Raised{};
    new (&p->layers) std::vector<void*>();
    Hold hold{reinterpret_cast<PyObject*>(p)};
    for (int i = 0; i < 5; ++i) {
      p->tensors[i] = i < 2 && !is_tensor(a[i]) ? PySequence_Tuple(a[i]) : same(a[i]);
      if (p->tensors[i] == nullptr) throw Raised{};
    }
    PyObject *k = p->tensors[0], *v = p->tensors[1];
    need(is_tensor(k) || PyTuple_GET_SIZE(k) > 0, "k, v: at least one layer");
    constexpr const char* kLayers = "k, v: layers of fp32, bf16 or fp16 [n_pages, n_kv_heads, 16, head_dim]";
    const at::Tensor& first = tensor(is_tensor(k) ? k : PyTuple_GET_ITEM(k, 0), kLayers);
    need(first.dim() == (is_tensor(k) ? 5 : 4), kLayers);
    const at::IntArrayRef shape = first.sizes().slice(is_tensor(k) ? 1 : 0);
    const int elem = elem_of(first.scalar_type()), dev = index_of(first);
    need(shape[2] == 16 && elem >= 0, kLayers);
    p->layers.reserve(16);
    add_layers(k, shape, first.scalar_type(), dev, p->layers);
    const size_t layers = p->layers.size();
    add_layers(v, shape, first.scalar_type(), dev, p->layers);
    need(p->layers.size() == 2 * layers, "k, v: the same number of layers");
    constexpr const char* kTable = "page_table: contiguous int32 [n_seqs, max_pages] on the pages' device";
    const at::Tensor& table = tensor(a[2], kTable);
    need(table.dim() == 2 && table.scalar_type() == at::kInt && table.is_contiguous() && index_of(table) == dev, kTable);
    const int64_t sizes[] = {static_cast<int64_t>(layers), shape[0], table.size(0), table.size(1), shape[1], shape[3]};
    for (const int64_t s : sizes) need(s <= INT32_MAX, "the pool is too large");
    dflash_page_pool& q = p->pool;
    memset(&q, 0, sizeof(q));
    q.k = p->layers.data();
    q.v = p->layers.data() + layers;
    q.page_table = static_cast<int32_t*>(table.data_ptr());
    q.seq_len = ints(a[3], sizes[2], dev, "seq_len");
    q.refs = ints(a[4], sizes[1], dev, "refs");
    q.n_layers = static_cast<int>(sizes[0]);
    q.n_pages = static_cast<int>(sizes[1]);
    q.n_seqs = static_cast<int>(sizes[2]);
    q.max_pages = static_cast<int>(sizes[3]);
    q.n_kv_heads = static_cast<int>(sizes[4]);
    q.head_dim = static_cast<int>(sizes[5]);
    q.elem = static_cast<decltype(q.elem)>(elem);
    p->dev = dev;
    p->workspace = 4 * (64 + 3 * static_cast<size_t>(sizes[1]) + 2 * static_cast<size_t>(sizes[2]));
    return hold.take();
  });
}

Pool* pool_of(PyObject* o) {
  need(Py_TYPE(o) == pool_type, "pool: a page pool");
  return reinterpret_cast<Pool*>(o);
}
template <int I>
PyObject* pool_tensor(PyObject* o, void*) {
  return same(reinterpret_cast<Pool*>(o)->tensors[I]);
}
PyObject* pool_dev(PyObject* o, void*) { return PyLong_FromLong(reinterpret_cast<Pool*>(o)->dev); }
PyObject* pool_n_seqs(PyObject* o, void*) { return PyLong_FromLong(reinterpret_cast<Pool*>(o)->pool.n_seqs); }
PyObject* pool_ws(PyObject* o, void*) { return PyLong_FromSize_t(reinterpret_cast<Pool*>(o)->workspace); }
PyObject* pool_ref(PyObject* o, void*) {
  const auto* p = reinterpret_cast<Pool*>(o);
  return PyBytes_FromStringAndSize(reinterpret_cast<const char*>(&p->pool), sizeof(p->pool));
}
PyGetSetDef pool_members[] = {{"k", pool_tensor<0>, nullptr, nullptr, nullptr},
                              {"v", pool_tensor<1>, nullptr, nullptr, nullptr},
                              {"page_table", pool_tensor<2>, nullptr, nullptr, nullptr},
                              {"seq_len", pool_tensor<3>, nullptr, nullptr, nullptr},
                              {"refs", pool_tensor<4>, nullptr, nullptr, nullptr},
                              {"dev", pool_dev, nullptr, nullptr, nullptr},
                              {"n_seqs", pool_n_seqs, nullptr, nullptr, nullptr},
                              {"ws_bytes", pool_ws, nullptr, nullptr, nullptr},
                              {"ref", pool_ref, nullptr, nullptr, nullptr},
                              {nullptr, nullptr, nullptr, nullptr, nullptr}};

// The caller's workspace, or one that is taken and lives as long as this.
struct Space {
  Space(const Pool* p, PyObject* o) : dev(p->dev), bytes(p->workspace) {
    if (o == Py_None) return;
    constexpr const char* kWhat = "workspace: contiguous, the pool's device";
    const at::Tensor& t = tensor(o, kWhat);
    need(index_of(t) == p->dev && t.is_contiguous(), kWhat);
    at = t.data_ptr();
    bytes = t.nbytes();
    given = true;
  }
  void* take() {
    if (!given) {
      own = room({static_cast<int64_t>(bytes)}, at::kByte, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)));
      at = own.data_ptr();
    }
    return at;
  }
  int dev;
  size_t bytes;
  bool given = false;
  at::Tensor own;
  void* at = nullptr;
};
int count_of(int64_t n) {
  need(n <= INT32_MAX, "too many entries");
  return static_cast<int>(n);
}
int64_t entries(PyObject* o, const char* what) { return tensor(o, what).numel(); }
template <typename F>
PyObject* done(const char* what, F&& f) {
  check(apart(f), what);
  Py_RETURN_NONE;
}

// fork(pool, src, dst, workspace, status)
PyObject* fork_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return faced([&]() -> PyObject* {
    arguments(n, 5);
    Pool* const p = pool_of(a[0]);
    const On on(p->dev);
    const int64_t B = entries(a[1], "src: contiguous int32");
    const int32_t *src = ints(a[1], B, p->dev, "src"), *dst = ints(a[2], B, p->dev, "dst");
    int* status = ints(a[4], 1, p->dev, "status");
    Space ws(p, a[3]);
    return done("dflash_pages_fork", [&] {
      return dflash_pages_fork(&p->pool, src, dst, count_of(B), ws.take(), ws.bytes, status, on.stream);
    });
  });
}

// truncate(pool, new_len, seq, status)
PyObject* truncate_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return faced([&]() -> PyObject* {
    arguments(n, 4);
    Pool* const p = pool_of(a[0]);
    const On on(p->dev);
    const int64_t B = a[2] != Py_None   ? entries(a[2], "seq: contiguous int32")
                      : a[1] != Py_None ? entries(a[1], "new_len: contiguous int32")
                                        : p->pool.n_seqs;
    const int32_t *seq = ints(a[2], B, p->dev, "seq"), *len = ints(a[1], B, p->dev, "new_len");
    int* status = ints(a[3], 1, p->dev, "status");
    return done("dflash_pages_truncate",
                [&] { return dflash_pages_truncate(&p->pool, seq, len, count_of(B), status, on.stream); });
  });
}

// reserve(pool, n_rows, seq, workspace, status)
PyObject* reserve_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return faced([&]() -> PyObject* {
    arguments(n, 5);
    Pool* const p = pool_of(a[0]);
    const On on(p->dev);
    const int64_t B = entries(a[1], "n_rows: contiguous int32");
    const int32_t *seq = ints(a[2], B, p->dev, "seq"), *rows = ints(a[1], B, p->dev, "n_rows");
    int* status = ints(a[4], 1, p->dev, "status");
    Space ws(p, a[3]);
    return done("dflash_pages_reserve", [&] {
      return dflash_pages_reserve(&p->pool, seq, rows, count_of(B), ws.take(), ws.bytes, status, on.stream);
    });
  });
}

// compact(pool, table_out, refs_out, page_map, n_used, workspace, status)
PyObject* compact_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return faced([&]() -> PyObject* {
    arguments(n, 7);
    Pool* const p = pool_of(a[0]);
    const On on(p->dev);
    const dflash_page_pool& q = p->pool;
    int32_t *table = ints(a[1], static_cast<int64_t>(q.n_seqs) * q.max_pages, p->dev, "table_out"),
            *refs = ints(a[2], q.n_pages, p->dev, "refs_out"), *map = ints(a[3], q.n_pages, p->dev, "page_map"),
            *used = ints(a[4], 1, p->dev, "n_used");
    int* status = ints(a[6], 1, p->dev, "status");
    Space ws(p, a[5]);
    return done("dflash_pages_compact",
                [&] { return dflash_pages_compact(&q, table, refs, map, used, ws.take(), ws.bytes, status, on.stream); });
  });
}

// copy(to, src, dst, from, status)
PyObject* copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return faced([&]() -> PyObject* {
    arguments(n, 5);
    Pool *const to = pool_of(a[0]), *const from = a[3] == Py_None ? to : pool_of(a[3]);
    const On on(to->dev);
    need(from->dev == to->dev, "both pools on one device");
    const int64_t B = entries(a[1], "src: contiguous int32");
    const int32_t *dst = ints(a[2], B, to->dev, "dst"), *src = ints(a[1], B, to->dev, "src");
    int* status = ints(a[4], 1, to->dev, "status");
    return done("dflash_pages_copy",
                [&] { return dflash_pages_copy(&to->pool, &from->pool, dst, src, count_of(B), status, on.stream); });
  });
}

// ------------------------------------------------------------------ the module

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyCFunction entry() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(F));
}
PyMethodDef methods[] = {{"matrix", entry<make_matrix>(), METH_FASTCALL, nullptr},
                         {"matrix_room", entry<make_matrix_room>(), METH_FASTCALL, nullptr},
                         {"quantize", entry<quantize>(), METH_FASTCALL, nullptr},
                         {"dequantize", entry<dequantize>(), METH_FASTCALL, nullptr},
                         {"gemm", entry<gemm>(), METH_FASTCALL, nullptr},
                         {"verify", entry<verify>(), METH_FASTCALL, nullptr},
                         {"pool", entry<make_pool>(), METH_FASTCALL, nullptr},
                         {"fork", entry<fork_pages>(), METH_FASTCALL, nullptr},
                         {"truncate", entry<truncate_pages>(), METH_FASTCALL, nullptr},
                         {"reserve", entry<reserve_pages>(), METH_FASTCALL, nullptr},
                         {"compact", entry<compact_pages>(), METH_FASTCALL, nullptr},
                         {"copy", entry<copy_pages>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyTypeObject* make_type(const char* name, int size, destructor dealloc, PyGetSetDef* members) {
  PyType_Slot slots[] = {{Py_tp_dealloc, reinterpret_cast<void*>(dealloc)}, {Py_tp_getset, members}, {0, nullptr}};
  PyType_Spec spec{name, size, 0, Py_TPFLAGS_DEFAULT | Py_TPFLAGS_DISALLOW_INSTANTIATION, slots};
  return reinterpret_cast<PyTypeObject*>(PyType_FromSpec(&spec));
}
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_faces", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__faces() {
  matrix_type = make_type("_faces.Matrix", sizeof(Matrix), free_matrix, matrix_members);
  pool_type = matrix_type != nullptr ? make_type("_faces.Pool", sizeof(Pool), free_pool, pool_members) : nullptr;
  return pool_type != nullptr ? PyModule_Create(&module_def) : nullptr;
}
