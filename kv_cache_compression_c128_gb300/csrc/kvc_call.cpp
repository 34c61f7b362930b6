// The operators' calls as functions of the Python interpreter.
//
// kvc_*: the C entry points; numbers, None (a null pointer) and bytes in, the status
// out.  (ctypes takes 1.9 us to convert the 18 arguments of one, as long as the
// launch itself.)
// store, dequantize, rotate, attend: the wrappers' quick forms, for tensors that are
// all as they should be, on the current device and stream, with the results given.
// They return the status, or None for whatever is not plainly right: the forms in
// Python then say what is wrong, or make what is missing.  (Reading the same
// attributes from Python takes 4 us a call.)
// bind() gives the addresses in the loaded libkvc.so.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "../../include/kvc.h"

namespace {

decltype(&kvc_attend_format) attend_entry;
decltype(&kvc_evict_format) evict_entry;
decltype(&kvc_store) store_entry;
decltype(&kvc_dequantize_format) dequantize_entry;
decltype(&kvc_rotate) rotate_entry;

constexpr int64_t kPage8 = 64 * (576 + 8), kPage4 = 64 * (352 + 16), kDim = 512, kRope = 64;

bool count_is(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments, %zd are needed", got, want);
  return false;
}

// A pointer: a number, None or the first of some bytes.
void* pointer(PyObject* x) {
  if (x == Py_None) return nullptr;
  if (PyBytes_Check(x)) return PyBytes_AS_STRING(x);
  return PyLong_AsVoidPtr(x);
}

struct Argument {
  PyObject* x;
  operator int64_t() const { return PyLong_AsLongLong(x); }
  operator int32_t() const { return static_cast<int32_t>(PyLong_AsLongLong(x)); }
  operator uint32_t() const { return static_cast<uint32_t>(PyLong_AsLongLong(x)); }
  operator size_t() const { return static_cast<size_t>(PyLong_AsLongLong(x)); }
  operator float() const { return static_cast<float>(PyFloat_AsDouble(x)); }
  template <typename T>
  operator T*() const { return static_cast<T*>(pointer(x)); }
};

// Calls `entry` with the Python arguments, each as the parameter's type.
template <typename... Params, size_t... I>
PyObject* call_with(kvc_status (*entry)(Params...), PyObject* const* a, std::index_sequence<I...>) {
  std::tuple<Params...> args{static_cast<Params>(Argument{a[I]})...};
  if (PyErr_Occurred()) return nullptr;
  if (entry == nullptr) {
    PyErr_SetString(PyExc_RuntimeError, "not bound");
    return nullptr;
  }
  kvc_status status;
  Py_BEGIN_ALLOW_THREADS
  status = std::apply(entry, args);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

template <typename... Params>
PyObject* call(kvc_status (*entry)(Params...), PyObject* const* a, Py_ssize_t count) {
  if (!count_is(count, sizeof...(Params))) return nullptr;
  return call_with(entry, a, std::index_sequence_for<Params...>{});
}

PyObject* raw_attend(PyObject*, PyObject* const* a, Py_ssize_t n) { return call(attend_entry, a, n); }
PyObject* raw_evict(PyObject*, PyObject* const* a, Py_ssize_t n) { return call(evict_entry, a, n); }
PyObject* raw_store(PyObject*, PyObject* const* a, Py_ssize_t n) { return call(store_entry, a, n); }
PyObject* raw_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) { return call(dequantize_entry, a, n); }
PyObject* raw_rotate(PyObject*, PyObject* const* a, Py_ssize_t n) { return call(rotate_entry, a, n); }

// ---- quick forms -----------------------------------------------------------------

// A tensor on `device` (-1: on any CUDA device, which it sets) of one of the types.
const at::Tensor* tensor(PyObject* x, int* device, c10::ScalarType type, int64_t dims) {
  if (!THPVariable_Check(x)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(x);
  if (!t.is_cuda() || t.scalar_type() != type || t.dim() != dims) return nullptr;
  if (*device < 0) *device = t.get_device();
  return t.get_device() == *device ? &t : nullptr;
}

const at::Tensor* dense(PyObject* x, int* device, c10::ScalarType type, int64_t dims) {
  const at::Tensor* const t = tensor(x, device, type, dims);
  return t != nullptr && t->is_contiguous() ? t : nullptr;
}

template <typename T = void>
T* data(const at::Tensor* t) { return t == nullptr ? nullptr : static_cast<T*>(t->data_ptr()); }

bool is_float(PyObject* x, c10::ScalarType* type) {
  if (!THPVariable_Check(x)) return false;
  *type = THPVariable_Unpack(x).scalar_type();
  return *type == at::kFloat || *type == at::kBFloat16;
}

int32_t code_of(c10::ScalarType type) { return type == at::kBFloat16 ? KVC_DTYPE_BF16 : KVC_DTYPE_F32; }

const at::Tensor* cache(PyObject* x, int* device, int32_t* form) {
  const at::Tensor* const t = dense(x, device, at::kByte, 2);
  if (t == nullptr || (t->size(1) != kPage8 && t->size(1) != kPage4)) return nullptr;
  *form = t->size(1) == kPage8 ? KVC_FORMAT_8BIT : KVC_FORMAT_4BIT;
  return t;
}

struct Rotation {
  const at::Tensor *positions, *table;
  int64_t row_stride, axis_stride;
  int32_t axes;
  const uint8_t* pairs;

  bool read(PyObject* at_, PyObject* table_, PyObject* pairs_, int64_t rows, int* device) {
    if (!THPVariable_Check(at_)) return false;
    const int64_t dims = THPVariable_Unpack(at_).dim();
    positions = tensor(at_, device, at::kLong, dims);
    table = dense(table_, device, at::kFloat, 2);
    if (positions == nullptr || table == nullptr || dims < 1 || dims > 2 || positions->size(0) != rows ||
        table->size(1) != kRope)
      return false;
    row_stride = positions->stride(0);
    axis_stride = dims == 2 ? positions->stride(1) : 0;
    axes = dims == 2 ? static_cast<int32_t>(positions->size(1)) : 1;
    pairs = nullptr;
    if (axes < 1 || axes > 4) return false;
    if (pairs_ == Py_None) return axes == 1;
    if (!PyBytes_CheckExact(pairs_) || PyBytes_GET_SIZE(pairs_) != 32) return false;
    pairs = reinterpret_cast<const uint8_t*>(PyBytes_AS_STRING(pairs_));
    for (int i = 0; i < 32; ++i)
      if (pairs[i] >= axes) return false;
    return true;
  }
};

// The current stream of `device`, if that is the current device.
bool stream_of(int device, void** stream) {
  const auto s = c10::cuda::getCurrentCUDAStream();
  *stream = s.stream();
  return s.device_index() == device;
}

template <typename Entry, typename... Args>
PyObject* finish(Entry entry, Args... args) {
  if (entry == nullptr) Py_RETURN_NONE;
  kvc_status status;
  Py_BEGIN_ALLOW_THREADS
  status = entry(args...);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

// What a quick form does not take, an exception of torch's included, is None.
template <PyObject* (*kForm)(PyObject* const*), int kCount>
PyObject* quick(PyObject*, PyObject* const* a, Py_ssize_t count) {
  if (!count_is(count, kCount)) return nullptr;
  PyObject* got = nullptr;
  try {
    got = kForm(a);
  } catch (...) {
    got = nullptr;
  }
  if (got != nullptr) return got;
  PyErr_Clear();
  Py_RETURN_NONE;
}

// x, kv_cache, slots, positions, cos_sin_cache, axes
PyObject* quick_store(PyObject* const* a) {
  int device = -1;
  int32_t form;
  c10::ScalarType type;
  if (!is_float(a[0], &type)) return nullptr;
  const at::Tensor *x = tensor(a[0], &device, type, 2), *kv = cache(a[1], &device, &form), *slots = dense(a[2], &device, at::kLong, 1);
  if (x == nullptr || kv == nullptr || slots == nullptr) return nullptr;
  const int64_t rows = x->size(0);
  Rotation r = {};
  const bool turns = a[3] != Py_None;
  void* stream;
  if (rows == 0 || x->size(1) != kDim || x->stride(1) != 1 || slots->size(0) != rows ||
      (turns ? !r.read(a[3], a[4], a[5], rows, &device) : a[4] != Py_None || a[5] != Py_None) ||
      !stream_of(device, &stream))
    return nullptr;
  return finish(store_entry, data(x), code_of(type), rows > 1 ? x->stride(0) : 0, rows, data<uint8_t>(kv), form, kv->size(0),
                data<int64_t>(slots), data<int64_t>(r.positions), r.row_stride, r.axis_stride, r.axes, r.pairs,
                data<float>(r.table), turns ? r.table->size(0) : int64_t{0}, stream);
}

// kv_cache, slots, out
PyObject* quick_dequantize(PyObject* const* a) {
  int device = -1;
  int32_t form;
  c10::ScalarType type;
  if (!is_float(a[2], &type)) return nullptr;
  const at::Tensor *kv = cache(a[0], &device, &form), *slots = dense(a[1], &device, at::kLong, 1), *out = dense(a[2], &device, type, 2);
  void* stream;
  if (kv == nullptr || slots == nullptr || out == nullptr || out->size(0) != slots->size(0) || out->size(1) != kDim ||
      !stream_of(device, &stream))
    return nullptr;
  return finish(dequantize_entry, data<uint8_t>(kv), form, kv->size(0), data<int64_t>(slots), slots->size(0), data(out),
                code_of(type), stream);
}

// x, positions, cos_sin_cache, axes, inverse, out
PyObject* quick_rotate(PyObject* const* a) {
  int device = -1;
  c10::ScalarType type;
  if (!is_float(a[0], &type)) return nullptr;
  const int64_t dims = THPVariable_Unpack(a[0]).dim();
  const at::Tensor *x = tensor(a[0], &device, type, dims), *out = tensor(a[5], &device, type, dims);
  if (x == nullptr || out == nullptr || dims < 2 || dims > 3 || x->sizes() != out->sizes() || x->numel() == 0 ||
      x->size(-1) != kRope || x->stride(-1) != 1 || out->stride(-1) != 1)
    return nullptr;
  const int64_t tokens = x->size(0), heads = dims == 3 ? x->size(1) : 1;
  const int inverse = PyObject_IsTrue(a[4]);
  Rotation r = {};
  void* stream;
  if (inverse < 0 || heads > INT32_MAX || !r.read(a[1], a[2], a[3], tokens, &device) || !stream_of(device, &stream)) return nullptr;
  const bool apart = heads > 1;
  return finish(rotate_entry, data(x), code_of(type), tokens > 1 ? x->stride(0) : 0, apart ? x->stride(1) : 0, tokens,
                static_cast<int32_t>(heads), data<int64_t>(r.positions), r.row_stride, r.axis_stride, r.axes, r.pairs,
                data<float>(r.table), r.table->size(0), inverse, data(out), tokens > 1 ? out->stride(0) : 0,
                apart ? out->stride(1) : 0, stream);
}

// q, kv_cache, page_table, lengths, scale, sinks, out, lse, slot_weights, slot_weights_in, flags, workspace
PyObject* quick_attend(PyObject* const* a) {
  int device = -1;
  int32_t form;
  const at::Tensor *kv = cache(a[1], &device, &form), *q = tensor(a[0], &device, at::kBFloat16, 3),
                   *pages = tensor(a[2], &device, at::kInt, 2), *lengths = dense(a[3], &device, at::kInt, 1),
                   *out = dense(a[6], &device, at::kBFloat16, 3), *lse = dense(a[7], &device, at::kFloat, 2),
                   *space = dense(a[11], &device, at::kByte, 1);
  if (kv == nullptr || q == nullptr || pages == nullptr || lengths == nullptr || out == nullptr || lse == nullptr || space == nullptr)
    return nullptr;
  const int64_t reqs = q->size(0), heads = q->size(1);
  if (reqs == 0 || heads < 1 || heads > 128 || q->size(2) != kDim || q->stride(2) != 1 || (heads > 1 && q->stride(1) == 0) ||
      pages->size(0) != reqs || pages->size(1) == 0 || (pages->stride(1) != 1 && pages->size(1) > 1) || lengths->size(0) != reqs ||
      out->sizes() != q->sizes() || lse->size(0) != reqs || lse->size(1) != heads)
    return nullptr;
  const at::Tensor *sinks = nullptr, *weights = nullptr, *weights_in = nullptr;
  if (a[5] != Py_None && ((sinks = dense(a[5], &device, at::kFloat, 1)) == nullptr || sinks->size(0) != heads)) return nullptr;
  int64_t slots = 0;
  if (a[8] != Py_None) {
    weights = tensor(a[8], &device, at::kFloat, 2);
    if (weights == nullptr || weights->size(0) != reqs || weights->size(1) == 0 || (weights->stride(1) != 1 && weights->size(1) > 1))
      return nullptr;
    slots = weights->size(1);
  }
  if (a[9] != Py_None) {
    weights_in = tensor(a[9], &device, at::kFloat, 2);
    if (weights_in == nullptr || weights == nullptr || weights_in->sizes() != weights->sizes() ||
        (weights_in->stride(1) != 1 && slots > 1))
      return nullptr;
  }
  const double scale = a[4] == Py_None ? 0.04419417382415922 : PyFloat_AsDouble(a[4]);  // 512 ** -0.5
  const long flags = PyLong_AsLong(a[10]);
  void* stream;
  if (PyErr_Occurred() || flags < 0 || flags > UINT32_MAX || !stream_of(device, &stream)) return nullptr;
  return finish(attend_entry, data(q), q->stride(0), q->stride(1), reqs, static_cast<int32_t>(heads), data<uint8_t>(kv), form,
                kv->size(0), data<int32_t>(pages), pages->size(1), pages->stride(0), data<int32_t>(lengths),
                static_cast<float>(scale), data<float>(sinks), data(out), data<float>(lse), data<float>(weights_in),
                weights_in == nullptr ? int64_t{0} : weights_in->stride(0), data<float>(weights),
                weights == nullptr ? int64_t{0} : weights->stride(0), slots, data(space), static_cast<size_t>(space->numel()),
                static_cast<uint32_t>(flags), stream);
}

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t count) {
  if (!count_is(count, 5)) return nullptr;
  void* const found[5] = {pointer(a[0]), pointer(a[1]), pointer(a[2]), pointer(a[3]), pointer(a[4])};
  if (PyErr_Occurred()) return nullptr;
  attend_entry = reinterpret_cast<decltype(attend_entry)>(found[0]);
  evict_entry = reinterpret_cast<decltype(evict_entry)>(found[1]);
  store_entry = reinterpret_cast<decltype(store_entry)>(found[2]);
  dequantize_entry = reinterpret_cast<decltype(dequantize_entry)>(found[3]);
  rotate_entry = reinterpret_cast<decltype(rotate_entry)>(found[4]);
  Py_RETURN_NONE;
}

using Function = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyMethodDef method(const char* name, Function f) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method("bind", bind),
    method("kvc_attend_format", raw_attend),
    method("kvc_evict_format", raw_evict),
    method("kvc_store", raw_store),
    method("kvc_dequantize_format", raw_dequantize),
    method("kvc_rotate", raw_rotate),
    method("store", quick<quick_store, 6>),
    method("dequantize", quick<quick_dequantize, 3>),
    method("rotate", quick<quick_rotate, 6>),
    method("attend", quick<quick_attend, 12>),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_kvc_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kvc_call() { return PyModule_Create(&module_def); }
