// Binding of the paged-cache calls for torch tensors: checks of arguments, marshalling, new outputs.
//
// A model makes these calls once per layer and step; through ctypes their checks cost three times what the launch
// does (16 us a call for 7), so this part of the binding is compiled.  Each function returns its output,
// or the library's status as an int where that is not CLO_OK; wrong arguments raise ValueError.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>

#include "clo.h"

namespace {

struct Raised {};  // a Python error is set

// Other Python threads run while this one allocates or launches: both can wait (for the driver, for room in the launch queue).
struct WithoutGil {
  PyThreadState* state = PyEval_SaveThread();
  WithoutGil() = default;
  WithoutGil(const WithoutGil&) = delete;
  ~WithoutGil() { PyEval_RestoreThread(state); }
};
template <typename F>
auto without_gil(F&& f) {
  WithoutGil released;
  return f();
}

[[noreturn]] void refuse(const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  PyErr_FormatV(PyExc_ValueError, fmt, ap);
  va_end(ap);
  throw Raised{};
}

const at::Tensor& cuda_tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda()) refuse("%s must be a CUDA tensor", name);
  return THPVariable_Unpack(o);
}

// The current device, after checking that the tensor is on it.
int device_of(const at::Tensor& t, const char* name) {
  const int dev = c10::cuda::current_device();
  if (t.get_device() != dev) refuse("%s is on cuda:%d, not on the current device", name, (int)t.get_device());
  return dev;
}

const at::Tensor& tensor_on(PyObject* o, const char* name, int dev, at::ScalarType type) {
  const at::Tensor& t = cuda_tensor(o, name);
  if (t.get_device() != dev) refuse("%s is on cuda:%d, not on the current device", name, (int)t.get_device());
  if (t.scalar_type() != type) refuse("%s has dtype %s; expected %s", name, c10::toString(t.scalar_type()), c10::toString(type));
  return t;
}

// A bf16 [n_tokens][n_heads][head_dim] tensor, any strides but the last.  None of the calls is recorded by autograd: a tensor whose
// gradient would get lost in one is refused.
clo_rows rows_of(const at::Tensor& t) { return clo_rows{t.data_ptr(), t.stride(0), t.stride(1)}; }

const at::Tensor& rows(PyObject* o, const char* name, int dev, clo_rows* r) {
  const at::Tensor& t = tensor_on(o, name, dev, at::kBFloat16);
  if (t.requires_grad() && c10::GradMode::is_enabled())
    refuse("%s requires a gradient, which the call does not record: detach it, or call under torch.no_grad()", name);
  if (t.dim() != 3) refuse("%s must have the shape [n_tokens][n_heads][head_dim]", name);
  if (t.stride(2) != 1 && t.size(2) > 1) refuse("%s must be contiguous along head_dim", name);
  *r = rows_of(t);
  return t;
}

void shape_is(const at::Tensor& t, const char* name, int64_t a, int64_t b, int64_t c) {
  if (t.size(0) != a || t.size(1) != b || t.size(2) != c)
    refuse("%s has shape (%lld, %lld, %lld); expected (%lld, %lld, %lld)", name, (long long)t.size(0), (long long)t.size(1), (long long)t.size(2),
           (long long)a, (long long)b, (long long)c);
}

template <typename T>
T* address(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw Raised{};
  return static_cast<T*>(p);
}

// None: torch's current stream; an integer: a handle; else an object with one.
void* stream_of(PyObject* o, int dev) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(dev).stream();
  if (PyLong_Check(o)) return address<void>(o);
  PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
  if (!h) throw Raised{};
  void* p = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (!p && PyErr_Occurred()) throw Raised{};
  return p;
}

// New memory for work on the caller's stream.  A stream that the caller names has its own, as under torch.cuda.stream: what the current
// stream has freed may still be in use there, and the named stream does not wait for it.  `returned`: the caller gets the memory and may
// go on to use it on the current stream, so the allocator is told of that one too.
at::Tensor new_tensor(at::IntArrayRef size, at::ScalarType type, int dev, PyObject* stream, bool returned) {
  const c10::Device device(c10::kCUDA, dev);
  if (stream == Py_None) return without_gil([&] { return at::detail::empty_cuda(size, type, device, std::nullopt); });
  cudaStream_t st = static_cast<cudaStream_t>(stream_of(stream, dev));
  if (st == cudaStreamLegacy) st = nullptr;  // the same stream by its other name
  WithoutGil released;
  const c10::cuda::CUDAStream current = c10::cuda::getCurrentCUDAStream(dev);
  const c10::cuda::CUDAStreamGuard guard(st ? c10::cuda::getStreamFromExternal(st, dev) : c10::cuda::getDefaultCUDAStream(dev));
  at::Tensor t = at::detail::empty_cuda(size, type, device, std::nullopt);
  if (returned && current.stream() != st) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), current);
  return t;
}

// The caller's output, or new rows for None.
at::Tensor output(PyObject* o, const char* name, int dev, int64_t a, int64_t b, int64_t c, clo_rows* r, PyObject* stream) {
  if (o == Py_None) {
    at::Tensor t = new_tensor({a, b, c}, at::kBFloat16, dev, stream, true);
    *r = clo_rows{t.data_ptr(), b * c, c};
    return t;
  }
  const at::Tensor& t = rows(o, name, dev, r);
  shape_is(t, name, a, b, c);
  for (int i = 0; i < 3; ++i)
    if (t.stride(i) == 0 && t.size(i) > 1) refuse("%s is written and must not be an expanded tensor", name);
  return t;
}

// Tells autograd that a tensor of the caller's was written, as torch's own in-place operations do (None: there is no such tensor).
void written(PyObject* o) {
  if (o == Py_None) return;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

template <typename T>
const T* vector_of(PyObject* o, const char* name, int dev, at::ScalarType type, int64_t n) {
  const at::Tensor& t = tensor_on(o, name, dev, type);
  if (t.numel() != n || !t.is_contiguous()) refuse("%s holds %lld elements; expected a contiguous vector of %lld", name, (long long)t.numel(), (long long)n);
  return static_cast<const T*>(t.data_ptr());
}

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse("%s must be an integer", name);
  }
  return v;
}
int32_t small(PyObject* o, const char* name) {
  const int64_t v = integer(o, name);
  if (v < INT32_MIN || v > INT32_MAX) refuse("%s is out of range", name);
  return (int32_t)v;
}

clo_paged_batch batch_of(PyObject* q_starts, PyObject* kv_lens, PyObject* table, int64_t total, PyObject* max_q, int dev, int cache_dev) {
  if (dev != cache_dev) refuse("the cache is on device %d, the call's rows on %d", cache_dev, dev);
  const at::Tensor& t = tensor_on(table, "block_table", dev, at::kInt);
  if (t.dim() != 2) refuse("block_table must have the shape [batch][max_pages]");
  if (t.stride(1) != 1 && t.size(1) > 1) refuse("block_table must have contiguous rows");
  if (total > INT32_MAX || t.size(0) > INT32_MAX - 1 || t.size(1) > INT32_MAX) refuse("the batch is too large");
  clo_paged_batch b;
  b.q_starts = vector_of<int32_t>(q_starts, "q_starts", dev, at::kInt, t.size(0) + 1);
  b.kv_lens = vector_of<int32_t>(kv_lens, "kv_lens", dev, at::kInt, t.size(0));
  b.block_table = static_cast<const int32_t*>(t.data_ptr());
  b.table_stride = t.stride(0);
  b.max_pages = (int32_t)t.size(1);
  b.batch = (int32_t)t.size(0);
  b.total_q = (int32_t)total;
  b.max_q = max_q == Py_None ? (int32_t)total : small(max_q, "max_q");
  return b;
}

// Runs a call's body; C++ exceptions become Python's.
template <typename F>
PyObject* guarded(Py_ssize_t have, Py_ssize_t want, F&& body) {
  if (have != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, have);
    return nullptr;
  }
  try {
    return body();
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// plan, x, positions, out, transpose, stream
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    const at::Tensor& first = cuda_tensor(a[1], "x");
    const int dev = device_of(first, "x");
    clo_rows x, y;
    const at::Tensor& t = rows(a[1], "x", dev, &x);
    const int64_t tokens = t.size(0), heads = t.size(1), d = t.size(2);
    if (heads > INT32_MAX || d > INT32_MAX) refuse("x is too large");
    const int64_t* pos = vector_of<int64_t>(a[2], "positions", dev, at::kLong, tokens);
    at::Tensor out = output(a[3], "out", dev, tokens, heads, d, &y, a[5]);
    const clo_rope_plan* plan = address<const clo_rope_plan>(a[0]);
    const int transpose = PyObject_IsTrue(a[4]);
    if (transpose < 0) throw Raised{};
    void* stream = stream_of(a[5], dev);
    const clo_status st = without_gil([&] { return clo_rope(plan, &x, &y, pos, tokens, (int32_t)heads, (int32_t)d, transpose, stream); });
    if (st) return PyLong_FromLong(st);
    written(a[3]);
    return THPVariable_Wrap(out);
  });
}

// cache, cache device, k, v, q_starts, kv_lens, block_table, plan (0: none), positions, q, q_out, max_q, stream, the cache's tensors (a tuple)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    const clo_paged_cache* c = address<const clo_paged_cache>(a[0]);
    const int dev = device_of(cuda_tensor(a[2], "k"), "k");
    clo_rows k, v, q{}, y{};
    const at::Tensor& kt = rows(a[2], "k", dev, &k);
    const int64_t total = kt.size(0);
    shape_is(kt, "k", total, c->n_kv_heads, c->head_dim);
    shape_is(rows(a[3], "v", dev, &v), "v", total, c->n_kv_heads, c->head_dim);
    const clo_paged_batch b = batch_of(a[4], a[5], a[6], total, a[11], dev, small(a[1], "device"));
    const int64_t* pos = a[8] == Py_None ? nullptr : vector_of<int64_t>(a[8], "positions", dev, at::kLong, total);
    at::Tensor out;
    int32_t heads = 0;
    if (a[9] != Py_None) {
      const at::Tensor& qt = rows(a[9], "q", dev, &q);
      if (qt.size(1) > INT32_MAX) refuse("q is too large");
      heads = (int32_t)qt.size(1);
      shape_is(qt, "q", total, heads, c->head_dim);
      out = output(a[10], "q_out", dev, total, heads, c->head_dim, &y, a[12]);
    } else if (a[10] != Py_None) {
      refuse("q_out without q");
    }
    const bool with_q = a[9] != Py_None;
    const clo_rope_plan* plan = address<const clo_rope_plan>(a[7]);
    void* stream = stream_of(a[12], dev);
    const clo_status st =
        without_gil([&] { return clo_paged_append(c, &b, plan, pos, &k, &v, with_q ? &q : nullptr, with_q ? &y : nullptr, heads, stream); });
    if (st) return PyLong_FromLong(st);
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(a[13]); ++i) written(PyTuple_GET_ITEM(a[13], i));
    written(a[10]);
    if (with_q) return THPVariable_Wrap(out);
    Py_RETURN_NONE;
  });
}

// cache, cache device, q_starts, kv_lens, block_table, total, k_out, v_out, max_q, stream
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const clo_paged_cache* c = address<const clo_paged_cache>(a[0]);
    const int dev = device_of(cuda_tensor(a[3], "kv_lens"), "kv_lens");
    const int64_t total = integer(a[5], "total");
    if (total < 0) refuse("total must not be negative");
    clo_rows k, v;
    at::Tensor kt = output(a[6], "k_out", dev, total, c->n_kv_heads, c->head_dim, &k, a[9]);
    at::Tensor vt = output(a[7], "v_out", dev, total, c->n_kv_heads, c->head_dim, &v, a[9]);
    const clo_paged_batch b = batch_of(a[2], a[3], a[4], total, a[8], dev, small(a[1], "device"));
    void* stream = stream_of(a[9], dev);
    const clo_status st = without_gil([&] { return clo_paged_read(c, &b, &k, &v, stream); });
    if (st) return PyLong_FromLong(st);
    written(a[6]);
    written(a[7]);
    PyObject* kw = THPVariable_Wrap(kt);
    PyObject* vw = THPVariable_Wrap(vt);
    PyObject* pair = kw && vw ? PyTuple_Pack(2, kw, vw) : nullptr;
    Py_XDECREF(kw);
    Py_XDECREF(vw);
    return pair;
  });
}

// cache, cache device, q, q_starts, kv_lens, block_table, out, max_q, softmax_scale, window, sinks, workspace, stream
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    const clo_paged_cache* c = address<const clo_paged_cache>(a[0]);
    const int dev = device_of(cuda_tensor(a[2], "q"), "q");
    clo_rows q, o;
    const at::Tensor& qt = rows(a[2], "q", dev, &q);
    const int64_t total = qt.size(0), heads = qt.size(1);
    if (qt.size(2) != c->head_dim) refuse("q has head_dim %lld; the cache has %d", (long long)qt.size(2), c->head_dim);
    if (heads > INT32_MAX) refuse("q is too large");
    const clo_paged_batch b = batch_of(a[3], a[4], a[5], total, a[7], dev, small(a[1], "device"));
    at::Tensor out = output(a[6], "out", dev, total, heads, c->head_dim, &o, a[12]);
    const double scale = PyFloat_AsDouble(a[8]);
    if (scale == -1.0 && PyErr_Occurred()) throw Raised{};
    const int32_t window = small(a[9], "window"), sinks = small(a[10], "sinks");
    void* stream = stream_of(a[12], dev);
    void* work = nullptr;
    int64_t bytes = 0;
    at::Tensor own;
    if (a[11] != Py_None) {
      const at::Tensor& w = tensor_on(a[11], "workspace", dev, at::kByte);
      if (!w.is_contiguous()) refuse("workspace must be contiguous");
      work = w.data_ptr();
      bytes = w.numel();
    } else {
      if (const clo_status st = clo_paged_attention_workspace(c, &b, (int32_t)heads, window, sinks, &bytes)) return PyLong_FromLong(st);
      if (bytes) {
        own = new_tensor({bytes}, at::kByte, dev, a[12], false);
        work = own.data_ptr();
      }
    }
    const clo_status st =
        without_gil([&] { return clo_paged_attention(c, &b, &q, &o, (int32_t)heads, (float)scale, window, sinks, work, bytes, stream); });
    if (st) return PyLong_FromLong(st);
    written(a[6]);
    written(a[11]);
    return THPVariable_Wrap(out);
  });
}

#define CLO_METHOD(name) \
  { #name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL, "" }
PyMethodDef methods[] = {CLO_METHOD(rope), CLO_METHOD(append), CLO_METHOD(read), CLO_METHOD(attention), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_clo_torch", "Marshalling of torch tensors for libclo.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__clo_torch() { return PyModule_Create(&module); }
