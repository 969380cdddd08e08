// Python binding of the paged cache's calls: checks torch tensors and passes their
// pointers and sizes to the C ABI.  A serving step makes several of these calls in
// a few microseconds of GPU time each, which marshalling in Python would exceed
// (15 us for a plan, 5 of them the call itself).
//
// bind() takes the addresses of the ABI's functions, so that the module uses the
// library that was loaded (the regular or the bounds-checked one), and the
// exception that a status other than KVQ_OK raises.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <initializer_list>

#include "kvq.h"

namespace {

decltype(&kvq_page_plan) f_plan;
decltype(&kvq_paged_append) f_append;
decltype(&kvq_paged_gather) f_gather;
decltype(&kvq_paged_decode) f_decode;
decltype(&kvq_paged_decode_workspace_bytes) f_workspace;
PyObject* error_type;  // KvqError(status, what)

struct Refused {};  // a Python exception is set

template <typename... A>
[[noreturn]] void refuse(const char* format, A... a) {
  PyErr_Format(PyExc_ValueError, format, a...);
  throw Refused();
}

// the argument as a tensor; nullptr for None
const at::Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse("%s is a tensor", name);
  return &THPVariable_Unpack(o);
}
const at::Tensor& given(PyObject* o, const char* name) {
  const at::Tensor* t = tensor(o, name);
  if (!t) refuse("%s is a tensor", name);
  return *t;
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}
int32_t integer32(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse("%s is out of range", name);
  return (int32_t)v;
}

// the one CUDA device that the tensors, and the pool where there is one, are on
int one_device(std::initializer_list<const at::Tensor*> all, int64_t pool = -1) {
  int64_t dev = pool;
  for (const at::Tensor* t : all) {
    if (!t) continue;
    if (!t->is_cuda()) refuse("expected CUDA tensors (the library has no CPU path)");
    const int64_t d = t->get_device();
    if (dev < 0) dev = d;
    if (d != dev) refuse("tensors on cuda:%d and cuda:%d", (int)dev, (int)d);
  }
  return (int)dev;
}

int32_t* ints(const at::Tensor* t, const char* name, std::initializer_list<int64_t> shape) {
  if (!t) return nullptr;
  if (t->scalar_type() != at::kInt || !t->sizes().equals(at::IntArrayRef(shape.begin(), shape.size())) || !t->is_contiguous())
    refuse("%s is a contiguous int32 tensor of %d dimensions, the first %d", name, (int)shape.size(), (int)*shape.begin());
  return static_cast<int32_t*>(t->data_ptr());
}

kvq_dtype type_of(at::ScalarType t, const char* name) {
  if (t == at::kFloat) return KVQ_F32;
  if (t == at::kBFloat16) return KVQ_BF16;
  if (t == at::kHalf) return KVQ_F16;
  refuse("%s is fp32, bf16 or fp16", name);
}

// [rows][heads][128] with contiguous heads: the row stride in elements
int64_t row_stride(const at::Tensor& t, const char* name, int64_t heads) {
  if (t.dim() != 3 || t.size(1) != heads || t.size(2) != 128) refuse("%s is [rows][%d][128]", name, (int)heads);
  if (t.size(0) && (t.stride(2) != 1 || (heads > 1 && t.stride(1) != 128)))
    refuse("%s: a row's heads and channels are contiguous", name);
  return t.size(0) > 1 ? t.stride(0) : heads * 128;
}

// The device and the stream of a call: the caller's, or the device's current one.  The
// caller's is made current for the length of the call, so that memory allocated in it
// belongs to the stream that uses it: a workspace given back on return goes to later work
// of that stream only, and a new output is not still in use by another.
class Place {
 public:
  Place(PyObject* o, int dev) : device_((c10::DeviceIndex)dev) {
    if (o == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
      return;
    }
    stream = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) throw Refused();
    stream_.reset_stream(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(stream), (c10::DeviceIndex)dev));
  }
  void* stream;

 private:
  c10::cuda::CUDAGuard device_;
  c10::cuda::OptionalCUDAStreamGuard stream_;
};

// A launch waits while the device's queue is full, an allocation may wait for the
// device: neither holds up the process's other Python threads.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

template <typename F, typename... A>
void call(const char* what, F f, A... a) {
  kvq_status s;
  {
    Unlocked u;
    s = f(a...);
  }
  if (s == KVQ_OK) return;
  if (PyObject* e = PyObject_CallFunction(error_type, "is", (int)s, what)) {
    PyErr_SetObject(error_type, e);
    Py_DECREF(e);
  }
  throw Refused();
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, int dev) {
  Unlocked u;
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)dev));
}

// n int32 elements of a buffer as a tensor of its own, without a dispatch
at::Tensor part(const at::Tensor& buf, int64_t offset, int64_t n) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(buf.storage()), buf.key_set(),
                                                          buf.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(offset);
  t.unsafeGetTensorImpl()->set_sizes_contiguous({n});
  return t;
}

// an output: the caller's, checked, or a new one
at::Tensor output(const at::Tensor* t, const char* name, at::IntArrayRef shape, at::ScalarType type, int dev) {
  if (!t) return empty(shape, type, dev);
  if (!t->sizes().equals(shape) || t->scalar_type() != type || !t->is_contiguous())
    refuse("%s is contiguous, of the result's shape and type", name);
  return *t;
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", n, want);
    return nullptr;
  }
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// bind(plan, append, gather, decode, workspace, error)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    f_plan = reinterpret_cast<decltype(f_plan)>(integer(a[0]));
    f_append = reinterpret_cast<decltype(f_append)>(integer(a[1]));
    f_gather = reinterpret_cast<decltype(f_gather)>(integer(a[2]));
    f_decode = reinterpret_cast<decltype(f_decode)>(integer(a[3]));
    f_workspace = reinterpret_cast<decltype(f_workspace)>(integer(a[4]));
    Py_INCREF(a[5]);
    error_type = a[5];
    Py_RETURN_NONE;
  });
}

// plan(num_pages, page_tokens, ctx_lens, new_lens, block_table, free_pages, free_count, n_slots, done, out, stream)
// out: None, or a tuple (slots, positions, cu_new, seq_lens, free_count); returns that tuple
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const int32_t num_pages = integer32(a[0], "num_pages"), page_tokens = integer32(a[1], "page_tokens");
    const int32_t n_slots = integer32(a[7], "n_slots");
    const at::Tensor &ctx = given(a[2], "ctx_lens"), &add = given(a[3], "new_lens"), &table = given(a[4], "block_table");
    const at::Tensor &free_pages = given(a[5], "free_pages"), &count = given(a[6], "free_count");
    const at::Tensor* done = tensor(a[8], "done");
    if (table.dim() != 2) refuse("block_table is [B][max_pages]");
    if (n_slots < 0) refuse("n_slots is out of range");
    const int64_t B = table.size(0), max_pages = table.size(1);
    if (B > INT32_MAX || max_pages > INT32_MAX) refuse("block_table is too large");
    const int dev = one_device({&ctx, &add, &table, &free_pages, &count, done});
    const int64_t sizes[5] = {n_slots, n_slots, B + 1, B, 1};
    const char* names[5] = {"slots", "positions", "cu_new", "seq_lens", "free_count"};
    const Place on(a[10], dev);
    at::Tensor out[5], buf;
    int32_t* p[5];
    int64_t used = 0;
    if (a[9] == Py_None) buf = empty(2 * (n_slots + 3ll) + 2 * B + 8, at::kInt, dev);  // one allocation of five arrays
    for (int i = 0; i < 5; ++i) {
      if (a[9] == Py_None) {
        out[i] = part(buf, used, sizes[i]);
        p[i] = static_cast<int32_t*>(buf.data_ptr()) + used;
        used += i < 2 ? (sizes[i] + 3) & ~3ll : sizes[i];  // slots and positions start on 16 bytes
      } else {
        if (!PyTuple_Check(a[9]) || PyTuple_GET_SIZE(a[9]) != 5) refuse("out is a tuple of five tensors");
        const at::Tensor& t = given(PyTuple_GET_ITEM(a[9], i), names[i]);
        one_device({&ctx, &t});
        p[i] = ints(&t, names[i], {sizes[i]});
      }
    }
    call("kvq_page_plan", f_plan, num_pages, page_tokens, (int32_t)B, ints(&ctx, "ctx_lens", {B}),
         ints(&add, "new_lens", {B}), ints(done, "done", {B}), ints(&table, "block_table", {B, max_pages}),
         (int32_t)max_pages, ints(&free_pages, "free_pages", {num_pages}), ints(&count, "free_count", {1}), p[4], p[0],
         p[1], n_slots, p[2], p[3], on.stream);
    if (a[9] != Py_None) {
      Py_INCREF(a[9]);
      return a[9];
    }
    PyObject* t = PyTuple_New(5);
    if (!t) throw Refused();
    for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(t, i, THPVariable_Wrap(out[i]));
    return t;
  });
}

// append(descriptor, kv_heads, device, k_new, v_new, slots, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 7, [&]() -> PyObject* {
    const int64_t H = integer(a[1]);
    const at::Tensor &k = given(a[3], "k_new"), &v = given(a[4], "v_new"), &slots = given(a[5], "slots");
    const int dev = one_device({&k, &v, &slots}, integer(a[2]));
    if (k.scalar_type() != v.scalar_type() || !k.sizes().equals(v.sizes())) refuse("k_new and v_new have one type and shape");
    const int64_t ks = row_stride(k, "k_new", H), vs = row_stride(v, "v_new", H), rows = k.size(0);
    const int32_t* at_slots = ints(&slots, "slots", {rows});
    if (rows > INT32_MAX) refuse("k_new has too many rows");
    const Place on(a[6], dev);
    call("kvq_paged_append", f_append, reinterpret_cast<const kvq_paged_cache*>(integer(a[0])), k.data_ptr(), ks,
         v.data_ptr(), vs, type_of(k.scalar_type(), "k_new"), (int32_t)rows, at_slots, on.stream);
    Py_RETURN_NONE;
  });
}

// gather(descriptor, kv_heads, device, slots, type code, rotate_back, k_out, v_out, stream) -> (k, v)
PyObject* gather(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const int64_t H = integer(a[1]), code = integer(a[4]);
    const at::Tensor& slots = given(a[3], "slots");
    const at::Tensor *k_out = tensor(a[6], "k_out"), *v_out = tensor(a[7], "v_out");
    const int dev = one_device({&slots, k_out, v_out}, integer(a[2]));
    const int64_t rows = slots.numel();
    const int32_t* at_slots = ints(&slots, "slots", {rows});
    if (rows > INT32_MAX) refuse("slots has too many entries");
    const at::ScalarType type = code == KVQ_F32 ? at::kFloat : code == KVQ_BF16 ? at::kBFloat16 : at::kHalf;
    const Place on(a[8], dev);
    const int64_t shape[3] = {rows, H, 128};
    at::Tensor k = output(k_out, "k_out", shape, type, dev), v = output(v_out, "v_out", shape, type, dev);
    call("kvq_paged_gather", f_gather, reinterpret_cast<const kvq_paged_cache*>(integer(a[0])), at_slots, (int32_t)rows,
         (kvq_dtype)code, integer32(a[5], "rotate_back"), k.data_ptr(), v.data_ptr(), on.stream);
    PyObject* t = PyTuple_New(2);
    if (!t) throw Refused();
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(k));
    PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(v));
    return t;
  });
}

// decode(descriptor, kv_heads, device, q, block_table, seq_lens, max_len, mask, softmax_scale, out, workspace, stream) -> out
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const auto* desc = reinterpret_cast<const kvq_paged_cache*>(integer(a[0]));
    const int64_t H = integer(a[1]);
    const at::Tensor &q = given(a[3], "q"), &table = given(a[4], "block_table"), &lens = given(a[5], "seq_lens");
    const at::Tensor *mask = tensor(a[7], "mask"), *out = tensor(a[9], "out"), *ws = tensor(a[10], "workspace");
    const int dev = one_device({&q, &table, &lens, mask, out, ws}, integer(a[2]));
    const double scale = PyFloat_AsDouble(a[8]);
    if (scale == -1.0 && PyErr_Occurred()) throw Refused();
    if (q.dim() != 3 || table.dim() != 2) refuse("q is [B][Hq][128], block_table [B][max_pages]");
    const int64_t B = q.size(0), Hq = q.size(1), max_pages = table.size(1);
    const int64_t stride = row_stride(q, "q", Hq);
    const kvq_dtype type = type_of(q.scalar_type(), "q");
    const int32_t *p_table = ints(&table, "block_table", {B, max_pages}), *p_lens = ints(&lens, "seq_lens", {B});
    const int32_t* p_mask = ints(mask, "mask", {B, H});
    if (B > INT32_MAX || Hq > INT32_MAX || max_pages > INT32_MAX) refuse("q or block_table is too large");
    const Place on(a[11], dev);
    const int64_t shape[3] = {B, Hq, 128};
    at::Tensor o = output(out, "out", shape, q.scalar_type(), dev);
    at::Tensor own;
    if (!ws) {
      own = empty((int64_t)std::max<size_t>(f_workspace(desc, (int32_t)B, (int32_t)Hq), 256), at::kByte, dev);
      ws = &own;
    } else if (!ws->is_contiguous()) {
      refuse("workspace is contiguous");
    }
    call("kvq_paged_decode", f_decode, desc, q.data_ptr(), stride, type, (int32_t)Hq, (int32_t)B, p_table,
         (int32_t)max_pages, p_lens, integer32(a[6], "max_len"), reinterpret_cast<const uint32_t*>(p_mask), (float)scale,
         o.data_ptr(), ws->data_ptr(), ws->nbytes(), on.stream);
    return THPVariable_Wrap(o);
  });
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"bind", FAST(bind), nullptr},     {"plan", FAST(plan), nullptr},
                         {"append", FAST(append), nullptr}, {"gather", FAST(gather), nullptr},
                         {"decode", FAST(decode), nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "kvq_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_kvq_torch() { return PyModule_Create(&module); }
