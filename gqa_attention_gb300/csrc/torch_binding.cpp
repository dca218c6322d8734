// torch_binding.cpp -- the block-scaled cache's helpers for torch tensors: checks of
// types, shapes and devices, outputs and workspaces from torch's allocator, and
// the calls of the C ABI (include/gqa_attn.h).  Argument marshalling only, like the
// ctypes binding; in C++ because these calls launch kernels of 2 to 20 us, and the
// same checks and allocations took 10 to 20 us in Python.
//
// The module does not link the library: every function takes the handle of the
// loaded libgqa_attn.so and looks its entry points up once per handle.
#include <Python.h>
#include <dlfcn.h>

#include <cmath>
#include <optional>
#include <string>
#include <vector>

#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gqa_attn.h"

namespace {

struct Library {
  void* handle;
  decltype(&gqa_kv_append_fp8_block) append;
  decltype(&gqa_kv_append_paged_fp8_block) append_paged;
  decltype(&gqa_kv_read_fp8_block) read;
  decltype(&gqa_kv_read_paged_fp8_block) read_paged;
  decltype(&gqa_attn_decode_fp8_block) decode;
  decltype(&gqa_attn_decode_paged_fp8_block) decode_paged;
  decltype(&gqa_attn_decode_fp8_block_default_splits) default_splits;
  decltype(&gqa_attn_decode_workspace_bytes) workspace_bytes;
};

// A refused call: raised as the package's GQAError(status, what).
struct Refused {
  int status;
  std::string what;
};
PyObject* g_error = nullptr;

template <typename F>
void symbol(void* handle, const char* name, F* out) {
  *out = reinterpret_cast<F>(dlsym(handle, name));
  if (!*out) throw Refused{GQA_ERR_UNSUPPORTED, std::string(name) + " is not in the library"};
}

// (under the interpreter's lock, like every function here)
const Library& library(PyObject* arg) {
  static std::vector<Library> known;
  void* handle = PyLong_AsVoidPtr(arg);
  if (PyErr_Occurred()) throw python_error();
  for (const Library& l : known)
    if (l.handle == handle) return l;
  Library l{handle};
  symbol(handle, "gqa_kv_append_fp8_block", &l.append);
  symbol(handle, "gqa_kv_append_paged_fp8_block", &l.append_paged);
  symbol(handle, "gqa_kv_read_fp8_block", &l.read);
  symbol(handle, "gqa_kv_read_paged_fp8_block", &l.read_paged);
  symbol(handle, "gqa_attn_decode_fp8_block", &l.decode);
  symbol(handle, "gqa_attn_decode_paged_fp8_block", &l.decode_paged);
  symbol(handle, "gqa_attn_decode_fp8_block_default_splits", &l.default_splits);
  symbol(handle, "gqa_attn_decode_workspace_bytes", &l.workspace_bytes);
  known.reserve(64);  // (references stay valid)
  if (known.size() == known.capacity()) throw Refused{GQA_ERR_UNSUPPORTED, "too many libraries"};
  known.push_back(l);
  return known.back();
}

[[noreturn]] void refuse(const char* call, const char* why) {
  throw Refused{GQA_ERR_INVALID_ARG, std::string(call) + ": " + why};
}
void need(bool ok, const char* call, const char* why) {
  if (!ok) refuse(call, why);
}
void check(gqa_status st, const char* call) {
  if (st != GQA_OK) throw Refused{st, call};
}

const at::Tensor& tensor(PyObject* o, const char* call) {
  if (!THPVariable_Check(o)) refuse(call, "a tensor is expected");
  return THPVariable_Unpack(o);
}
std::optional<at::Tensor> maybe_tensor(PyObject* o, const char* call) {
  if (o == Py_None) return std::nullopt;
  return tensor(o, call);
}
int as_int(PyObject* o, const char* call) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  need(v >= INT32_MIN && v <= INT32_MAX, call, "an integer is out of range");
  return static_cast<int>(v);
}
int as_dim(int64_t v, const char* call) {
  need(v <= INT32_MAX, call, "a dimension is out of range");
  return static_cast<int>(v);
}
bool dense(const at::Tensor& t, at::ScalarType type, c10::DeviceIndex dev) {
  return t.scalar_type() == type && t.is_cuda() && t.get_device() == dev && t.is_contiguous();
}
template <typename T>
T* ptr(const std::optional<at::Tensor>& t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

// The tensors of a cache, checked.
struct Cache {
  at::Tensor k8, v8, ks, vs, lens;
  std::optional<at::Tensor> table;
  c10::DeviceIndex dev;
  int units, per, H, d, B, max_blocks, block;
  int s_max() const { return table ? static_cast<int>(int64_t(max_blocks) * per) : per; }
};

Cache cache(PyObject* const* a, PyObject* block, PyObject* table, const char* call) {
  Cache c{tensor(a[0], call), tensor(a[1], call), tensor(a[2], call), tensor(a[3], call),
          tensor(a[4], call), maybe_tensor(table, call)};
  c.block = as_int(block, call);
  need(c.k8.is_cuda() && c.k8.dim() == 4 && c.k8.sizes() == c.v8.sizes(), call,
       "the codes are uint8 [B, S_max, H_kv, d] or [num_pages, page_size, H_kv, d], K and V on one "
       "CUDA device");
  c.dev = c.k8.get_device();
  need(dense(c.k8, at::kByte, c.dev) && dense(c.v8, at::kByte, c.dev), call,
       "the codes are dense uint8, K and V on one CUDA device");
  c.units = as_dim(c.k8.size(0), call);
  c.per = as_dim(c.k8.size(1), call);
  c.H = as_dim(c.k8.size(2), call);
  c.d = as_dim(c.k8.size(3), call);
  need(c.block > 0, call, "block is positive");
  const int64_t shape[3] = {c.units, (int64_t(c.per) + c.block - 1) / c.block, c.H};
  need(c.ks.sizes() == at::IntArrayRef(shape, 3) && c.vs.sizes() == at::IntArrayRef(shape, 3) &&
           dense(c.ks, at::kFloat, c.dev) && dense(c.vs, at::kFloat, c.dev),
       call, "the scales are dense float32 [units, ceil(tokens / block), H_kv] on the codes' device");
  c.B = c.units;
  c.max_blocks = 0;
  if (c.table) {
    need(c.table->dim() == 2 && dense(*c.table, at::kInt, c.dev), call,
         "block_table is dense int32 [B, max_blocks] on the codes' device");
    c.B = as_dim(c.table->size(0), call);
    c.max_blocks = as_dim(c.table->size(1), call);
    need(int64_t(c.max_blocks) * c.per <= INT32_MAX, call, "max_blocks * page_size is out of range");
  }
  need(c.lens.dim() == 1 && c.lens.size(0) == c.B && dense(c.lens, at::kInt, c.dev), call,
       "seq_lens is dense int32 [B] on the codes' device");
  return c;
}

// The stream of a call: given, or the current one of the device.  What a call
// allocates belongs to that stream (torch's allocator orders reuse by it).
struct Stream {
  gqa_stream_t raw;
  bool given;
};
struct AllocateOn {
  AllocateOn(const Stream& s, c10::DeviceIndex dev) {
    if (s.given)
      guard.reset_stream(
          c10::cuda::getStreamFromExternal(reinterpret_cast<cudaStream_t>(s.raw), dev));
  }
  c10::cuda::OptionalCUDAStreamGuard guard;
};
Stream stream_of(PyObject* o, c10::DeviceIndex dev) {
  if (o == Py_None)
    return {reinterpret_cast<gqa_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream()), false};
  if (PyLong_Check(o)) {
    void* p = PyLong_AsVoidPtr(o);
    if (PyErr_Occurred()) throw python_error();
    return {static_cast<gqa_stream_t>(p), true};
  }
  PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
  if (!h) throw python_error();
  void* p = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (PyErr_Occurred()) throw python_error();
  return {static_cast<gqa_stream_t>(p), true};
}

// An output, from torch's allocator without its dispatcher (1.4 us a tensor, of a call of 5).
at::Tensor empty(at::IntArrayRef sizes, at::ScalarType type, c10::DeviceIndex dev) {
  return at::detail::empty_cuda(sizes, type, c10::Device(c10::kCUDA, dev), std::nullopt);
}
// Memory that a call's own kernels use, without a tensor around it: back in the
// allocator at the end of the call, which hands it on in the order of its stream.
struct Scratch {
  void* ptr = nullptr;
  void take(size_t bytes, const Stream& s) {
    ptr = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(
        bytes, reinterpret_cast<cudaStream_t>(s.raw));
  }
  ~Scratch() {
    if (ptr) c10::cuda::CUDACachingAllocator::raw_delete(ptr);
  }
};

PyObject* raise(const Refused& r) {
  PyObject* e = PyObject_CallFunction(g_error, "is", r.status, r.what.c_str());
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return nullptr;
}

PyObject* pair(const at::Tensor& x, const at::Tensor& y) {
  PyObject* a = THPVariable_Wrap(x);
  PyObject* b = a ? THPVariable_Wrap(y) : nullptr;
  PyObject* t = b ? PyTuple_New(2) : nullptr;
  if (!t) {
    Py_XDECREF(a);
    Py_XDECREF(b);
    return nullptr;
  }
  PyTuple_SET_ITEM(t, 0, a);
  PyTuple_SET_ITEM(t, 1, b);
  return t;
}

// append(handle, k8, v8, k_scale, v_scale, seq_lens, block, block_table, stream, k_new, v_new, n_new)
PyObject* append_(PyObject* const* a) {
  static const char* call = "kv_append_fp8_block";
  const Library& lib = library(a[0]);
  const Cache c = cache(a + 1, a[6], a[7], call);
  const at::Tensor &k = tensor(a[9], call), &v = tensor(a[10], call);
  const std::optional<at::Tensor> n_new = maybe_tensor(a[11], call);
  need(k.dim() == 4 && k.size(0) == c.B && k.size(2) == c.H && k.size(3) == c.d &&
           v.sizes() == k.sizes() && k.scalar_type() == at::kBFloat16 &&
           v.scalar_type() == at::kBFloat16 && k.is_cuda() && v.is_cuda() &&
           k.get_device() == c.dev && v.get_device() == c.dev,
       call, "the new rows are bfloat16 [B, T, H_kv, d] on the cache's device");
  need(!n_new || (n_new->dim() == 1 && n_new->size(0) == c.B && dense(*n_new, at::kInt, c.dev)),
       call, "n_new is dense int32 [B] on the cache's device");
  const int64_t T = k.size(1);
  if (T == 0) Py_RETURN_NONE;
  // the stride between tokens; a dimension of size 1 has none of its own
  const int64_t step = T > 1 ? k.stride(1) : c.B > 1 ? k.stride(0) : int64_t(c.H) * c.d;
  for (const at::Tensor* x : {&k, &v})
    need(x->stride(3) == 1 && (c.H == 1 || x->stride(2) == c.d) && (T == 1 || x->stride(1) == step) &&
             (c.B == 1 || x->stride(0) == T * step),
         call, "the rows of k_new and v_new are H_kv * d dense elements, one stride apart");
  const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, c.dev));
  const Stream s = stream_of(a[8], c.dev);
  float *ks = static_cast<float*>(c.ks.data_ptr()), *vs = static_cast<float*>(c.vs.data_ptr());
  const int32_t* lens = static_cast<const int32_t*>(c.lens.data_ptr());
  check(c.table ? lib.append_paged(k.data_ptr(), v.data_ptr(), step, ptr<int32_t>(n_new),
                                   ptr<int32_t>(c.table), lens, c.B, as_dim(T, call), c.units, c.per,
                                   c.max_blocks, c.H, c.d, c.block, c.k8.data_ptr(),
                                   c.v8.data_ptr(), ks, vs, s.raw)
                : lib.append(k.data_ptr(), v.data_ptr(), step, ptr<int32_t>(n_new), lens, c.B,
                             as_dim(T, call), c.per, c.H, c.d, c.block, c.k8.data_ptr(),
                             c.v8.data_ptr(), ks, vs, s.raw),
        call);
  Py_RETURN_NONE;
}

// read(handle, k8, v8, k_scale, v_scale, seq_lens, block, block_table, stream, start, k_out, v_out)
PyObject* read_(PyObject* const* a) {
  static const char* call = "kv_read_fp8_block";
  const Library& lib = library(a[0]);
  const Cache c = cache(a + 1, a[6], a[7], call);
  const int start = as_int(a[9], call);
  std::optional<at::Tensor> k = maybe_tensor(a[10], call), v = maybe_tensor(a[11], call);
  const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, c.dev));
  const Stream s = stream_of(a[8], c.dev);
  const AllocateOn on(s, c.dev);
  if (!k) {
    need(start >= 0 && start < c.s_max(), call, "start lies in the cache");
    k = at::zeros({c.B, c.s_max() - start, c.H, c.d}, c.k8.options().dtype(at::kBFloat16));
  }
  if (!v) v = at::zeros(k->sizes(), c.k8.options().dtype(at::kBFloat16));
  need(k->dim() == 4 && k->size(0) == c.B && k->size(2) == c.H && k->size(3) == c.d &&
           v->sizes() == k->sizes() && dense(*k, at::kBFloat16, c.dev) &&
           dense(*v, at::kBFloat16, c.dev),
       call, "k_out and v_out are dense bfloat16 [B, S_out, H_kv, d] on the cache's device");
  const float *ks = static_cast<const float*>(c.ks.data_ptr()),
              *vs = static_cast<const float*>(c.vs.data_ptr());
  const int32_t* lens = static_cast<const int32_t*>(c.lens.data_ptr());
  const int S_out = as_dim(k->size(1), call);
  check(c.table ? lib.read_paged(c.k8.data_ptr(), c.v8.data_ptr(), ks, vs, ptr<int32_t>(c.table),
                                 lens, c.B, c.units, c.per, c.max_blocks, c.H, c.d, c.block, start,
                                 S_out, k->data_ptr(), v->data_ptr(), s.raw)
                : lib.read(c.k8.data_ptr(), c.v8.data_ptr(), ks, vs, lens, c.B, c.per, c.H, c.d,
                           c.block, start, S_out, k->data_ptr(), v->data_ptr(), s.raw),
        call);
  return pair(*k, *v);
}

// decode(handle, k8, v8, k_scale, v_scale, seq_lens, block, block_table, stream, q, scale, n_split,
//        workspace, out, lse)
PyObject* decode_(PyObject* const* a) {
  static const char* call = "decode_fp8_block";
  const Library& lib = library(a[0]);
  const Cache c = cache(a + 1, a[6], a[7], call);
  const at::Tensor& q = tensor(a[9], call);
  need((q.dim() == 3 || q.dim() == 4) && q.size(0) == c.B && q.size(-1) == c.d &&
           dense(q, at::kBFloat16, c.dev),
       call, "q is dense bfloat16 [B, H_q, d] or [B, T_q, H_q, d] on the cache's device");
  const int T_q = q.dim() == 4 ? as_dim(q.size(1), call) : 1, H_q = as_dim(q.size(-2), call);
  double scale = 1.0 / std::sqrt(static_cast<double>(c.d));
  if (a[10] != Py_None) {
    scale = PyFloat_AsDouble(a[10]);
    if (PyErr_Occurred()) throw python_error();
  }
  std::optional<at::Tensor> ws = maybe_tensor(a[12], call), out = maybe_tensor(a[13], call),
                            lse = maybe_tensor(a[14], call);
  const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, c.dev));
  const at::IntArrayRef rows = q.sizes().slice(0, q.dim() - 1);
  need(!out || (out->sizes() == q.sizes() && dense(*out, at::kBFloat16, c.dev)), call,
       "out is dense bfloat16, of q's shape, on the cache's device");
  need(!lse || (lse->sizes() == rows && dense(*lse, at::kFloat, c.dev)), call,
       "lse is dense float32, of q's shape without d, on the cache's device");
  const Stream s = stream_of(a[8], c.dev);
  const AllocateOn on(s, c.dev);
  if (!out) out = empty(q.sizes(), at::kBFloat16, c.dev);
  if (!lse) lse = empty(rows, at::kFloat, c.dev);
  Scratch scratch;
  const int n_split = a[11] == Py_None ? lib.default_splits(c.B, T_q, H_q, c.H, c.s_max())
                                       : as_int(a[11], call);
  if (n_split > 1) {
    const int64_t bytes = static_cast<int64_t>(
        lib.workspace_bytes(as_dim(int64_t(c.B) * T_q, call), H_q, c.d, n_split));
    need(!ws || (ws->is_cuda() && ws->get_device() == c.dev && ws->is_contiguous() &&
                 static_cast<int64_t>(ws->nbytes()) >= bytes),
         call, "the workspace is too small, or not dense on the cache's device");
    // (none for sizes that the call below refuses)
    if (!ws && bytes > 0) scratch.take(static_cast<size_t>(bytes), s);
  }
  void* const space = ws ? ws->data_ptr() : scratch.ptr;
  const float *ks = static_cast<const float*>(c.ks.data_ptr()),
              *vs = static_cast<const float*>(c.vs.data_ptr());
  const int32_t* lens = static_cast<const int32_t*>(c.lens.data_ptr());
  float* l = static_cast<float*>(lse->data_ptr());
  const float tau = static_cast<float>(scale);
  check(c.table ? lib.decode_paged(q.data_ptr(), c.k8.data_ptr(), c.v8.data_ptr(), ks, vs,
                                   ptr<int32_t>(c.table), lens, c.B, T_q, c.units, c.per,
                                   c.max_blocks, H_q, c.H, c.d, c.block, tau, n_split,
                                   space, out->data_ptr(), l, s.raw)
                : lib.decode(q.data_ptr(), c.k8.data_ptr(), c.v8.data_ptr(), ks, vs, lens, c.B, T_q,
                             c.per, H_q, c.H, c.d, c.block, tau, n_split, space,
                             out->data_ptr(), l, s.raw),
        call);
  return pair(*out, *lse);
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& r) {
    return raise(r);
  }
  END_HANDLE_TH_ERRORS
}

PyObject* init_(PyObject*, PyObject* error) {
  Py_INCREF(error);
  Py_XSETREF(g_error, error);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"init", init_, METH_O, "init(error): the exception class of refused calls"},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(entry<append_, 12>)),
     METH_FASTCALL, nullptr},
    {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(entry<read_, 12>)),
     METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(entry<decode_, 15>)),
     METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch_binding", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__torch_binding() { return PyModule_Create(&module); }
