// Argument marshalling of the per-layer calls of a decode step (paged_rope_append,
// paged_page_bounds, paged_sparse_attn, paged_prefix_attn) for Python: tensors are checked and
// taken apart here, where that costs about a microsecond, and libkara is called on the current
// stream. In Python the same checks and a ctypes call with two dozen arguments take 15 us, several
// times what the kernels of a decode step need.
//
// Every function takes its arguments by position, raises ValueError for a tensor that does not
// fit, and returns the output tensor or, when the library refuses the call, its status code.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <dlfcn.h>

#include <cmath>
#include <initializer_list>
#include <string>

#include "kara.h"

namespace {

struct Library {
  decltype(&paged_rope_append) rope_append = nullptr;
  decltype(&paged_page_bounds) page_bounds = nullptr;
  decltype(&paged_sparse_attn) sparse_attn = nullptr;
  decltype(&paged_prefix_attn) prefix_attn = nullptr;
  decltype(&kara_workspace_bytes) workspace_bytes = nullptr;
} g_lib;

[[noreturn]] void refuse(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw python_error();
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "[";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + "]";
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kInt: return "torch.int32";
    case at::kFloat: return "torch.float32";
    case at::kByte: return "torch.uint8";
    default: return "another type";
  }
}

// The tensors of one call, all on the device of the first, which must be the current one.
struct Call {
  int device = -1;

  const at::Tensor& tensor(PyObject* o, at::ScalarType type, const char* name) {
    if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a CUDA tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
    if (t.scalar_type() != type)
      refuse(std::string(name) + " must be " + type_name(type) + ", got " + at::toString(t.scalar_type()));
    if (device < 0) {
      device = t.get_device();
      if (device != c10::cuda::current_device())
        refuse(std::string(name) + " is on " + t.device().str() + ", the current device is cuda:" +
               std::to_string(c10::cuda::current_device()));
    } else if (t.get_device() != device) {
      refuse(std::string(name) + " is on " + t.device().str() + ", the other tensors on cuda:" +
             std::to_string(device));
    }
    return t;
  }

  // A contiguous tensor of this shape.
  const at::Tensor& dense(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape,
                          const char* name) {
    const at::Tensor& t = tensor(o, type, name);
    if (!t.is_contiguous()) refuse(std::string(name) + " must be contiguous");
    const at::IntArrayRef want(shape);
    if (t.sizes() != want)
      refuse(std::string(name) + " must be " + shape_text(want) + ", got " + shape_text(t.sizes()));
    return t;
  }
  template <typename T>
  T* address(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape,
             const char* name) {
    return static_cast<T*>(dense(o, type, shape, name).data_ptr());
  }
  template <typename T>
  T* optional(PyObject* o, at::ScalarType type, std::initializer_list<int64_t> shape,
              const char* name) {
    return o == Py_None ? nullptr : address<T>(o, type, shape, name);
  }

  // [tokens, heads, d] bf16 whose rows are contiguous; the stride between tokens.
  void* heads(PyObject* o, int64_t count, int64_t d, const char* name, int64_t* stride,
              int64_t* tokens) {
    const at::Tensor& t = tensor(o, at::kBFloat16, name);
    if (t.dim() != 3 || (count > 0 && t.size(1) != count) || t.size(2) != d)
      refuse(std::string(name) + " must be [tokens, " + (count > 0 ? std::to_string(count) : "heads") +
             ", " + std::to_string(d) + "], got " + shape_text(t.sizes()));
    if (t.size(0) > 0 && (t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != d)))
      refuse(std::string(name) + "'s heads must be contiguous within a token");
    *tokens = t.size(0);
    *stride = t.size(0) > 1 ? t.stride(0) : t.size(1) * d;
    return t.data_ptr();
  }

  at::TensorOptions on(at::ScalarType type) const {
    return at::TensorOptions().dtype(type).device(at::kCUDA, static_cast<c10::DeviceIndex>(device));
  }
  // The caller's status word, or a new zeroed one kept in `keep`.
  int32_t* status(PyObject* o, at::Tensor* keep) {
    if (o == Py_None) {
      *keep = at::zeros({1}, on(at::kInt));
      return static_cast<int32_t*>(keep->data_ptr());
    }
    const at::Tensor& t = tensor(o, at::kInt, "status");
    if (t.numel() < 1) refuse("status must hold one value");
    return static_cast<int32_t*>(t.data_ptr());
  }
  // The caller's output, or a new one.
  at::Tensor output(PyObject* o, std::initializer_list<int64_t> shape, const char* name) {
    return o == Py_None ? at::empty(at::IntArrayRef(shape), on(at::kBFloat16))
                        : dense(o, at::kBFloat16, shape, name);
  }
  at::Tensor workspace(PyObject* o, size_t bytes) {
    if (o == Py_None)
      return at::empty({static_cast<int64_t>(bytes < 256 ? 256 : bytes)}, on(at::kByte));
    const at::Tensor& t = tensor(o, at::kByte, "workspace");
    if (!t.is_contiguous()) refuse("workspace must be contiguous");
    return t;                                  // its size is checked by the call
  }
  cudaStream_t stream() const {
    return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  }
};

int64_t integer(PyObject* o, const char* name) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw python_error();
  if (x < INT32_MIN || x > INT32_MAX) refuse(std::string(name) + " is out of range");
  return x;
}

// block_table, ctx_len, num_blocks, num_kv_heads, head_dim, page_size at args[0 .. 5].
kara_pool pool_of(Call& c, PyObject* const* args) {
  const at::Tensor& table = c.tensor(args[0], at::kInt, "block_table");
  if (table.dim() != 2 || !table.is_contiguous()) refuse("block_table must be contiguous, [B, blocks]");
  kara_pool p = {};
  p.block_table = static_cast<int32_t*>(table.data_ptr());
  p.batch = static_cast<int32_t>(table.size(0));
  p.max_blocks_per_seq = static_cast<int32_t>(table.size(1));
  p.ctx_len = c.address<int32_t>(args[1], at::kInt, {table.size(0)}, "ctx_len");
  p.num_blocks = static_cast<int32_t>(integer(args[2], "num_blocks"));
  p.num_kv_heads = static_cast<int32_t>(integer(args[3], "num_kv_heads"));
  p.head_dim = static_cast<int32_t>(integer(args[4], "head_dim"));
  p.page_size = static_cast<int32_t>(integer(args[5], "page_size"));
  return p;
}
constexpr int kPoolArgs = 6;

void* cache_of(Call& c, PyObject* o, const kara_pool& p, const char* name) {
  return c.address<void>(o, at::kBFloat16, {p.num_blocks, p.page_size, p.num_kv_heads, p.head_dim},
                         name);
}
void* queries_of(Call& c, PyObject* o, const kara_pool& p, int64_t* heads) {
  const at::Tensor& t = c.tensor(o, at::kBFloat16, "q");
  *heads = t.dim() == 3 ? t.size(1) : 0;
  return c.address<void>(o, at::kBFloat16, {p.batch, *heads, p.head_dim}, "q");
}
float scale_of(PyObject* o, const kara_pool& p) {
  if (o == Py_None) return static_cast<float>(1.0 / std::sqrt(static_cast<double>(p.head_dim)));
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return static_cast<float>(x);
}

PyObject* result(kara_status code, const at::Tensor& out) {
  return code == KARA_OK ? THPVariable_Wrap(out) : PyLong_FromLong(code);
}

void expect(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) refuse("wrong number of arguments");
  if (g_lib.rope_append == nullptr) refuse("the library is not bound");
}

// q, k, v, k_cache, v_cache, pool (6), inv_freq, positions, cu_tokens, interleaved, bounds,
// q_ring, window, q_out, k_out, status
PyObject* rope_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 21);
  Call c;
  int64_t heads_q = 0;
  if (THPVariable_Check(a[0]) && THPVariable_Unpack(a[0]).dim() == 3)
    heads_q = THPVariable_Unpack(a[0]).size(1);
  c.tensor(a[0], at::kBFloat16, "q");
  const kara_pool p = pool_of(c, a + 5);
  void* kc = cache_of(c, a[3], p, "k_cache");
  void* vc = cache_of(c, a[4], p, "v_cache");
  int64_t qs, ks, vs, tq, tk, tv;
  void* q = c.heads(a[0], 0, p.head_dim, "q", &qs, &tq);
  void* k = c.heads(a[1], p.num_kv_heads, p.head_dim, "k", &ks, &tk);
  void* v = c.heads(a[2], p.num_kv_heads, p.head_dim, "v", &vs, &tv);
  if (tk != tq || tv != tq) refuse("q, k and v must hold the same tokens");
  PyObject* const* b = a + 5 + kPoolArgs;
  const at::Tensor& freq = c.tensor(b[0], at::kFloat, "inv_freq");
  if (freq.dim() != 1 || !freq.is_contiguous()) refuse("inv_freq must be contiguous, [rotary_dim / 2]");
  const int32_t* pos = c.address<int32_t>(b[1], at::kInt, {tq}, "positions");
  const int32_t* cu = c.optional<int32_t>(b[2], at::kInt, {p.batch + 1}, "cu_tokens");
  if (cu == nullptr && tq != p.batch) refuse("without cu_tokens there must be one token per sequence");
  const int interleaved = PyObject_IsTrue(b[3]);
  if (interleaved < 0) throw python_error();
  void* bounds = c.optional<void>(b[4], at::kBFloat16,
                                  {p.num_blocks, p.num_kv_heads, 2, p.head_dim}, "bounds");
  const int64_t window = integer(b[6], "window");
  void* ring = c.optional<void>(b[5], at::kBFloat16, {p.batch, 2 * window, heads_q, p.head_dim},
                                "q_ring");
  at::Tensor out = c.output(b[7], {tq, heads_q, p.head_dim}, "q_out");
  void* k_out = c.optional<void>(b[8], at::kBFloat16, {tq, p.num_kv_heads, p.head_dim}, "k_out");
  at::Tensor keep;
  int32_t* st = c.status(b[9], &keep);
  return result(
      g_lib.rope_append(q, k, v, qs, ks, vs, static_cast<int32_t>(tq), cu, pos,
                        static_cast<const float*>(freq.data_ptr()),
                        static_cast<int32_t>(2 * freq.numel()), interleaved, kc, vc, &p,
                        static_cast<int32_t>(heads_q), bounds, ring, static_cast<int32_t>(window),
                        out.data_ptr(), k_out, st, c.stream()),
      out);
  END_HANDLE_TH_ERRORS
}

// k_cache, pool (6), bounds, from_slot, new_slots, status
PyObject* page_bounds(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 11);
  Call c;
  c.tensor(a[0], at::kBFloat16, "k_cache");
  const kara_pool p = pool_of(c, a + 1);
  void* kc = cache_of(c, a[0], p, "k_cache");
  PyObject* const* b = a + 1 + kPoolArgs;
  const int32_t* from = c.optional<int32_t>(b[1], at::kInt, {p.batch}, "from_slot");
  const int64_t new_slots = integer(b[2], "new_slots");
  at::Tensor bounds =
      b[0] == Py_None
          ? at::zeros({p.num_blocks, p.num_kv_heads, 2, p.head_dim}, c.on(at::kBFloat16))
          : c.dense(b[0], at::kBFloat16, {p.num_blocks, p.num_kv_heads, 2, p.head_dim}, "bounds");
  at::Tensor keep;
  int32_t* st = c.status(b[3], &keep);
  return result(g_lib.page_bounds(kc, &p, from, static_cast<int32_t>(new_slots), bounds.data_ptr(),
                                  st, c.stream()),
                bounds);
  END_HANDLE_TH_ERRORS
}

// q, k_cache, v_cache, bounds, pool (6), num_pages, sink_pages, recent_pages, new_slots, scale,
// sel, out, workspace, status
PyObject* sparse_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 19);
  Call c;
  c.tensor(a[0], at::kBFloat16, "q");
  const kara_pool p = pool_of(c, a + 4);
  int64_t heads;
  void* q = queries_of(c, a[0], p, &heads);
  void* kc = cache_of(c, a[1], p, "k_cache");
  void* vc = cache_of(c, a[2], p, "v_cache");
  void* bounds = c.address<void>(a[3], at::kBFloat16,
                                 {p.num_blocks, p.num_kv_heads, 2, p.head_dim}, "bounds");
  PyObject* const* b = a + 4 + kPoolArgs;
  const int32_t pages = static_cast<int32_t>(integer(b[0], "num_pages"));
  const int32_t sink = static_cast<int32_t>(integer(b[1], "sink_pages"));
  const int32_t recent = static_cast<int32_t>(integer(b[2], "recent_pages"));
  const int32_t new_slots = static_cast<int32_t>(integer(b[3], "new_slots"));
  const float scale = scale_of(b[4], p);
  int32_t* sel = c.optional<int32_t>(b[5], at::kInt, {p.batch, p.num_kv_heads, pages}, "sel");
  at::Tensor out = c.output(b[6], {p.batch, heads, p.head_dim}, "out");
  at::Tensor ws = c.workspace(
      b[7], b[7] != Py_None ? 0
                            : g_lib.workspace_bytes(KARA_OP_SPARSE, &p, 0, 0,
                                                    static_cast<int32_t>(heads), pages));
  at::Tensor keep;
  int32_t* st = c.status(b[8], &keep);
  return result(g_lib.sparse_attn(q, kc, vc, bounds, &p, static_cast<int32_t>(heads), scale, pages,
                                  sink, recent, new_slots, sel, out.data_ptr(), ws.data_ptr(),
                                  static_cast<size_t>(ws.numel()), st, c.stream()),
                out);
  END_HANDLE_TH_ERRORS
}

// q, k_cache, v_cache, pool (6), group_ptr, prefix_pages, group_rows, new_slots, scale, out,
// workspace, status
PyObject* prefix_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  expect(n, 17);
  Call c;
  c.tensor(a[0], at::kBFloat16, "q");
  const kara_pool p = pool_of(c, a + 3);
  int64_t heads;
  void* q = queries_of(c, a[0], p, &heads);
  void* kc = cache_of(c, a[1], p, "k_cache");
  void* vc = cache_of(c, a[2], p, "v_cache");
  PyObject* const* b = a + 3 + kPoolArgs;
  const at::Tensor& pages = c.tensor(b[1], at::kInt, "prefix_pages");
  if (pages.dim() != 1 || !pages.is_contiguous()) refuse("prefix_pages must be contiguous, [groups]");
  const int64_t groups = pages.numel();
  const int32_t* ptr = c.address<int32_t>(b[0], at::kInt, {groups + 1}, "group_ptr");
  const int32_t* rows = c.optional<int32_t>(b[2], at::kInt, {p.batch}, "group_rows");
  const int32_t new_slots = static_cast<int32_t>(integer(b[3], "new_slots"));
  const float scale = scale_of(b[4], p);
  at::Tensor out = c.output(b[5], {p.batch, heads, p.head_dim}, "out");
  at::Tensor ws = c.workspace(
      b[6], b[6] != Py_None ? 0
                            : g_lib.workspace_bytes(KARA_OP_PREFIX, &p, 0, 0,
                                                    static_cast<int32_t>(heads), 0));
  at::Tensor keep;
  int32_t* st = c.status(b[7], &keep);
  return result(g_lib.prefix_attn(q, kc, vc, &p, static_cast<int32_t>(heads), scale, ptr,
                                  static_cast<const int32_t*>(pages.data_ptr()),
                                  static_cast<int32_t>(groups), rows, new_slots, out.data_ptr(),
                                  ws.data_ptr(), static_cast<size_t>(ws.numel()), st, c.stream()),
                out);
  END_HANDLE_TH_ERRORS
}

// The library's path: resolves the entry points (the copy that is already loaded).
PyObject* bind(PyObject*, PyObject* path) {
  const char* text = PyUnicode_AsUTF8(path);
  if (text == nullptr) return nullptr;
  void* handle = dlopen(text, RTLD_NOW | RTLD_LOCAL);
  if (handle == nullptr) {
    PyErr_SetString(PyExc_ImportError, dlerror());
    return nullptr;
  }
  auto find = [&](auto& fn, const char* name) {
    fn = reinterpret_cast<std::decay_t<decltype(fn)>>(dlsym(handle, name));
    return fn != nullptr;
  };
  Library lib;
  if (!find(lib.rope_append, "paged_rope_append") || !find(lib.page_bounds, "paged_page_bounds") ||
      !find(lib.sparse_attn, "paged_sparse_attn") || !find(lib.prefix_attn, "paged_prefix_attn") ||
      !find(lib.workspace_bytes, "kara_workspace_bytes")) {
    PyErr_SetString(PyExc_ImportError, "the library lacks an entry point");
    return nullptr;
  }
  g_lib = lib;
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction as_method(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef g_methods[] = {
    {"bind", bind, METH_O, nullptr},
    {"rope_append", as_method(rope_append), METH_FASTCALL, nullptr},
    {"page_bounds", as_method(page_bounds), METH_FASTCALL, nullptr},
    {"sparse_attn", as_method(sparse_attn), METH_FASTCALL, nullptr},
    {"prefix_attn", as_method(prefix_attn), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&g_module); }
