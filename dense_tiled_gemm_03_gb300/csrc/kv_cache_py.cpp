// kv_cache_py.cpp -- the Python binding of the paged key/value cache
// (include/kv_cache.h): KVCache, tree_attn, cache_append, cache_weigh and
// cache_evict as an extension module over torch's tensors.
//
// Argument marshalling only. It is compiled code because these calls are small
// and many (a decode step makes several per layer) and each hands over some ten
// tensors with their sizes and strides: read one attribute at a time from
// Python, that took 6 to 8 us of calls whose kernels run for 3 to 10.
// Measured on a GB300's Arm cores, from Python and here, the cache's description
// included: tree_attn 10.6 and 4.1 us, cache_append 10.7 and 3.6, cache_weigh
// 10.7 and 3.6, cache_evict 8.5 and 3.5 (2 to 2.5 of them the launch).
//
// bind() hands over the C functions' addresses, so that the one loaded
// libgemm_tn.so is called, and the exception type of its errors.
#include <Python.h>
#include <structmember.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <string>

#include "kv_cache.h"

namespace {

using at::Tensor;

decltype(&tree_attn_fwd) g_attn = nullptr;
decltype(&kv_cache_append) g_append = nullptr;
decltype(&kv_cache_weigh) g_weigh = nullptr;
decltype(&kv_cache_evict) g_evict = nullptr;
PyObject* g_error = nullptr;   // GemmTnError(status, where)

// ---------------------------------------------------------------- arguments

// Places positional and keyword arguments (a vectorcall's) in `out`, None as
// nullptr; the first `required` must be there.
template <int kCount>
bool place(const char* fn, const char* const (&names)[kCount], int required, PyObject* const* args, Py_ssize_t positional,
           PyObject* kwnames, PyObject* (&out)[kCount]) {
  for (PyObject*& o : out) o = nullptr;
  if (positional > kCount) {
    PyErr_Format(PyExc_TypeError, "%s() takes at most %d arguments (%zd given)", fn, kCount, positional);
    return false;
  }
  bool given[kCount] = {};
  for (Py_ssize_t i = 0; i < positional; ++i) {
    given[i] = true;
    out[i] = args[i] == Py_None ? nullptr : args[i];
  }
  const Py_ssize_t keywords = kwnames != nullptr ? PyTuple_GET_SIZE(kwnames) : 0;
  for (Py_ssize_t x = 0; x < keywords; ++x) {
    Py_ssize_t size = 0;
    const char* name = PyUnicode_AsUTF8AndSize(PyTuple_GET_ITEM(kwnames, x), &size);
    if (name == nullptr) return false;
    int i = 0;
    while (i < kCount && std::strcmp(names[i], name) != 0) ++i;
    if (i == kCount) {
      PyErr_Format(PyExc_TypeError, "%s() got an unexpected keyword argument '%s'", fn, name);
      return false;
    }
    if (given[i]) {
      PyErr_Format(PyExc_TypeError, "%s() got multiple values for argument '%s'", fn, name);
      return false;
    }
    given[i] = true;
    PyObject* value = args[positional + x];
    out[i] = value == Py_None ? nullptr : value;
  }
  for (int i = 0; i < required; ++i)
    if (!given[i]) {
      PyErr_Format(PyExc_TypeError, "%s() missing required argument '%s'", fn, names[i]);
      return false;
    }
  return true;
}

const Tensor* tensor(PyObject* o, const char* what) {
  if (o != nullptr && THPVariable_Check(o)) return &THPVariable_Unpack(o);
  PyErr_Format(PyExc_TypeError, "%s must be a tensor", what);
  return nullptr;
}

int64_t cuda_index(const Tensor& t) { return t.is_cuda() ? t.get_device() : -1; }

std::string shape_text(at::IntArrayRef shape) {
  std::string s = "(";
  for (size_t i = 0; i < shape.size(); ++i) s += (i > 0 ? ", " : "") + std::to_string(shape[i]);
  return s + (shape.size() == 1 ? ",)" : ")");
}

// ---------------------------------------------------------------- KVCache

// What seven tensors make up, as they are when it is read: a tensor may be given
// other storage later (set_, resize_, an assignment to .data), so every call
// describes the tensors anew.
struct Description {
  long long batch, capacity, index, kv_heads, head_dim;
  int code;
  at::ScalarType type;
  kv_cache c;
  PyObject *lens, *weight, *pos, *seen;   // borrowed; nullptr where there is none
};

struct Cache {
  PyObject_HEAD
  PyObject *k, *v, *page_table, *lens, *weight, *pos, *seen;   // None where there is none
  PyObject* dtype;
  Description made;   // as it was made; its pointers are not used again
};

// Whether the tensor's storage holds it (it may have been made smaller, or been freed).
bool stored(const Tensor& t, const char* what) {
  if (t.numel() == 0) return true;
  int64_t extent = 1;
  for (int64_t i = 0; i < t.dim(); ++i) extent += (t.size(i) - 1) * t.stride(i);
  const uint64_t bytes = static_cast<uint64_t>(t.storage_offset() + extent) * t.element_size();
  if (t.storage().nbytes() >= bytes) return true;
  PyErr_Format(PyExc_ValueError, "the storage of %s is smaller than the tensor", what);
  return false;
}

// The pointer of a contiguous tensor of 32-bit numbers of that shape, nullptr for no tensor; false with an exception set.
bool numbers(PyObject* o, at::ScalarType type, int64_t index, const char* what, at::IntArrayRef shape, void** to) {
  *to = nullptr;
  if (o == nullptr) return true;
  const Tensor* t = tensor(o, what);
  if (t == nullptr) return false;
  if (cuda_index(*t) != index || t->scalar_type() != type || t->sizes() != shape || !t->is_contiguous()) {
    PyErr_Format(PyExc_ValueError, "%s must be a contiguous %s %s tensor on the cache's device", what,
                 type == at::kInt ? "int32" : "float32", shape_text(shape).c_str());
    return false;
  }
  *to = t->data_ptr();
  return stored(*t, what);
}
bool ints(PyObject* o, const Description* c, const char* what, at::IntArrayRef shape, int32_t** to) {
  void* p = nullptr;
  const bool ok = numbers(o, at::kInt, c->index, what, shape, &p);
  *to = static_cast<int32_t*>(p);
  return ok;
}
bool floats(PyObject* o, const Description* c, const char* what, at::IntArrayRef shape, float** to) {
  void* p = nullptr;
  const bool ok = numbers(o, at::kFloat, c->index, what, shape, &p);
  *to = static_cast<float*>(p);
  return ok;
}

bool status_word(PyObject* o, const Description* c, int** to) {
  *to = nullptr;
  if (o == nullptr) return true;
  const Tensor* t = tensor(o, "status");
  if (t == nullptr) return false;
  if (cuda_index(*t) != c->index || t->scalar_type() != at::kInt || t->numel() < 1 || !t->is_contiguous()) {
    PyErr_SetString(PyExc_ValueError, "status must be a contiguous int32 tensor of at least one element on the cache's device");
    return false;
  }
  *to = static_cast<int*>(t->data_ptr());
  return true;
}

// A [batch, tokens, heads, head_dim] tensor of that shape.
bool rows_of(PyObject* o, const Description* c, const char* what, at::IntArrayRef shape, kv_rows* to) {
  const Tensor* t = tensor(o, what);
  if (t == nullptr) return false;
  if (cuda_index(*t) != c->index) {
    PyErr_Format(PyExc_ValueError, "%s must be on the cache's device", what);
    return false;
  }
  if (t->scalar_type() != c->type) {
    PyErr_Format(PyExc_TypeError, "%s must have the cache's dtype", what);
    return false;
  }
  if (t->sizes() != shape) {
    PyErr_Format(PyExc_ValueError, "%s must be [batch, tokens, heads, head_dim] = %s", what, shape_text(shape).c_str());
    return false;
  }
  const at::IntArrayRef s = t->strides();
  if (s[3] != 1) {
    PyErr_Format(PyExc_ValueError, "%s must have unit stride along head_dim", what);
    return false;
  }
  *to = {t->data_ptr(), s[0], s[1], s[2]};
  return true;
}

int cache_traverse(PyObject* self, visitproc visit, void* arg) {
  Cache* c = reinterpret_cast<Cache*>(self);
  for (PyObject* o : {c->k, c->v, c->page_table, c->lens, c->weight, c->pos, c->seen, c->dtype}) Py_VISIT(o);
  return 0;
}
int cache_clear(PyObject* self) {
  Cache* c = reinterpret_cast<Cache*>(self);
  for (PyObject** o : {&c->k, &c->v, &c->page_table, &c->lens, &c->weight, &c->pos, &c->seen, &c->dtype}) Py_CLEAR(*o);
  return 0;
}
void cache_dealloc(PyObject* self) {
  PyObject_GC_UnTrack(self);
  cache_clear(self);
  Py_TYPE(self)->tp_free(self);
}

PyMemberDef cache_members[] = {
    {"k", T_OBJECT, offsetof(Cache, k), READONLY, nullptr},
    {"v", T_OBJECT, offsetof(Cache, v), READONLY, nullptr},
    {"page_table", T_OBJECT, offsetof(Cache, page_table), READONLY, nullptr},
    {"lens", T_OBJECT, offsetof(Cache, lens), READONLY, nullptr},
    {"weight", T_OBJECT, offsetof(Cache, weight), READONLY, nullptr},
    {"pos", T_OBJECT, offsetof(Cache, pos), READONLY, nullptr},
    {"seen", T_OBJECT, offsetof(Cache, seen), READONLY, nullptr},
    {"dtype", T_OBJECT, offsetof(Cache, dtype), READONLY, nullptr},
    {"batch", T_LONGLONG, offsetof(Cache, made.batch), READONLY, nullptr},
    {"capacity", T_LONGLONG, offsetof(Cache, made.capacity), READONLY, "max_pages * page_size"},
    {"index", T_LONGLONG, offsetof(Cache, made.index), READONLY, "the device's"},
    {"kv_heads", T_LONGLONG, offsetof(Cache, made.kv_heads), READONLY, nullptr},
    {"head_dim", T_LONGLONG, offsetof(Cache, made.head_dim), READONLY, nullptr},
    {nullptr, 0, 0, 0, nullptr},
};

PyObject* cache_new(PyObject* type, PyObject* const* args, size_t nargsf, PyObject* kwnames);

PyTypeObject* cache_type() {
  static PyTypeObject type = [] {
    PyTypeObject t = {PyVarObject_HEAD_INIT(nullptr, 0)};
    t.tp_name = "dense_tiled_gemm_03_gb300.KVCache";
    t.tp_basicsize = sizeof(Cache);
    t.tp_flags = Py_TPFLAGS_DEFAULT | Py_TPFLAGS_HAVE_GC;
    t.tp_doc =
        "KVCache(k, v, page_table, lens, weight=None, pos=None, seen=None)\n--\n\n"
        "A paged key/value cache in the caller's tensors (nothing is copied; the\n"
        "tensors are kept alive, and each call finds their storage where it then\n"
        "is; tensors whose sizes, strides or types have changed are refused).\n\n"
        "k, v: [num_pages, page_size, kv_heads, head_dim] CUDA fp16/bf16 views with\n"
        "unit stride along head_dim and the same strides; permute a\n"
        "[num_pages, kv_heads, page_size, head_dim] pool into this order. page_size 8,\n"
        "16, 32, 64 or a multiple of 128; head_dim 64 or 128. page_table: int32\n"
        "[batch, max_pages]; lens: int32 [batch], slots in use. Where an operator\n"
        "needs them: weight, fp32 [batch, kv_heads, capacity], the accumulated\n"
        "attention weight of each slot; pos, int32 of that shape, the position of\n"
        "the token in it; seen, int32 [batch], the next token's position\n"
        "(capacity = max_pages * page_size).";
    t.tp_traverse = cache_traverse;
    t.tp_clear = cache_clear;
    t.tp_dealloc = cache_dealloc;
    t.tp_members = cache_members;
    t.tp_vectorcall = cache_new;
    return t;
  }();
  return &type;
}

// Describes the cache of k, v, page_table, lens, weight, pos and seen (nullptr for
// the last three: none); false with an exception set.
bool describe(PyObject* const (&in)[7], Description* to) {
  const Tensor *k = tensor(in[0], "k"), *v = k != nullptr ? tensor(in[1], "v") : nullptr;
  const Tensor* table = v != nullptr ? tensor(in[2], "page_table") : nullptr;
  const Tensor* lens = table != nullptr ? tensor(in[3], "lens") : nullptr;
  if (lens == nullptr) return false;
  auto refuse = [](PyObject* kind, const char* what) {
    PyErr_SetString(kind, what);
    return false;
  };
  const int64_t index = cuda_index(*k);
  if (index < 0 || cuda_index(*v) != index || cuda_index(*table) != index || cuda_index(*lens) != index)
    return refuse(PyExc_ValueError, "the cache's tensors must be CUDA tensors on one device");
  const at::ScalarType dtype = k->scalar_type();
  if (v->scalar_type() != dtype) return refuse(PyExc_TypeError, "k and v must have the same dtype");
  if (dtype != at::kHalf && dtype != at::kBFloat16)
    return refuse(PyExc_TypeError, "unsupported dtype of k and v: expected float16 or bfloat16");
  const at::IntArrayRef shape = k->sizes(), strides = k->strides();
  if (shape.size() != 4 || v->sizes() != shape || v->strides() != strides)
    return refuse(PyExc_ValueError, "k and v must be [num_pages, page_size, kv_heads, head_dim] with the same strides");
  if (strides[3] != 1) return refuse(PyExc_ValueError, "k and v must have unit stride along head_dim");
  if (table->scalar_type() != at::kInt || lens->scalar_type() != at::kInt)
    return refuse(PyExc_TypeError, "page_table and lens must be int32");
  if (table->dim() != 2) return refuse(PyExc_ValueError, "page_table must be [batch, max_pages]");
  const int64_t batch = table->size(0), max_pages = table->size(1), heads = shape[2], dim = shape[3];
  if (table->stride(1) != 1 && max_pages > 1)
    return refuse(PyExc_ValueError, "page_table must have unit stride along max_pages");
  if (lens->dim() != 1 || lens->size(0) != batch || !lens->is_contiguous())
    return refuse(PyExc_ValueError, "lens must be a contiguous [batch] tensor");
  const int64_t capacity = max_pages * shape[1];
  void *weight = nullptr, *pos = nullptr, *seen = nullptr;
  if (!stored(*k, "k") || !stored(*v, "v") || !stored(*table, "page_table") || !stored(*lens, "lens") ||
      !numbers(in[4], at::kFloat, index, "weight", {batch, heads, capacity}, &weight) ||
      !numbers(in[5], at::kInt, index, "pos", {batch, heads, capacity}, &pos) ||
      !numbers(in[6], at::kInt, index, "seen", {batch}, &seen))
    return false;
  to->lens = in[3];
  to->weight = in[4];
  to->pos = in[5];
  to->seen = in[6];
  to->batch = batch;
  to->capacity = capacity;
  to->index = index;
  to->kv_heads = heads;
  to->head_dim = dim;
  to->code = dtype == at::kHalf ? GEMM_TN_F16 : GEMM_TN_BF16;
  to->type = dtype;
  to->c = kv_cache{};
  to->c.k = k->data_ptr();
  to->c.v = v->data_ptr();
  to->c.num_pages = shape[0];
  to->c.page_size = shape[1];
  to->c.kv_heads = heads;
  to->c.head_dim = dim;
  to->c.page_stride = strides[0];
  to->c.slot_stride = strides[1];
  to->c.head_stride = heads > 1 ? strides[2] : dim;
  to->c.page_table = static_cast<const int32_t*>(table->data_ptr());
  to->c.table_stride = batch > 1 ? table->stride(0) : max_pages;
  to->c.max_pages = max_pages;
  to->c.lens = static_cast<int32_t*>(lens->data_ptr());
  to->c.weight = static_cast<float*>(weight);
  to->c.pos = static_cast<int32_t*>(pos);
  to->c.seen = static_cast<int32_t*>(seen);
  return true;
}

PyObject* cache_new(PyObject* type, PyObject* const* args, size_t nargsf, PyObject* kwnames) {
  HANDLE_TH_ERRORS
  static const char* const names[] = {"k", "v", "page_table", "lens", "weight", "pos", "seen"};
  PyObject* in[7];
  Description made;
  if (!place("KVCache", names, 4, args, PyVectorcall_NARGS(nargsf), kwnames, in) || !describe(in, &made)) return nullptr;
  PyObject* torch_type = PyObject_GetAttrString(in[0], "dtype");
  if (torch_type == nullptr) return nullptr;
  Cache* c = PyObject_GC_New(Cache, reinterpret_cast<PyTypeObject*>(type));
  if (c == nullptr) {
    Py_DECREF(torch_type);
    return nullptr;
  }
  PyObject** to[] = {&c->k, &c->v, &c->page_table, &c->lens, &c->weight, &c->pos, &c->seen};
  for (int i = 0; i < 7; ++i) {
    *to[i] = in[i] != nullptr ? in[i] : Py_None;
    Py_INCREF(*to[i]);
  }
  c->dtype = torch_type;
  c->made = made;
  PyObject_GC_Track(reinterpret_cast<PyObject*>(c));
  return reinterpret_cast<PyObject*>(c);
  END_HANDLE_TH_ERRORS
}

// The cache's tensors as they are now, in *now.
const Description* cache_of(PyObject* o, Description* now) {
  if (o == nullptr || Py_TYPE(o) != cache_type()) {
    PyErr_SetString(PyExc_TypeError, "cache must be a KVCache");
    return nullptr;
  }
  const Cache* c = reinterpret_cast<const Cache*>(o);
  auto held = [](PyObject* x) { return x != Py_None ? x : nullptr; };
  PyObject* const in[7] = {c->k, c->v, c->page_table, c->lens, held(c->weight), held(c->pos), held(c->seen)};
  if (!describe(in, now)) return nullptr;
  const kv_cache &x = now->c, &y = c->made.c;
  if (now->batch == c->made.batch && now->index == c->made.index && now->type == c->made.type && x.num_pages == y.num_pages &&
      x.page_size == y.page_size && x.kv_heads == y.kv_heads && x.head_dim == y.head_dim && x.max_pages == y.max_pages &&
      x.page_stride == y.page_stride && x.slot_stride == y.slot_stride && x.head_stride == y.head_stride &&
      x.table_stride == y.table_stride)
    return now;
  PyErr_SetString(PyExc_ValueError, "the cache's tensors have changed their sizes, strides or types since it was made");
  return nullptr;
}

// ---------------------------------------------------------------- calls

// One call of the library on the cache's device and its current stream; false
// with GemmTnError set. The call itself throws nothing.
template <class Call>
bool run(const Description* c, const char* name, Call call) {
  int rc;
  {
    const c10::cuda::CUDAGuard device(static_cast<c10::DeviceIndex>(c->index));
    cudaStream_t stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(c->index)).stream();
    Py_BEGIN_ALLOW_THREADS
    rc = call(reinterpret_cast<gemm_tn_stream_t>(stream));
    Py_END_ALLOW_THREADS
  }
  if (rc == GEMM_TN_OK) return true;
  PyObject* error = PyObject_CallFunction(g_error, "is", rc, name);
  if (error != nullptr) {
    PyErr_SetObject(g_error, error);
    Py_DECREF(error);
  }
  return false;
}

// The factor on q.k; 0 (the C ABI's word for the default) for None.
bool factor(PyObject* o, float* to) {
  *to = 0.0f;
  if (o == nullptr) return true;
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) return false;
  *to = static_cast<float>(x);
  if (*to == 0.0f) {
    PyErr_SetString(PyExc_ValueError, "scale must be positive");
    return false;
  }
  return true;
}

bool queries(PyObject* o, const Description* c, at::IntArrayRef* shape, kv_rows* to) {
  const Tensor* q = tensor(o, "q");
  if (q == nullptr) return false;
  *shape = q->sizes();
  if (shape->size() != 4 || (*shape)[0] != c->batch || (*shape)[3] != c->head_dim) {
    PyErr_SetString(PyExc_ValueError,
                    "q must be [batch, tokens, heads, head_dim] with the cache's batch size and head_dim");
    return false;
  }
  return rows_of(o, c, "q", *shape, to);
}

// rows and counts; max_rows is rows' width, `tokens` without rows.
bool counted(const Description* c, PyObject* rows, PyObject* counts, int64_t tokens, int32_t** d_rows, int32_t** d_counts,
             int64_t* max_rows) {
  *max_rows = tokens;
  if (rows != nullptr) {
    const Tensor* t = tensor(rows, "rows");
    if (t == nullptr) return false;
    if (t->dim() != 2) {
      PyErr_SetString(PyExc_ValueError, "rows must be [batch, max_rows]");
      return false;
    }
    *max_rows = t->size(1);
  }
  return ints(rows, c, "rows", {c->batch, *max_rows}, d_rows) && ints(counts, c, "counts", {c->batch}, d_counts);
}

PyObject* or_own(PyObject* out, PyObject* own) { return out != nullptr ? out : own; }

PyObject* tree_attn(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  HANDLE_TH_ERRORS
  static const char* const names[] = {"q", "cache", "k_new", "v_new", "mask", "token_lens", "scale", "out", "lse", "status"};
  PyObject* in[10];
  if (!place("tree_attn", names, 2, args, nargs, kwnames, in)) return nullptr;
  Description now;
  const Description* c = cache_of(in[1], &now);
  at::IntArrayRef shape;
  kv_rows q, k_new, v_new;
  if (c == nullptr || !queries(in[0], c, &shape, &q)) return nullptr;
  const int64_t batch = shape[0], tokens = shape[1], heads = shape[2];
  if ((in[2] == nullptr) != (in[3] == nullptr)) {
    PyErr_SetString(PyExc_ValueError, "k_new and v_new come together");
    return nullptr;
  }
  const bool has_new = in[2] != nullptr;
  if (has_new) {
    const int64_t new_shape[] = {batch, tokens, c->kv_heads, c->head_dim};
    if (!rows_of(in[2], c, "k_new", new_shape, &k_new) || !rows_of(in[3], c, "v_new", new_shape, &v_new)) return nullptr;
  }
  const uint64_t* mask = nullptr;
  if (in[4] != nullptr) {
    const Tensor* t = tensor(in[4], "mask");
    if (t == nullptr) return nullptr;
    const int64_t mask_shape[] = {batch, tokens, (tokens + 63) / 64};
    if (cuda_index(*t) != c->index || t->scalar_type() != at::kLong || t->sizes() != at::IntArrayRef(mask_shape) ||
        !t->is_contiguous()) {
      PyErr_SetString(PyExc_ValueError,
                      "mask must be a contiguous int64 [batch, tokens, ceil(tokens / 64)] tensor on the cache's device");
      return nullptr;
    }
    mask = static_cast<const uint64_t*>(t->data_ptr());
  }
  int32_t* token_lens;
  float *lse, scale;
  int* status;
  if (!ints(in[5], c, "token_lens", {batch}, &token_lens) || !factor(in[6], &scale) ||
      !floats(in[8], c, "lse", {batch, tokens, heads}, &lse) || !status_word(in[9], c, &status))
    return nullptr;
  Tensor made;
  const Tensor* out = &made;
  if (in[7] == nullptr) {
    const at::TensorOptions options = THPVariable_Unpack(in[0]).options();
    made = token_lens == nullptr ? at::empty(shape, options) : at::zeros(shape, options);
  } else {
    out = tensor(in[7], "out");
    if (out == nullptr) return nullptr;
    if (out->sizes() != shape || out->scalar_type() != c->type || cuda_index(*out) != c->index || !out->is_contiguous()) {
      PyErr_SetString(PyExc_ValueError, "out must be a contiguous tensor with q's shape, dtype and device");
      return nullptr;
    }
  }
  void* o = out->data_ptr();
  if (!run(c, "tree_attn_fwd", [&](gemm_tn_stream_t stream) {
        return g_attn(c->code, batch, tokens, heads, &c->c, &q, has_new ? &k_new : nullptr, has_new ? &v_new : nullptr, mask,
                      token_lens, o, lse, scale, status, stream);
      }))
    return nullptr;
  if (in[7] == nullptr) return THPVariable_Wrap(made);
  Py_INCREF(in[7]);
  return in[7];
  END_HANDLE_TH_ERRORS
}

PyObject* cache_append(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  HANDLE_TH_ERRORS
  static const char* const names[] = {"cache", "k_new", "v_new", "counts", "rows", "lens_out", "seen_out", "status"};
  PyObject* in[8];
  if (!place("cache_append", names, 3, args, nargs, kwnames, in)) return nullptr;
  Description now;
  const Description* c = cache_of(in[0], &now);
  const Tensor* t = c != nullptr ? tensor(in[1], "k_new") : nullptr;
  if (t == nullptr) return nullptr;
  const at::IntArrayRef shape = t->sizes();
  if (shape.size() != 4 || shape[0] != c->batch || shape[2] != c->kv_heads || shape[3] != c->head_dim) {
    PyErr_SetString(PyExc_ValueError, "k_new must be [batch, tokens, kv_heads, head_dim] with the cache's sizes");
    return nullptr;
  }
  if (in[6] != nullptr && c->seen == nullptr) {
    PyErr_SetString(PyExc_ValueError, "seen_out needs a cache with seen");
    return nullptr;
  }
  kv_rows k_new, v_new;
  int32_t *rows, *counts, *lens_out, *seen_out;
  int64_t max_rows;
  int* status;
  if (!rows_of(in[1], c, "k_new", shape, &k_new) || !rows_of(in[2], c, "v_new", shape, &v_new) ||
      !counted(c, in[4], in[3], shape[1], &rows, &counts, &max_rows) ||
      !ints(or_own(in[5], c->lens), c, "lens_out", {c->batch}, &lens_out) ||
      !ints(or_own(in[6], c->seen), c, "seen_out", {c->batch}, &seen_out) || !status_word(in[7], c, &status))
    return nullptr;
  if (!run(c, "kv_cache_append", [&](gemm_tn_stream_t stream) {
        return g_append(c->code, c->batch, shape[1], &c->c, &k_new, &v_new, rows, counts, max_rows, lens_out, seen_out, status,
                        stream);
      }))
    return nullptr;
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

PyObject* cache_weigh(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  HANDLE_TH_ERRORS
  static const char* const names[] = {"cache", "q", "lse", "counts", "rows", "causal", "scale", "out", "status"};
  PyObject* in[9];
  if (!place("cache_weigh", names, 3, args, nargs, kwnames, in)) return nullptr;
  Description now;
  const Description* c = cache_of(in[0], &now);
  at::IntArrayRef shape;
  kv_rows q;
  if (c == nullptr || !queries(in[1], c, &shape, &q)) return nullptr;
  if (c->weight == nullptr) {
    PyErr_SetString(PyExc_ValueError, "the cache has no weight");
    return nullptr;
  }
  if (tensor(in[2], "lse") == nullptr) return nullptr;
  // None would be no argument: causal is True unless something false is given
  bool given = nargs > 5;
  for (Py_ssize_t x = 0; kwnames != nullptr && x < PyTuple_GET_SIZE(kwnames); ++x)
    given = given || PyUnicode_CompareWithASCIIString(PyTuple_GET_ITEM(kwnames, x), "causal") == 0;
  const int causal = !given ? 1 : (in[5] != nullptr ? PyObject_IsTrue(in[5]) : 0);
  if (causal < 0) return nullptr;
  PyObject* result = or_own(in[7], c->weight);
  float *lse, *out, scale;
  int32_t *rows, *counts;
  int64_t max_rows;
  int* status;
  if (!floats(in[2], c, "lse", {shape[0], shape[1], shape[2]}, &lse) ||
      !counted(c, in[4], in[3], shape[1], &rows, &counts, &max_rows) || !factor(in[6], &scale) ||
      !floats(result, c, "out", {c->batch, c->kv_heads, c->capacity}, &out) || !status_word(in[8], c, &status))
    return nullptr;
  if (!run(c, "kv_cache_weigh", [&](gemm_tn_stream_t stream) {
        return g_weigh(c->code, c->batch, shape[1], shape[2], &c->c, &q, lse, rows, counts, max_rows, causal, scale, out,
                       status, stream);
      }))
    return nullptr;
  Py_INCREF(result);
  return result;
  END_HANDLE_TH_ERRORS
}

PyObject* cache_evict(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  HANDLE_TH_ERRORS
  static const char* const names[] = {"cache", "keep", "recent", "weight_out", "pos_out", "lens_out", "status"};
  PyObject* in[7];
  if (!place("cache_evict", names, 2, args, nargs, kwnames, in)) return nullptr;
  Description now;
  const Description* c = cache_of(in[0], &now);
  if (c == nullptr) return nullptr;
  if (in[1] == nullptr) {
    PyErr_SetString(PyExc_TypeError, "keep must be a whole number");
    return nullptr;
  }
  const long long keep = PyLong_AsLongLong(in[1]);
  if (keep == -1 && PyErr_Occurred()) return nullptr;
  const long long recent = in[2] != nullptr ? PyLong_AsLongLong(in[2]) : 0;
  if (recent == -1 && PyErr_Occurred()) return nullptr;
  if (c->weight == nullptr) {
    PyErr_SetString(PyExc_ValueError, "the cache has no weight");
    return nullptr;
  }
  if (in[4] != nullptr && c->pos == nullptr) {
    PyErr_SetString(PyExc_ValueError, "pos_out needs a cache with pos");
    return nullptr;
  }
  const int64_t shape[] = {c->batch, c->kv_heads, c->capacity};
  float* weight_out;
  int32_t *pos_out, *lens_out;
  int* status;
  if (!floats(or_own(in[3], c->weight), c, "weight_out", shape, &weight_out) ||
      !ints(or_own(in[4], c->pos), c, "pos_out", shape, &pos_out) ||
      !ints(or_own(in[5], c->lens), c, "lens_out", {c->batch}, &lens_out) || !status_word(in[6], c, &status))
    return nullptr;
  if (!run(c, "kv_cache_evict", [&](gemm_tn_stream_t stream) {
        return g_evict(c->code, c->batch, &c->c, keep, recent, weight_out, pos_out, lens_out, status, stream);
      }))
    return nullptr;
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// bind(error, tree_attn_fwd, kv_cache_append, kv_cache_weigh, kv_cache_evict): the exception type and four addresses.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  void* at[4];
  if (nargs != 5) {
    PyErr_SetString(PyExc_TypeError, "bind() takes the exception type and four addresses");
    return nullptr;
  }
  for (int i = 0; i < 4; ++i) {
    at[i] = PyLong_AsVoidPtr(args[1 + i]);
    if (at[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is 0");
      return nullptr;
    }
  }
  Py_INCREF(args[0]);
  Py_XDECREF(g_error);
  g_error = args[0];
  g_attn = reinterpret_cast<decltype(g_attn)>(at[0]);
  g_append = reinterpret_cast<decltype(g_append)>(at[1]);
  g_weigh = reinterpret_cast<decltype(g_weigh)>(at[2]);
  g_evict = reinterpret_cast<decltype(g_evict)>(at[3]);
  Py_RETURN_NONE;
}

template <class F>
PyCFunction as_function(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef functions[] = {
    {"bind", as_function(bind), METH_FASTCALL, nullptr},
    {"tree_attn", as_function(tree_attn), METH_FASTCALL | METH_KEYWORDS,
     "tree_attn(q, cache, k_new=None, v_new=None, mask=None, token_lens=None, scale=None, out=None, lse=None, status=None)\n"
     "--\n\n"
     "Attention of new (drafted) tokens over a paged cache and over one\n"
     "another through tree_attn_fwd. q: [batch, tokens, heads, head_dim], k_new,\n"
     "v_new: [batch, tokens, kv_heads, head_dim] (both None: the cache only),\n"
     "CUDA tensors of the cache's dtype with unit stride along head_dim; heads a\n"
     "multiple of kv_heads. mask: int64 [batch, tokens, ceil(tokens / 64)] words\n"
     "(tree_mask), None for the causal chain; token_lens: int32 [batch], new\n"
     "tokens of each sequence (None: all); scale: the factor on q.k (None:\n"
     "1/sqrt(head_dim)); out: optional contiguous tensor of q's shape and dtype,\n"
     "whose rows from token_lens on are left as they are (without it they come\n"
     "back as zeros); lse: optional contiguous fp32 [batch, tokens, heads] that\n"
     "receives the log of each row's sum of exponentials; status: optional\n"
     "one-element int32 CUDA tensor for device-side errors. Returns out."},
    {"cache_append", as_function(cache_append), METH_FASTCALL | METH_KEYWORDS,
     "cache_append(cache, k_new, v_new, counts=None, rows=None, lens_out=None, seen_out=None, status=None)\n--\n\n"
     "Puts new tokens' keys and values into the cache through kv_cache_append.\n"
     "k_new, v_new: [batch, tokens, kv_heads, head_dim] with unit stride along\n"
     "head_dim. rows: int32 [batch, max_rows], which tokens, in order (None: the\n"
     "first ones); counts: int32 [batch], how many (None: all). weight becomes 0\n"
     "and pos the token's position where the cache has them. lens_out, seen_out:\n"
     "int32 [batch] that receive the new lengths (None: the cache's own lens and\n"
     "seen are advanced)."},
    {"cache_weigh", as_function(cache_weigh), METH_FASTCALL | METH_KEYWORDS,
     "cache_weigh(cache, q, lse, counts=None, rows=None, causal=True, scale=None, out=None, status=None)\n--\n\n"
     "Adds to each cached key's weight the attention that counted queries gave\n"
     "it, through kv_cache_weigh. q: [batch, tokens, heads, head_dim], lse: fp32\n"
     "[batch, tokens, heads] as tree_attn fills it; rows, counts: the counted\n"
     "tokens as in cache_append. causal: the counted tokens are the newest\n"
     "slots' queries and see the slots up to their own; False: every one sees\n"
     "every slot. out: fp32 tensor of weight's shape that receives the sums\n"
     "(None: the cache's weight, in place). Returns out."},
    {"cache_evict", as_function(cache_evict), METH_FASTCALL | METH_KEYWORDS,
     "cache_evict(cache, keep, recent=0, weight_out=None, pos_out=None, lens_out=None, status=None)\n--\n\n"
     "Cuts sequences longer than `keep` slots down to the newest `recent` ones\n"
     "and the heaviest others, for each KV head by its own weights, through\n"
     "kv_cache_evict. weight_out, pos_out, lens_out: tensors like the cache's\n"
     "that receive the results (None: the cache's own, in place)."},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kv_cache", nullptr, -1, functions, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv_cache() {
  if (PyType_Ready(cache_type()) < 0) return nullptr;
  PyObject* m = PyModule_Create(&module);
  if (m == nullptr) return nullptr;
  if (PyModule_AddObjectRef(m, "KVCache", reinterpret_cast<PyObject*>(cache_type())) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  // the torch whose headers this was compiled with
  if (PyModule_AddStringConstant(m, "built_against", KV_CACHE_TORCH) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
