// feed_forward_py.cpp -- the Python binding of a feed-forward block's operators
// (include/feed_forward.h): mm_tn_gated, gated_grad, mm_nt, quantize_e4m3 and
// mm_tn_e4m3 as an extension module over torch's tensors.
//
// Argument marshalling only; compiled code for the small calls (a decode step's
// kernels run for 2 to 6 us): from Python, through ctypes, quantising 16 x 4096
// took 26.7 us a call and a gated projection of 24 tokens 13.5.
//
// bind() hands over the C functions' addresses, so that the one loaded
// libgemm_tn.so is called, and the exception type of its errors.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_strided.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>

#include "feed_forward.h"
#include "py_args.h"

namespace {

using namespace py_args;

decltype(&gemm_tn_gated) g_gated = nullptr;
decltype(&gated_grad) g_gated_grad = nullptr;
decltype(&gemm_nt) g_nt = nullptr;
decltype(&quantize_e4m3) g_quantize = nullptr;
decltype(&gemm_tn_e4m3) g_e4m3 = nullptr;
PyObject* g_error = nullptr;   // GemmTnError(status, where)

bool refuse(PyObject* kind, const std::string& what) {
  PyErr_SetString(kind, what.c_str());
  return false;
}

// ---------------------------------------------------------------- matrices

struct Matrix {
  const Tensor* t = nullptr;
  void* data = nullptr;
  int64_t rows = 0, cols = 0, pitch = 0;
  at::ScalarType type() const { return t->scalar_type(); }
};

// A 2-D CUDA tensor on `index` (-1: any device, which becomes *index) with unit
// stride along its rows.
bool matrix(PyObject* o, const char* what, int64_t* index, Matrix* to) {
  const Tensor* t = tensor(o, what);
  if (t == nullptr) return false;
  const int64_t at = cuda_index(*t);
  if (at < 0 || (*index >= 0 && at != *index)) return refuse(PyExc_ValueError, std::string(what) + " must be a CUDA tensor on the operands' one device");
  *index = at;
  if (t->dim() != 2 || (t->size(1) > 1 && t->stride(1) != 1))
    return refuse(PyExc_ValueError, std::string(what) + " must be 2-D with unit stride along the last dimension");
  if (!stored(*t, what)) return false;
  to->t = t;
  to->data = t->data_ptr();
  to->rows = t->size(0);
  to->cols = t->size(1);
  to->pitch = to->rows > 1 ? t->stride(0) : std::max<int64_t>(to->cols, 1);
  return true;
}

// The same of a given shape and type.
bool matrix_of(PyObject* o, const char* what, int64_t index, int64_t rows, int64_t cols, at::ScalarType type, Matrix* to) {
  if (!matrix(o, what, &index, to)) return false;
  if (to->type() != type) return refuse(PyExc_TypeError, std::string(what) + " must be " + c10::toString(type));
  if (to->rows != rows || to->cols != cols) {
    const int64_t shape[] = {rows, cols};
    return refuse(PyExc_ValueError, std::string(what) + " must be " + shape_text(shape));
  }
  return true;
}

// A new one.
bool made(Tensor&& t, Tensor* keep, Matrix* to) {
  *keep = std::move(t);
  to->t = keep;
  to->data = keep->data_ptr();
  to->rows = keep->size(0);
  to->cols = keep->size(1);
  to->pitch = to->rows > 1 ? keep->stride(0) : std::max<int64_t>(to->cols, 1);
  return true;
}

bool half_type(const Matrix& a, int* code) {
  if (a.type() == at::kHalf || a.type() == at::kBFloat16) {
    *code = a.type() == at::kHalf ? GEMM_TN_F16 : GEMM_TN_BF16;
    return true;
  }
  return refuse(PyExc_TypeError, std::string("unsupported dtype ") + c10::toString(a.type()) + ": expected float16 or bfloat16");
}

bool element(at::ScalarType type, const char* what, int* code) {
  if (type == at::kHalf || type == at::kBFloat16 || type == at::kFloat) {
    *code = type == at::kHalf ? GEMM_TN_ELEM_F16 : type == at::kBFloat16 ? GEMM_TN_ELEM_BF16 : GEMM_TN_ELEM_F32;
    return true;
  }
  return refuse(PyExc_TypeError, std::string("unsupported ") + what + " " + c10::toString(type) + ": expected float16, bfloat16 or float32");
}

bool same_type(const Matrix& a, const Matrix& b) {
  return a.type() == b.type() || refuse(PyExc_TypeError, "a and b must have the same dtype");
}

// ---------------------------------------------------------------- other arguments

bool gate(PyObject* o, int* code) {
  *code = GEMM_TN_ACT_SILU;
  if (o == nullptr) return true;
  const char* name = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
  if (name != nullptr && std::strcmp(name, "silu") == 0) return true;
  if (name != nullptr && std::strcmp(name, "gelu") == 0) {
    *code = GEMM_TN_ACT_GELU;
    return true;
  }
  if (name != nullptr && std::strcmp(name, "relu") == 0) {
    *code = GEMM_TN_ACT_RELU;
    return true;
  }
  PyErr_Clear();
  return refuse(PyExc_ValueError, "activation must be \"silu\", \"gelu\" or \"relu\"");
}

bool flag(PyObject* o, int* to) {
  *to = o != nullptr ? PyObject_IsTrue(o) : 0;
  return *to >= 0;
}

// The product's type: what is asked for, else out's, else `otherwise`.
bool output_type(PyObject* asked, PyObject* out, at::ScalarType otherwise, at::ScalarType* to) {
  *to = otherwise;
  if (asked != nullptr) {
    if (!THPDtype_Check(asked)) return refuse(PyExc_TypeError, "out_dtype must be a torch.dtype");
    *to = reinterpret_cast<THPDtype*>(asked)->scalar_type;
  } else if (out != nullptr) {
    const Tensor* t = tensor(out, "out");
    if (t == nullptr) return false;
    *to = t->scalar_type();
  }
  return true;
}

bool status_word(PyObject* o, int64_t index, int** to) {
  *to = nullptr;
  if (o == nullptr) return true;
  const Tensor* t = tensor(o, "status");
  if (t == nullptr) return false;
  if (cuda_index(*t) != index || t->scalar_type() != at::kInt || t->numel() < 1 || !t->is_contiguous() || !stored(*t, "status"))
    return PyErr_Occurred() ? false
                            : refuse(PyExc_ValueError, "status must be a contiguous int32 tensor of at least one element on the operands' device");
  *to = static_cast<int*>(t->data_ptr());
  return true;
}

// One call of the library on that device and its current stream; false with
// GemmTnError set. The call itself throws nothing.
template <class Call>
bool run(int64_t index, const char* name, Call call) {
  int rc;
  {
    const c10::cuda::CUDAGuard device(static_cast<c10::DeviceIndex>(index));
    cudaStream_t stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(index)).stream();
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

// The given output, or the new one.
PyObject* result(PyObject* given, const Tensor& made) {
  if (given == nullptr) return THPVariable_Wrap(made);
  Py_INCREF(given);
  return given;
}

int64_t round_up(int64_t x, int64_t q) { return (x + q - 1) / q * q; }

// ---------------------------------------------------------------- calls

PyObject* mm_tn_gated(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  HANDLE_TH_ERRORS
  static const char* const names[] = {"a", "b", "out", "pre", "activation", "status"};
  PyObject* in[6];
  if (!place("mm_tn_gated", names, 2, args, nargs, kwnames, in)) return nullptr;
  int64_t index = -1;
  Matrix a, b, h, pre;
  int code, act, *status;
  if (!matrix(in[0], "a", &index, &a) || !matrix(in[1], "b", &index, &b) || !same_type(a, b) || !half_type(a, &code)) return nullptr;
  if (b.rows % 2 != 0 || b.cols != a.cols) {
    refuse(PyExc_ValueError, "b must be [2N, K], the two projections' rows, with a's K = " + std::to_string(a.cols));
    return nullptr;
  }
  const int64_t m = a.rows, n = b.rows / 2, k = a.cols;
  Tensor keep;
  if (!(in[2] == nullptr ? made(at::empty({m, n}, a.t->options()), &keep, &h) : matrix_of(in[2], "out", index, m, n, a.type(), &h)) ||
      (in[3] != nullptr && !matrix_of(in[3], "pre", index, m, 2 * n, a.type(), &pre)) || !gate(in[4], &act) ||
      !status_word(in[5], index, &status))
    return nullptr;
  if (!run(index, "gemm_tn_gated", [&](gemm_tn_stream_t stream) {
        return g_gated(code, m, n, k, a.data, a.pitch, b.data, b.pitch, h.data, h.pitch, pre.data, pre.pitch, act, status, stream);
      }))
    return nullptr;
  return result(in[2], keep);
  END_HANDLE_TH_ERRORS
}

PyObject* gated_grad_call(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  HANDLE_TH_ERRORS
  static const char* const names[] = {"grad", "pre", "out", "activation"};
  PyObject* in[4];
  if (!place("gated_grad", names, 2, args, nargs, kwnames, in)) return nullptr;
  int64_t index = -1;
  Matrix grad, pre, out;
  int code, act;
  if (!matrix(in[0], "grad", &index, &grad) || !half_type(grad, &code)) return nullptr;
  const int64_t m = grad.rows, n = grad.cols;
  Tensor keep;
  // a new one's rows lie a multiple of 128 bytes apart: the products read them in place, in whole lines
  if (!matrix_of(in[1], "pre", index, m, 2 * n, grad.type(), &pre) ||
      !(in[2] == nullptr ? made(at::empty_strided({m, 2 * n}, {std::max<int64_t>(round_up(2 * n, 64), 1), 1}, grad.t->options()), &keep, &out)
                         : matrix_of(in[2], "out", index, m, 2 * n, grad.type(), &out)) ||
      !gate(in[3], &act))
    return nullptr;
  if (!run(index, "gated_grad", [&](gemm_tn_stream_t stream) {
        return g_gated_grad(code, m, n, grad.data, grad.pitch, pre.data, pre.pitch, out.data, out.pitch, act, stream);
      }))
    return nullptr;
  return result(in[2], keep);
  END_HANDLE_TH_ERRORS
}

PyObject* mm_nt(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  HANDLE_TH_ERRORS
  static const char* const names[] = {"a", "b", "out", "out_dtype", "accumulate", "status"};
  PyObject* in[6];
  if (!place("mm_nt", names, 2, args, nargs, kwnames, in)) return nullptr;
  int64_t index = -1;
  Matrix a, b, c;
  int code, add, *status;
  at::ScalarType type;
  if (!matrix(in[0], "a", &index, &a) || !matrix(in[1], "b", &index, &b) || !same_type(a, b) || !half_type(a, &code) ||
      !output_type(in[3], in[2], a.type(), &type) || !flag(in[4], &add))
    return nullptr;
  if (a.rows != b.rows) {
    refuse(PyExc_ValueError, "a and b must be [K, M] and [K, N]: " + std::to_string(a.rows) + " and " + std::to_string(b.rows) + " rows");
    return nullptr;
  }
  if (type != a.type() && type != at::kFloat) {
    refuse(PyExc_TypeError, std::string("unsupported output dtype ") + c10::toString(type));
    return nullptr;
  }
  if (add != 0 && (in[2] == nullptr || type != at::kFloat)) {
    refuse(PyExc_ValueError, "accumulate needs an fp32 out");
    return nullptr;
  }
  const int64_t m = a.cols, n = b.cols, k = a.rows;
  Tensor keep;
  if (!(in[2] == nullptr ? made(at::empty({m, n}, a.t->options().dtype(type)), &keep, &c)
                         : matrix_of(in[2], "out", index, m, n, type, &c)) ||
      !status_word(in[5], index, &status))
    return nullptr;
  if (!run(index, "gemm_nt", [&](gemm_tn_stream_t stream) {
        return g_nt(code, m, n, k, a.data, a.pitch, b.data, b.pitch, c.data, c.pitch,
                    type == at::kFloat ? GEMM_TN_OUT_F32 : GEMM_TN_OUT_INPUT, add, status, stream);
      }))
    return nullptr;
  return result(in[2], keep);
  END_HANDLE_TH_ERRORS
}

PyObject* quantize(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  HANDLE_TH_ERRORS
  static const char* const names[] = {"x", "block_rows", "transpose", "out", "scale"};
  PyObject* in[5];
  if (!place("quantize_e4m3", names, 1, args, nargs, kwnames, in)) return nullptr;
  int64_t index = -1;
  Matrix x, q;
  int source, transpose;
  if (!matrix(in[0], "x", &index, &x) || !element(x.type(), "dtype", &source) || !flag(in[2], &transpose)) return nullptr;
  const long long block = in[1] != nullptr ? PyLong_AsLongLong(in[1]) : 1;
  if (block == -1 && PyErr_Occurred()) return nullptr;
  if (block != 1 && block != 128) {
    refuse(PyExc_ValueError, "block_rows must be 1 or 128");
    return nullptr;
  }
  const int64_t lines = transpose ? x.cols : x.rows, along = transpose ? x.rows : x.cols;
  const int64_t s_lines = (lines + block - 1) / block, s_blocks = (along + 127) / 128;
  Tensor keep_q, keep_s;
  if (!(in[3] == nullptr ? made(at::empty_strided({lines, along}, {std::max<int64_t>(round_up(along, 128), 1), 1},
                                                  x.t->options().dtype(at::kFloat8_e4m3fn)), &keep_q, &q)
                         : matrix_of(in[3], "out", index, lines, along, at::kFloat8_e4m3fn, &q)))
    return nullptr;
  const Tensor* scale = &keep_s;
  if (in[4] == nullptr) {
    // a single row's scales lie side by side with the other rows', columns of them a multiple of 16 bytes apart
    const int64_t line = block == 1 ? 1 : std::max<int64_t>(round_up(s_blocks, 4), 1);
    const int64_t blk = block == 1 ? std::max<int64_t>(round_up(s_lines, 4), 1) : 1;
    keep_s = at::empty_strided({s_lines, s_blocks}, {line, blk}, x.t->options().dtype(at::kFloat));
  } else {
    scale = tensor(in[4], "scale");
    if (scale == nullptr) return nullptr;
    const int64_t shape[] = {s_lines, s_blocks};
    if (scale->scalar_type() != at::kFloat) {
      refuse(PyExc_TypeError, "scale must be float32");
      return nullptr;
    }
    if (cuda_index(*scale) != index || scale->sizes() != at::IntArrayRef(shape)) {
      refuse(PyExc_ValueError, "scale must be " + shape_text(shape) + " on x's device");
      return nullptr;
    }
    if (!stored(*scale, "scale")) return nullptr;
  }
  // a dimension of one is never stepped along, whatever its stride
  const int64_t s_line = s_lines > 1 ? scale->stride(0) : 1, s_blk = s_blocks > 1 ? scale->stride(1) : 1;
  float* to = static_cast<float*>(scale->data_ptr());
  if (!run(index, "quantize_e4m3", [&](gemm_tn_stream_t stream) {
        return g_quantize(source, x.rows, x.cols, x.data, x.pitch, q.data, q.pitch, to, s_line, s_blk, static_cast<int>(block),
                          transpose, stream);
      }))
    return nullptr;
  PyObject* first = result(in[3], keep_q);
  PyObject* second = first != nullptr ? result(in[4], keep_s) : nullptr;
  PyObject* both = second != nullptr ? PyTuple_Pack(2, first, second) : nullptr;
  Py_XDECREF(first);
  Py_XDECREF(second);
  return both;
  END_HANDLE_TH_ERRORS
}

// fp32 scales [lines, blocks] of any strides.
struct Scales {
  const float* data = nullptr;
  int64_t lines = 0, blocks = 0, s_line = 0, s_blk = 0;
};
bool scales(PyObject* o, const char* what, int64_t index, Scales* to) {
  const Tensor* t = tensor(o, what);
  if (t == nullptr) return false;
  if (t->scalar_type() != at::kFloat) return refuse(PyExc_TypeError, std::string(what) + " must be float32");
  if (cuda_index(*t) != index || t->dim() != 2) return refuse(PyExc_ValueError, std::string(what) + " must be 2-D on the operands' device");
  if (!stored(*t, what)) return false;
  *to = {static_cast<const float*>(t->data_ptr()), t->size(0), t->size(1), t->size(0) > 1 ? t->stride(0) : 1,
         t->size(1) > 1 ? t->stride(1) : 1};
  return true;
}

PyObject* mm_tn_e4m3(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames) {
  HANDLE_TH_ERRORS
  static const char* const names[] = {"a", "a_scale", "b", "b_scale", "out", "out_dtype", "accumulate", "status"};
  PyObject* in[8];
  if (!place("mm_tn_e4m3", names, 4, args, nargs, kwnames, in)) return nullptr;
  int64_t index = -1;
  Matrix a, b, c;
  Scales sa, sb;
  int out_code, add, *status;
  at::ScalarType type;
  if (!matrix(in[0], "a", &index, &a) || !matrix(in[2], "b", &index, &b)) return nullptr;
  if (a.type() != at::kFloat8_e4m3fn || b.type() != at::kFloat8_e4m3fn) {
    refuse(PyExc_TypeError, "a and b must be float8_e4m3fn");
    return nullptr;
  }
  if (!scales(in[1], "a_scale", index, &sa) || !scales(in[3], "b_scale", index, &sb) ||
      !output_type(in[5], in[4], at::kBFloat16, &type) || !element(type, "output dtype", &out_code) || !flag(in[6], &add))
    return nullptr;
  const int64_t m = a.rows, n = b.rows, k = a.cols, blocks = (k + 127) / 128, shared = (n + 127) / 128;
  if (b.cols != k) {
    refuse(PyExc_ValueError, "inner dimensions differ: " + std::to_string(k) + " and " + std::to_string(b.cols));
    return nullptr;
  }
  if (sa.lines != m || sa.blocks != blocks) {
    const int64_t shape[] = {m, blocks};
    refuse(PyExc_ValueError, "a_scale must be " + shape_text(shape));
    return nullptr;
  }
  if ((sb.lines != n && sb.lines != shared) || sb.blocks != blocks) {
    const int64_t each[] = {n, blocks}, together[] = {shared, blocks};
    refuse(PyExc_ValueError, "b_scale must be " + shape_text(each) + " or " + shape_text(together));
    return nullptr;
  }
  if (add != 0 && (in[4] == nullptr || type != at::kFloat)) {
    refuse(PyExc_ValueError, "accumulate needs an fp32 out");
    return nullptr;
  }
  Tensor keep;
  if (!(in[4] == nullptr ? made(at::empty({m, n}, a.t->options().dtype(type)), &keep, &c)
                         : matrix_of(in[4], "out", index, m, n, type, &c)) ||
      !status_word(in[7], index, &status))
    return nullptr;
  // one row: its pitch is never stepped over, and a view's may be anything
  const int64_t lda = m > 1 ? a.pitch : round_up(k, 16), ldb = n > 1 ? b.pitch : round_up(k, 16);
  if (!run(index, "gemm_tn_e4m3", [&](gemm_tn_stream_t stream) {
        return g_e4m3(m, n, k, a.data, lda, sa.data, sa.s_line, sa.s_blk, b.data, ldb, sb.data, sb.s_line, sb.s_blk,
                      sb.lines == n ? 1 : 128, c.data, c.pitch, out_code, add, status, stream);
      }))
    return nullptr;
  return result(in[4], keep);
  END_HANDLE_TH_ERRORS
}

// bind(error, gemm_tn_gated, gated_grad, gemm_nt, quantize_e4m3, gemm_tn_e4m3): the exception type and five addresses.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  void* at[5];
  if (nargs != 6) {
    PyErr_SetString(PyExc_TypeError, "bind() takes the exception type and five addresses");
    return nullptr;
  }
  for (int i = 0; i < 5; ++i) {
    at[i] = PyLong_AsVoidPtr(args[1 + i]);
    if (at[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is 0");
      return nullptr;
    }
  }
  Py_INCREF(args[0]);
  Py_XDECREF(g_error);
  g_error = args[0];
  g_gated = reinterpret_cast<decltype(g_gated)>(at[0]);
  g_gated_grad = reinterpret_cast<decltype(g_gated_grad)>(at[1]);
  g_nt = reinterpret_cast<decltype(g_nt)>(at[2]);
  g_quantize = reinterpret_cast<decltype(g_quantize)>(at[3]);
  g_e4m3 = reinterpret_cast<decltype(g_e4m3)>(at[4]);
  Py_RETURN_NONE;
}

PyMethodDef functions[] = {
    {"bind", as_function(bind), METH_FASTCALL, nullptr},
    {"mm_tn_gated", as_function(mm_tn_gated), METH_FASTCALL | METH_KEYWORDS,
     "mm_tn_gated(a, b, out=None, pre=None, activation='silu', status=None)\n--\n\n"
     "act(A Bg^T) * (A Bu^T) through gemm_tn_gated. a: [M, K]; b: [2N, K], the\n"
     "gate's rows Bg then the other projection's Bu, CUDA fp16/bf16 with unit\n"
     "stride along K; out: optional [M, N]; pre: optional [M, 2N] that receives\n"
     "both projections side by side, for gated_grad; activation: 'silu', 'gelu'\n"
     "(erf form) or 'relu'; status: optional one-element int32 CUDA tensor for the\n"
     "device watchdog. Returns out."},
    {"gated_grad", as_function(gated_grad_call), METH_FASTCALL | METH_KEYWORDS,
     "gated_grad(grad, pre, out=None, activation='silu')\n--\n\n"
     "The gradient of act(G) * U through gated_grad. grad: [M, N], of the\n"
     "output; pre: [M, 2N], G and U side by side (mm_tn_gated's); out: optional\n"
     "[M, 2N], dG and dU side by side (may be pre itself). With mm_tn_gated's a\n"
     "and b, the gradients are mm_nn(out, b) and mm_nt(out, a). Without out, its\n"
     "rows lie a multiple of 128 bytes apart, which suits both. Returns out."},
    {"mm_nt", as_function(mm_nt), METH_FASTCALL | METH_KEYWORDS,
     "mm_nt(a, b, out=None, out_dtype=None, accumulate=False, status=None)\n--\n\n"
     "C = A^T B through gemm_nt. a: [K, M], b: [K, N] CUDA tensors of one\n"
     "fp16/bf16 dtype with unit stride along their last dimension; out: optional\n"
     "[M, N] of out_dtype: a's or torch.float32 (None: out's, or a's).\n"
     "accumulate: the product is added to out, which is fp32. Returns out."},
    {"quantize_e4m3", as_function(quantize), METH_FASTCALL | METH_KEYWORDS,
     "quantize_e4m3(x, block_rows=1, transpose=False, out=None, scale=None)\n--\n\n"
     "x [M, K] (CUDA fp16, bf16 or fp32, unit stride along K) as (q, scale)\n"
     "through quantize_e4m3: q float8_e4m3fn [M, K], or of x's transpose [K, M]; a\n"
     "power of two for each block of block_rows (1 or 128) rows and 128 columns of\n"
     "q. Without out and scale, q's rows lie a multiple of 128 bytes apart, which\n"
     "suits mm_tn_e4m3 best, and the scales of single rows (block_rows 1) side by\n"
     "side (scale.stride(0) is 1)."},
    {"mm_tn_e4m3", as_function(mm_tn_e4m3), METH_FASTCALL | METH_KEYWORDS,
     "mm_tn_e4m3(a, a_scale, b, b_scale, out=None, out_dtype=None, accumulate=False, status=None)\n--\n\n"
     "The product of two matrices quantised in blocks of 128 through\n"
     "gemm_tn_e4m3. a: [M, K], b: [N, K] CUDA float8_e4m3fn, rows a multiple of 16\n"
     "bytes apart (quantize_e4m3's are); a_scale: fp32 [M, ceil(K / 128)]; b_scale:\n"
     "[N, ceil(K / 128)], or [ceil(N / 128), ceil(K / 128)] where 128 rows share\n"
     "theirs; any strides. out: optional [M, N] of out_dtype: fp16, bf16 or fp32\n"
     "(None: out's, or bf16). accumulate: the product is added to out, which is\n"
     "fp32. Returns out."},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_feed_forward", nullptr, -1, functions, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__feed_forward() {
  PyObject* m = PyModule_Create(&module);
  if (m == nullptr) return nullptr;
  // the torch whose headers this was compiled with
  if (PyModule_AddStringConstant(m, "built_against", BUILT_AGAINST_TORCH) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
