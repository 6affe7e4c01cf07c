// kv_append, PagedAttention.attend and linear_w4 from Python: argument marshalling only, checks of torch
// tensors and the call of the C ABI, as the rest of the binding does it in Python. Compiled because a call with
// up to 14 tensors took 10 to 20 us there (attributes read, 27 arguments through ctypes), several
// times what its kernel takes for a few tokens.
//
// Every function takes its arguments by position, the C entry's address and the stream (None: the current one)
// first, and returns the output or, as an int, a status that is not GDN_OK. An output left out (None)
// is allocated here, for the current stream alone.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <string>

#include "gdn_attention.h"
#include "gdn_prefill.h"

namespace {

using at::Tensor;
constexpr int64_t kIntMax = INT32_MAX;  // sizes cross the C ABI as int32

struct Refused {};  // a Python error is set

[[noreturn]] void refuse(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw Refused();
}
const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a tensor", name);
    throw Refused();
  }
  return THPVariable_Unpack(o);
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}
bool here(const Tensor& t) { return t.is_cuda() && t.get_device() == c10::cuda::current_device(); }

// A [rows, columns] bf16 CUDA tensor with packed columns.
struct Rows {
  void* at = nullptr;
  int64_t ld = 0, rows = 0, cols = 0;
  Rows() = default;
  Rows(PyObject* o, const char* name) : Rows(tensor(o, name), name) {}
  Rows(const Tensor& t, const char* name) {
    const std::string n(name);
    if (t.scalar_type() != at::kBFloat16 || t.dim() != 2 || !here(t))
      refuse(n + " must be a two-dimensional bf16 CUDA tensor on the current device");
    rows = t.size(0);
    cols = t.size(1);
    ld = t.stride(0);
    if (t.stride(1) != 1 && cols > 1 && rows) refuse("the columns of " + n + " must be packed");
    if (rows > 1 && ld < cols) refuse("the rows of " + n + " must not overlap");
    if (rows <= 1) ld = (cols + 7) / 8 * 8;  // the stride of one row, or none, does not matter
    at = t.data_ptr();
  }
  bool like(const Rows& o) const { return rows == o.rows && cols == o.cols; }
};
// A [slots, heads, head_dim] bf16 CUDA tensor whose slots' rows are packed.
struct Cache {
  void* at;
  int64_t n, heads, d, ld;
  Cache(PyObject* o, const char* name) {
    const Tensor& t = tensor(o, name);
    const std::string c(name);
    if (t.scalar_type() != at::kBFloat16 || t.dim() != 3 || !here(t))
      refuse(c + " must be a [slots, heads, head_dim] bf16 CUDA tensor on the current device");
    n = t.size(0), heads = t.size(1), d = t.size(2), ld = t.stride(0);
    if (n > kIntMax || (n && ((t.stride(2) != 1 && d > 1) || (t.stride(1) != d && heads > 1) || (ld < heads * d && n > 1))))
      refuse("the heads of a slot of " + c + " must be packed, and its slots must not overlap");
    if (n <= 1) ld = (heads * d + 7) / 8 * 8;
    at = t.data_ptr();
  }
};
// The address of a contiguous CUDA tensor of n values, or with None none.
void* dense(PyObject* o, const char* name, at::ScalarType type, int64_t n) {
  const Tensor& t = tensor(o, name);
  if (t.scalar_type() != type || !t.is_contiguous() || t.numel() != n || !here(t))
    refuse(std::string(name) + " must be a contiguous " + c10::toString(type) + " CUDA tensor of " + std::to_string(n) +
           " values on the current device");
  return t.data_ptr();
}
void* maybe(PyObject* o, const char* name, at::ScalarType type, int64_t n) {
  return o == Py_None ? nullptr : dense(o, name, type, n);
}
void* current() { return c10::cuda::getCurrentCUDAStream().stream(); }
void* stream_of(PyObject* o) { return o == Py_None ? current() : PyLong_AsVoidPtr(o); }

// An output: the caller's, or a new one.
struct Out : Rows {
  PyObject* owned = nullptr;  // a reference to return
  Out() = default;
  Out(const Out&) = delete;
  Out& operator=(const Out&) = delete;
  ~Out() { Py_XDECREF(owned); }
  void make(PyObject* o, const char* name, int64_t rows_, int64_t cols_, const Tensor& like, const char* size) {
    if (o != Py_None) {
      static_cast<Rows&>(*this) = Rows(o, name);
      if (rows != rows_ || cols != cols_) refuse(size);
      Py_INCREF(o);
      owned = o;
    } else {
      Tensor t = at::empty({rows_, cols_}, like.options().requires_grad(false));
      at = t.data_ptr();
      rows = rows_, cols = cols_, ld = cols_;
      owned = THPVariable_Wrap(std::move(t));
      if (!owned) throw Refused();
    }
  }
  PyObject* result(gdn_status st) {
    if (st != GDN_OK) return PyLong_FromLong(st);
    PyObject* o = owned;
    owned = nullptr;
    return o;
  }
};
#define CALL(st, ...)       \
  Py_BEGIN_ALLOW_THREADS;   \
  st = __VA_ARGS__;         \
  Py_END_ALLOW_THREADS

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    throw Refused();
  }
}

// entry, stream, q, k, v, token_pos, slots, inv_freq, k_cache, v_cache, q_norm_w, k_norm_w, norm_eps, interleaved, q_out, error
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    count(n, 16);
    const auto entry = reinterpret_cast<decltype(&gdn_kv_append)>(PyLong_AsVoidPtr(a[0]));
    const Cache kc(a[8], "k_cache"), vc(a[9], "v_cache");
    const Rows k(a[3], "k"), v(a[4], "v");
    const int64_t T = k.rows, d = kc.d;
    if (vc.n != kc.n || vc.heads != kc.heads || vc.d != d) refuse("k_cache and v_cache have different sizes");
    if (k.cols != kc.heads * d || !v.like(k)) refuse("k and v must be [tokens, " + std::to_string(kc.heads * d) + "]");
    if (T > kIntMax) return PyLong_FromLong(GDN_ERR_UNSUPPORTED);
    Rows q;
    Out out;
    int64_t heads = 0;
    if (a[2] != Py_None) {
      q = Rows(a[2], "q");
      heads = d ? q.cols / d : 0;
      if (q.rows != T || heads * d != q.cols || heads == 0 || heads > kIntMax)
        refuse("q must be [tokens, heads * " + std::to_string(d) + "]");
      out.make(a[14], "q_out", T, q.cols, THPVariable_Unpack(a[2]), "q_out must have q's shape");
    } else if (a[14] != Py_None) {
      refuse("q_out without q");
    }
    const int64_t half = a[7] == Py_None ? 0 : tensor(a[7], "inv_freq").numel();
    if (half > kIntMax / 2 || kc.heads > kIntMax || d > kIntMax) return PyLong_FromLong(GDN_ERR_UNSUPPORTED);
    const void* freq = maybe(a[7], "inv_freq", at::kFloat, half);
    const void* pos = dense(a[5], "token_pos", at::kInt, T);
    const void* slots = dense(a[6], "slots", at::kLong, T);
    const void* qw = maybe(a[10], "q_norm_w", at::kBFloat16, d);
    const void* kw = maybe(a[11], "k_norm_w", at::kBFloat16, d);
    void* error = maybe(a[15], "error", at::kInt, 1);
    const double eps = PyFloat_AsDouble(a[12]);
    const int pairs = PyObject_IsTrue(a[13]);
    if ((eps == -1.0 && PyErr_Occurred()) || pairs < 0) throw Refused();
    void* stream = stream_of(a[1]);
    gdn_status st;
    CALL(st, entry((int32_t)T, (int32_t)heads, (int32_t)kc.heads, (int32_t)d, q.at, q.ld, k.at, k.ld, v.at, v.ld,
                   static_cast<const int32_t*>(pos), static_cast<const int64_t*>(slots), kc.n, static_cast<const float*>(freq),
                   (int32_t)(2 * half), pairs, qw, kw, (float)eps, out.at, out.ld, kc.at, kc.ld, vc.at, vc.ld,
                   static_cast<uint32_t*>(error), stream));
    if (!out.owned && st == GDN_OK) Py_RETURN_NONE;
    return out.result(st);
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// entry, stream, handle, workspace, its stream, kv heads, head_dim, block, columns, q, k_cache, v_cache, block_table, cu_seqlens,
// context_lens, gate, out, max_len
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    count(n, 18);
    const auto entry = reinterpret_cast<decltype(&gdn_attn_paged)>(PyLong_AsVoidPtr(a[0]));
    const int64_t heads = integer(a[5]), d = integer(a[6]), block = integer(a[7]), cols = integer(a[8]);
    const Rows q(a[9], "q");
    const Cache kc(a[10], "k_cache"), vc(a[11], "v_cache");
    if (kc.heads != heads || kc.d != d || vc.heads != heads || vc.d != d || vc.n != kc.n || kc.n % block)
      refuse("k_cache and v_cache must be [slots, " + std::to_string(heads) + ", " + std::to_string(d) + "], whole blocks of " +
             std::to_string(block) + " slots");
    if (q.cols != cols) refuse("q must be [tokens, " + std::to_string(cols) + "]");
    const Tensor& table = tensor(a[12], "block_table");
    if (table.dim() != 2) refuse("block_table must be [requests, blocks]");
    const int64_t T = q.rows, S = table.size(0), wide = table.size(1);
    int64_t most = T;
    if (a[17] != Py_None) {
      int over = 0;
      most = PyLong_AsLongLongAndOverflow(a[17], &over);
      if (most == -1 && PyErr_Occurred()) throw Refused();
      if (over) most = over > 0 ? T : -1;
      if (most > T) most = T;
    }
    if (T > kIntMax || S >= kIntMax || wide > kIntMax || most < 0) return PyLong_FromLong(GDN_ERR_ARG);
    Rows gate;
    if (a[15] != Py_None) {
      gate = Rows(a[15], "gate");
      if (!gate.like(q)) refuse("gate must have q's shape");
    }
    Out out;
    out.make(a[16], "out", T, cols, THPVariable_Unpack(a[9]), "out must have q's shape");
    const void* blocks = dense(a[12], "block_table", at::kInt, S * wide);
    const void* cu = dense(a[13], "cu_seqlens", at::kInt, S + 1);
    const void* ctx = dense(a[14], "context_lens", at::kInt, S);
    void* stream = stream_of(a[1]);
    // the workspace is kept until what runs here is done; another stream that was given has been seen to
    if (a[1] == Py_None && stream != PyLong_AsVoidPtr(a[4]))
      tensor(a[3], "workspace").record_stream(c10::cuda::getCurrentCUDAStream());
    gdn_status st;
    CALL(st, entry(static_cast<gdn_attn_t*>(PyLong_AsVoidPtr(a[2])), (int32_t)S, (int32_t)T, (int32_t)most, q.at, q.ld, kc.at, kc.ld,
                   vc.at, vc.ld, (int32_t)(kc.n / block), static_cast<const int32_t*>(blocks), (int32_t)wide,
                   static_cast<const int32_t*>(cu), static_cast<const int32_t*>(ctx), gate.at, gate.ld, out.at, out.ld, stream));
    return out.result(st);
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// entry, stream, x, codes, scales, zeros, bias, activation, residual, out
PyObject* linear_w4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    count(n, 10);
    const auto entry = reinterpret_cast<decltype(&gdn_linear_w4)>(PyLong_AsVoidPtr(a[0]));
    const Rows x(a[2], "x");
    const Tensor &codes = tensor(a[3], "codes"), &scales = tensor(a[4], "scales");
    const int64_t M = x.rows, K = x.cols;
    if (codes.dim() != 2 || scales.dim() != 2 || codes.size(1) * 2 != K || scales.size(0) != codes.size(0))
      refuse("codes must be [N, K / 2] and scales [N, K / group]");
    const int64_t N = scales.size(0), groups = scales.size(1);
    if (groups == 0 || K % groups) refuse("the groups must divide K evenly");
    if (M > kIntMax || N > kIntMax || K > kIntMax) return PyLong_FromLong(GDN_ERR_UNSUPPORTED);
    const bool mx = scales.scalar_type() == at::kByte;
    Out out;
    out.make(a[9], "out", M, N, THPVariable_Unpack(a[2]), "out must be [M, N]");
    Rows r;
    if (a[8] != Py_None) {
      r = Rows(a[8], "residual");
      if (!r.like(out)) refuse("residual must be [M, N]");
    }
    const void* c = dense(a[3], "codes", at::kByte, N * (K / 2));
    const void* s = dense(a[4], "scales", mx ? at::kByte : at::kBFloat16, N * groups);
    const void* z = maybe(a[5], "zeros", at::kByte, N * groups);
    const void* b = maybe(a[6], "bias", at::kBFloat16, N);
    const int64_t act = integer(a[7]);
    void* stream = stream_of(a[1]);
    gdn_status st;
    CALL(st, entry((int32_t)M, (int32_t)N, (int32_t)K, x.at, x.ld, mx, (int32_t)(K / groups), static_cast<const uint8_t*>(c), s,
                   static_cast<const uint8_t*>(z), b, (int32_t)act, r.at, r.ld, out.at, out.ld, stream));
    return out.result(st);
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyMethodDef methods[] = {{"kv_append", (PyCFunction)(void (*)(void))kv_append, METH_FASTCALL, nullptr},
                         {"attend", (PyCFunction)(void (*)(void))attend, METH_FASTCALL, nullptr},
                         {"linear_w4", (PyCFunction)(void (*)(void))linear_w4, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module_def); }
