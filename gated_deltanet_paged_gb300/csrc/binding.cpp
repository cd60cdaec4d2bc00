// binding.cpp -- Python binding of the attention layer's calls: rotary
// positions, the append to a paged key / value cache, paged attention.
//
// At decode sizes these calls last 2 to 10 microseconds on the GPU.  Checked from
// Python and made through ctypes each took 11 to 25 us of host time, most of it
// in property lookups and in allocating outputs between launches; here the same
// checks, the allocations and the C call take 4 to 7.  Every function checks
// types, shapes and devices, makes one call of include/gdn_paged.h on the current
// stream, and raises on a non-zero status.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gdn_paged.h"

namespace {

PyObject* g_error = nullptr;  // the package's GdnError(function, status)

// A Python exception is set.
struct Raised {};

[[noreturn]] void fail(PyObject* type, const char* format, ...) {
  va_list args;
  va_start(args, format);
  PyErr_FormatV(type, format, args);
  va_end(args);
  throw Raised{};
}

const char* dtype_name(at::ScalarType t) { return c10::toString(t); }

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (o == Py_None) fail(PyExc_ValueError, "%s is required", name);
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "%s must be a tensor, got %s", name, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

void check(const at::Tensor& t, const char* name, at::ScalarType type, const c10::Device* device) {
  if (t.scalar_type() != type)
    fail(PyExc_TypeError, "%s must be %s, got %s", name, dtype_name(type), dtype_name(t.scalar_type()));
  if (!t.is_cuda()) fail(PyExc_ValueError, "%s must be a CUDA tensor", name);
  if (device && t.device() != *device) fail(PyExc_ValueError, "%s must be on the device of the other tensors", name);
}

gdn_bf16* bf16(const at::Tensor& t) { return static_cast<gdn_bf16*>(t.data_ptr()); }

// A bf16 [T, H, D] tensor with dense heads; the token stride may be padded (a
// slice of a fused projection).
struct Heads {
  const at::Tensor* t;
  int64_t T, H, D, stride;
};
Heads heads(PyObject* o, const char* name, const c10::Device* device, int64_t D = -1) {
  const at::Tensor& t = tensor(o, name);
  check(t, name, at::kBFloat16, device);
  if (t.dim() != 3) fail(PyExc_ValueError, "%s must have 3 dims", name);
  const Heads h{&t, t.size(0), t.size(1), t.size(2), t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2)};
  if ((h.D > 1 && t.stride(2) != 1) || (h.H > 1 && t.stride(1) != h.D) || (h.T > 1 && h.stride < h.H * h.D))
    fail(PyExc_ValueError, "%s must be [T, H, D] with dense heads", name);
  if (D >= 0 && h.D != D) fail(PyExc_ValueError, "%s must have %lld dimensions per head, got %lld", name, (long long)D, (long long)h.D);
  return h;
}

// A contiguous tensor of `dims` dimensions.
const at::Tensor& dense(PyObject* o, const char* name, at::ScalarType type, const c10::Device& device, int64_t dims = 1) {
  const at::Tensor& t = tensor(o, name);
  check(t, name, type, &device);
  if (!t.is_contiguous()) fail(PyExc_ValueError, "%s must be contiguous", name);
  if (t.dim() != dims) fail(PyExc_ValueError, "%s must have %lld dims", name, (long long)dims);
  return t;
}

int32_t as_int(int64_t x, const char* name) {
  if (x < 0 || x > 0x7FFFFFFF) fail(PyExc_ValueError, "%s is out of range", name);
  return static_cast<int32_t>(x);
}

gdn_kv_cache cache(PyObject* k_cache, PyObject* v_cache, const c10::Device& device) {
  const at::Tensor &k = tensor(k_cache, "k_cache"), &v = tensor(v_cache, "v_cache");
  check(k, "k_cache", at::kBFloat16, &device);
  check(v, "v_cache", at::kBFloat16, &device);
  if (k.dim() != 4 || (k.size(3) > 1 && k.stride(3) != 1))
    fail(PyExc_ValueError, "k_cache must be [num_pages, page_size, Hkv, D] with dense D");
  if (k.sizes() != v.sizes() || k.strides() != v.strides())
    fail(PyExc_ValueError, "k_cache and v_cache must have the same shape and strides");
  gdn_kv_cache c;
  c.k = bf16(k);
  c.v = bf16(v);
  c.num_pages = as_int(k.size(0), "num_pages");
  c.page_size = as_int(k.size(1), "page_size");
  c.num_heads = as_int(k.size(2), "Hkv");
  c.head_dim = as_int(k.size(3), "D");
  c.page_stride = k.stride(0);
  c.token_stride = k.stride(1);
  c.head_stride = k.stride(2);
  return c;
}

const int32_t* ints(const at::Tensor& t) { return static_cast<const int32_t*>(t.data_ptr()); }

// The page table, checked against T new tokens; *cu receives cu_seqlens.
gdn_page_table table(PyObject* const* a, PyObject* cu_seqlens, int64_t T, const c10::Device& device, const int32_t** cu) {
  const at::Tensor& pages = dense(a[0], "page_indices", at::kInt, device);
  const at::Tensor& indptr = dense(a[1], "page_indptr", at::kInt, device);
  const at::Tensor& last = dense(a[2], "last_page_len", at::kInt, device);
  const int64_t S = last.size(0);
  if (indptr.size(0) != S + 1) fail(PyExc_ValueError, "page_indptr must hold one entry more than last_page_len");
  *cu = nullptr;
  if (cu_seqlens == Py_None) {
    if (T != S)
      fail(PyExc_ValueError, "without cu_seqlens every sequence has one new token: got %lld tokens, %lld sequences",
           (long long)T, (long long)S);
  } else {
    const at::Tensor& c = dense(cu_seqlens, "cu_seqlens", at::kInt, device);
    if (c.size(0) != S + 1) fail(PyExc_ValueError, "cu_seqlens must hold one entry more than last_page_len");
    *cu = ints(c);
  }
  return gdn_page_table{ints(pages), as_int(pages.size(0), "page_indices"), ints(indptr), ints(last),
                        as_int(S, "last_page_len")};
}

// rotary_dim of an int64 frequency tensor (None: 0).
int32_t rotary_dim(PyObject* o, int64_t D, const c10::Device& device, const int64_t** frequencies) {
  *frequencies = nullptr;
  if (o == Py_None) return 0;
  const at::Tensor& f = dense(o, "frequencies", at::kLong, device);
  if (f.size(0) < 1 || 2 * f.size(0) > D) fail(PyExc_ValueError, "frequencies must hold between 1 and D / 2 entries");
  *frequencies = static_cast<const int64_t*>(f.data_ptr());
  return static_cast<int32_t>(2 * f.size(0));
}

at::Tensor make(at::IntArrayRef sizes, at::ScalarType type, const c10::Device& device) {
  return at::empty(sizes, at::TensorOptions().dtype(type).device(device));
}

// A dense bf16 [T, H, D] output: the caller's, or a new one.
at::Tensor output(PyObject* o, const char* name, const Heads& like, const c10::Device& device) {
  if (o == Py_None) return make({like.T, like.H, like.D}, at::kBFloat16, device);
  const at::Tensor& t = dense(o, name, at::kBFloat16, device, 3);
  if (t.size(0) != like.T || t.size(1) != like.H || t.size(2) != like.D)
    fail(PyExc_ValueError, "%s must be [%lld, %lld, %lld]", name, (long long)like.T, (long long)like.H, (long long)like.D);
  return t;
}

int32_t* err_word(PyObject* o, const c10::Device& device) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, "err_word");
  check(t, "err_word", at::kInt, &device);
  if (t.numel() < 1) fail(PyExc_ValueError, "err_word must hold an entry");
  return static_cast<int32_t*>(t.data_ptr());
}

double number(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw Raised{};
  return x;
}
int64_t whole_number(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw Raised{};
  return x;
}
bool truth(PyObject* o) {
  const int x = PyObject_IsTrue(o);
  if (x < 0) throw Raised{};
  return x != 0;
}

void ok(const char* function, int status) {
  if (status == GDN_OK) return;
  PyObject* e = g_error ? PyObject_CallFunction(g_error, "si", function, status) : nullptr;
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  } else if (!PyErr_Occurred()) {
    PyErr_Format(PyExc_RuntimeError, "%s failed: %s (status %d)", function, gdn_status_string(status), status);
  }
  throw Raised{};
}

void* stream(const c10::Device& device) { return c10::cuda::getCurrentCUDAStream(device.index()).stream(); }

void arguments(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) fail(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
}

// (x, frequencies, positions, interleaved, inverse, amplitude, out) -> out
PyObject* rope(PyObject* const* a, Py_ssize_t n) {
  arguments(n, 7);
  const Heads x = heads(a[0], "x", nullptr);
  const c10::Device device = x.t->device();
  const int64_t* frequencies;
  const int32_t rotary = rotary_dim(a[1], x.D, device, &frequencies);
  if (!rotary) fail(PyExc_ValueError, "frequencies is required");
  const at::Tensor& positions = dense(a[2], "positions", at::kInt, device);
  if (positions.size(0) != x.T) fail(PyExc_ValueError, "positions must hold one entry per token");
  at::Tensor out;
  int64_t stride = x.H * x.D;
  if (a[6] == Py_None) {
    out = make({x.T, x.H, x.D}, at::kBFloat16, device);
  } else {
    const Heads y = heads(a[6], "out", &device, x.D);
    if (y.T != x.T || y.H != x.H) fail(PyExc_ValueError, "out must have the shape of x");
    out = *y.t;
    stride = y.stride;
  }
  const c10::cuda::CUDAGuard guard(device);
  ok("gdn_rope", gdn_rope(bf16(*x.t), x.stride, bf16(out), stride, ints(positions), frequencies, as_int(x.T, "T"),
                          as_int(x.H, "H"), as_int(x.D, "D"), rotary, truth(a[3]), truth(a[4]),
                          static_cast<float>(number(a[5])), stream(device)));
  return THPVariable_Wrap(std::move(out));
}

// (k, v, k_cache, v_cache, cu_seqlens, page_indices, page_indptr, last_page_len, q,
//  frequencies, interleaved, amplitude, q_out, err_word) -> q_out or None
PyObject* kv_append(PyObject* const* a, Py_ssize_t n) {
  arguments(n, 14);
  const Heads k = heads(a[0], "k", nullptr);
  const c10::Device device = k.t->device();
  const gdn_kv_cache c = cache(a[2], a[3], device);
  const Heads v = heads(a[1], "v", &device, c.head_dim);
  if (k.D != c.head_dim) fail(PyExc_ValueError, "k must have %d dimensions per head, got %lld", c.head_dim, (long long)k.D);
  if (v.T != k.T || k.H != c.num_heads || v.H != c.num_heads) fail(PyExc_ValueError, "k and v must be [T, Hkv, D]");
  const int32_t* cu;
  const gdn_page_table t = table(a + 5, a[4], k.T, device, &cu);
  const int64_t* frequencies;
  const int32_t rotary = rotary_dim(a[9], c.head_dim, device, &frequencies);
  Heads q{nullptr, 0, 0, 0, 0};
  at::Tensor q_out;
  if (a[8] != Py_None) {
    q = heads(a[8], "q", &device, c.head_dim);
    if (q.T != k.T) fail(PyExc_ValueError, "q must hold as many tokens as k");
    q_out = output(a[12], "q_out", q, device);
  } else if (a[12] != Py_None) {
    fail(PyExc_ValueError, "q_out needs q");
  }
  const c10::cuda::CUDAGuard guard(device);
  ok("gdn_kv_append_paged",
     gdn_kv_append_paged(q.t ? bf16(*q.t) : nullptr, q.stride, q.t ? bf16(q_out) : nullptr, bf16(*k.t), k.stride,
                         bf16(*v.t), v.stride, cu, as_int(k.T, "T"), as_int(q.H, "Hq"), &c, &t, frequencies, rotary,
                         truth(a[10]), static_cast<float>(number(a[11])), err_word(a[13], device), stream(device)));
  if (!q.t) Py_RETURN_NONE;
  return THPVariable_Wrap(std::move(q_out));
}

// (decode, q, k_cache, v_cache, cu_seqlens, page_indices, page_indptr, last_page_len,
//  scale, softcap, window, slopes, full_lens, o, lse, return_lse, err_word, workspace)
// -> o or (o, lse)
PyObject* attention(PyObject* const* a, Py_ssize_t n) {
  arguments(n, 18);
  const bool decode = truth(a[0]);
  const Heads q = heads(a[1], "q", nullptr);
  const c10::Device device = q.t->device();
  const gdn_kv_cache c = cache(a[2], a[3], device);
  if (q.D != c.head_dim) fail(PyExc_ValueError, "q must have %d dimensions per head, got %lld", c.head_dim, (long long)q.D);
  const int32_t* cu;
  const gdn_page_table t = table(a + 5, a[4], q.T, device, &cu);
  gdn_attention_options options = {};
  options.softcap = static_cast<float>(number(a[9]));
  options.window = -1;
  if (a[10] != Py_None) {
    const int64_t window = whole_number(a[10]);
    options.window = window < 0 ? -1 : as_int(window, "window");
  }
  if (a[11] != Py_None) {
    const at::Tensor& slopes = dense(a[11], "slopes", at::kFloat, device);
    if (slopes.size(0) != q.H) fail(PyExc_ValueError, "slopes must hold one entry per query head");
    options.slopes = static_cast<const float*>(slopes.data_ptr());
  }
  if (a[12] != Py_None) {
    const at::Tensor& full = dense(a[12], "full_lens", at::kInt, device);
    if (full.size(0) != t.num_seqs) fail(PyExc_ValueError, "full_lens must hold one entry per sequence");
    options.full_lens = ints(full);
  }
  const int32_t T = as_int(q.T, "T"), Hq = as_int(q.H, "Hq");
  at::Tensor o = output(a[13], "o", q, device), lse;
  const bool return_lse = truth(a[15]);
  if (a[14] != Py_None) {
    lse = dense(a[14], "lse", at::kFloat, device, 2);
    if (lse.size(0) != q.T || lse.size(1) != q.H) fail(PyExc_ValueError, "lse must be [T, Hq]");
  } else if (return_lse) {
    lse = make({q.T, q.H}, at::kFloat, device);
  }
  const int64_t need = static_cast<int64_t>(
      decode ? gdn_attention_decode_workspace_bytes(t.num_seqs, Hq, c.num_heads, c.head_dim, t.num_entries, c.page_size)
             : gdn_attention_workspace_bytes(t.num_seqs, T, Hq, c.num_heads, c.head_dim, t.num_entries, c.page_size));
  at::Tensor workspace;
  if (a[17] != Py_None) {
    workspace = dense(a[17], "workspace", at::kByte, device);
    if (workspace.size(0) < need)
      fail(PyExc_ValueError, "workspace holds %lld bytes, the call needs %lld", (long long)workspace.size(0), (long long)need);
  } else if (need) {
    workspace = make({need}, at::kByte, device);
  }
  void* ws = workspace.defined() ? workspace.data_ptr() : nullptr;
  float* lse_ptr = lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr;
  const float scale = static_cast<float>(number(a[8]));
  const c10::cuda::CUDAGuard guard(device);
  if (decode)
    ok("gdn_attention_decode_paged",
       gdn_attention_decode_paged(bf16(*q.t), q.stride, bf16(o), lse_ptr, Hq, &c, &t, scale, &options, ws, need,
                                  err_word(a[16], device), stream(device)));
  else
    ok("gdn_attention_paged", gdn_attention_paged(bf16(*q.t), q.stride, bf16(o), lse_ptr, cu, T, Hq, &c, &t, scale,
                                                  &options, ws, need, err_word(a[16], device), stream(device)));
  PyObject* first = THPVariable_Wrap(std::move(o));
  if (!return_lse || !first) return first;
  PyObject* second = THPVariable_Wrap(std::move(lse));
  if (!second) {
    Py_DECREF(first);
    return nullptr;
  }
  PyObject* both = PyTuple_Pack(2, first, second);
  Py_DECREF(first);
  Py_DECREF(second);
  return both;
}

// No C++ exception leaves for the interpreter: ours carry a Python one already,
// torch's become the ones torch raises.
template <PyObject* (*kFunction)(PyObject* const*, Py_ssize_t)>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  try {
    return kFunction(args, n);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XDECREF(g_error);
  g_error = type;
  Py_RETURN_NONE;
}

#define GDN_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<f>)), METH_FASTCALL
PyMethodDef g_methods[] = {
    {"rope", GDN_FAST(rope), nullptr},
    {"kv_append", GDN_FAST(kv_append), nullptr},
    {"attention", GDN_FAST(attention), nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_attention", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attention() { return PyModule_Create(&g_module); }
