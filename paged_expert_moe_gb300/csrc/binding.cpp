// Python binding of the calls of a serving step (moe_kv_append, moe_prefix_attention,
// moe_sample_tokens, moe_batch_tables, moe_chunk_attention, moe_router_select, moe_adjust_logits):
// argument checks and marshalling only, as _lib.py does for the others through ctypes. Their kernels
// take a few microseconds. A call of moe_kv_append, of which the
// library's part is 1.7 us, issues in 11.5 us through ctypes, in 5.4 when a dozen tensors are
// asked for their attributes one by one from C, in 2.15 here, where they are at::Tensors.
//
// The library's entry points come in through setup(). Refused arguments raise AssertionError;
// what torch throws (an allocation that fails) is raised as its own Python exception.
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>

#include "attn_plan.h"

namespace {

decltype(&moe_kv_append) f_append;
decltype(&moe_prefix_attention) f_attention;
decltype(&pmoe_attention_plan) f_plan;
decltype(&moe_sample_tokens) f_sample;
decltype(&moe_batch_tables) f_tables;
decltype(&moe_chunk_attention) f_chunk;
decltype(&moe_chunk_attention_scratch_bytes) f_chunk_bytes;
decltype(&moe_router_select) f_select;
decltype(&moe_adjust_logits) f_adjust;
PyObject *n_cuda_stream, *n_device_index;

struct Refused {};  // a Python error is set

[[noreturn]] void refuse(const char* format, ...) {
  va_list v;
  va_start(v, format);
  PyErr_FormatV(PyExc_AssertionError, format, v);
  va_end(v);
  throw Refused{};
}

// Every entry: refusals and C++ exceptions leave it as Python errors.
template <class F>
PyObject* guarded(F&& f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// The device of a call, which its first argument, a CUDA tensor, gives: every other tensor has
// to be there too, and the stream (the last argument), since the kernels read all of them from
// one device. Before anything else is asked of the tensors.
c10::DeviceIndex place(PyObject* const* a, Py_ssize_t n, const char* const* names) {
  if (!THPVariable_Check(a[0]) || !THPVariable_Unpack(a[0]).defined()) refuse("%s: not a tensor", names[0]);
  const at::Device d = THPVariable_Unpack(a[0]).device();
  if (!d.is_cuda()) refuse("%s: not a CUDA tensor", names[0]);
  for (Py_ssize_t i = 1; i + 1 < n; ++i) {
    // (the check of what is no tensor is slow, and most arguments that are none are these: with it,
    // and a device guard that always asks twice, moe_kv_append issues in 2.65 us instead of 2.15)
    if (a[i] == Py_None || PyLong_Check(a[i]) || PyFloat_Check(a[i])) continue;
    if (!THPVariable_Check(a[i]) || !THPVariable_Unpack(a[i]).defined()) continue;
    const at::Device o = THPVariable_Unpack(a[i]).device();
    if (o != d) refuse("%s: on %s, %s on %s", names[i], o.str().c_str(), names[0], d.str().c_str());
  }
  if (a[n - 1] != Py_None) {
    PyObject* v = PyObject_GetAttr(a[n - 1], n_device_index);
    if (v == nullptr) {  // another library's stream, which need not say
      if (!PyErr_ExceptionMatches(PyExc_AttributeError)) throw Refused{};
      PyErr_Clear();
      return d.index();
    }
    const long long index = PyLong_AsLongLong(v);
    Py_DECREF(v);
    if (index == -1 && PyErr_Occurred()) throw Refused{};
    if (index != d.index()) refuse("stream: of cuda:%lld, %s on %s", index, names[0], d.str().c_str());
  }
  return d.index();
}

// A tensor of one of two types.
const at::Tensor& tensor(PyObject* x, const char* name, at::ScalarType type, at::ScalarType other) {
  if (!THPVariable_Check(x)) refuse("%s: not a tensor", name);
  const at::Tensor& t = THPVariable_Unpack(x);
  if (!t.defined()) refuse("%s: not a tensor", name);
  if (t.scalar_type() != type && t.scalar_type() != other) refuse("%s: dtype %s", name, c10::toString(t.scalar_type()));
  return t;
}
const at::Tensor& tensor(PyObject* x, const char* name, at::ScalarType type, at::ScalarType other, int64_t dims) {
  const at::Tensor& t = tensor(x, name, type, other);
  if (t.dim() != dims) refuse("%s: %lld dimensions are needed", name, (long long)dims);
  return t;
}

// The address of a contiguous tensor of n elements; null for None.
template <class T = void>
T* vec(PyObject* x, at::ScalarType type, int64_t n, const char* name) {
  if (x == Py_None) return nullptr;
  const at::Tensor& t = tensor(x, name, type, type);
  if (t.numel() != n) refuse("%s: %lld elements, %lld are needed", name, (long long)t.numel(), (long long)n);
  if (!t.is_contiguous()) refuse("%s: not contiguous", name);
  return static_cast<T*>(t.data_ptr());
}

// Elements from page to page of [pages, kv_heads, page_size, head_dim], contiguous but for that
// stride. A dimension of size 1 has no stride of its own, whatever torch keeps there.
int64_t page_stride(const at::Tensor& t) {
  const auto a = t.sizes(), s = t.strides();
  const int64_t page = a[1] * a[2] * a[3];
  if ((a[3] > 1 && s[3] != 1) || (a[2] > 1 && s[2] != a[3]) || (a[1] > 1 && s[1] != a[2] * a[3]))
    refuse("k_cache, v_cache: pages are not contiguous");
  return a[0] > 1 ? s[0] : page;
}

// A paged cache: two such tensors of one type, size and page stride.
pmoe_kv_desc cache(PyObject* k_cache, PyObject* v_cache, PyObject* k_scale, PyObject* v_scale) {
  const at::Tensor& k = tensor(k_cache, "k_cache", at::kBFloat16, at::kFloat8_e4m3fn, 4);
  const at::Tensor& v = tensor(v_cache, "v_cache", k.scalar_type(), k.scalar_type(), 4);
  const auto a = k.sizes();
  for (const int64_t n : a)
    if (n > INT32_MAX) refuse("k_cache, v_cache: too large");
  pmoe_kv_desc d{};
  d.page_stride = page_stride(k);
  if (a != v.sizes() || d.page_stride != page_stride(v)) refuse("k_cache and v_cache: different");
  d.num_pages = (int32_t)a[0], d.kv_heads = (int32_t)a[1], d.page_size = (int32_t)a[2], d.head_dim = (int32_t)a[3];
  d.dtype = k.scalar_type() == at::kBFloat16 ? PMOE_KV_BF16 : PMOE_KV_E4M3;
  if (d.dtype == PMOE_KV_E4M3) {
    if (k_scale == Py_None || v_scale == Py_None) refuse("k_scale, v_scale: needed with an e4m3 cache");
    d.k_scale = vec<float>(k_scale, at::kFloat, a[1], "k_scale");
    d.v_scale = vec<float>(v_scale, at::kFloat, a[1], "v_scale");
  }
  d.k = k.data_ptr(), d.v = v.data_ptr();
  return d;
}

// bf16 [T, heads, dim] with contiguous heads.
struct Heads {
  void* p;
  int64_t stride;  // elements from token to token
  Heads(PyObject* x, const char* name, int64_t T, int64_t n, int64_t dim) {
    const at::Tensor& t = tensor(x, name, at::kBFloat16, at::kBFloat16, 3);
    const auto a = t.sizes(), s = t.strides();
    if (a[0] != T || a[1] != n || a[2] != dim)
      refuse("%s: [%lld, %lld, %lld] is needed", name, (long long)T, (long long)n, (long long)dim);
    if ((s[2] != 1 && dim > 1) || (s[1] != dim && n > 1)) refuse("%s: heads are not contiguous", name);
    stride = T > 1 ? s[0] : n * dim;  // one token has no stride of its own
    p = t.data_ptr();
  }
};

// Makes the call's device the current one where it is not.
struct OnDevice {
  c10::cuda::OptionalCUDAGuard guard;
  explicit OnDevice(c10::DeviceIndex device) {
    if (c10::cuda::current_device() != device) guard.set_index(device);
  }
};

// The raw handle of `stream`, or of the device's current one for None.
cudaStream_t raw_stream(PyObject* stream, c10::DeviceIndex device) {
  if (stream == Py_None) return c10::cuda::getCurrentCUDAStream(device).stream();
  PyObject* v = PyObject_GetAttr(stream, n_cuda_stream);
  if (v == nullptr) throw Refused{};
  const long long s = PyLong_AsLongLong(v);
  Py_DECREF(v);
  if (s == -1 && PyErr_Occurred()) throw Refused{};
  return reinterpret_cast<cudaStream_t>(static_cast<uintptr_t>(s));
}

long long integer(PyObject* x, const char* name) {
  const long long n = PyLong_AsLongLong(x);
  if (n == -1 && PyErr_Occurred()) throw Refused{};
  if (n > INT32_MAX || n < INT32_MIN) refuse("%s: too large", name);
  return n;
}
double real(PyObject* x) {
  const double v = PyFloat_AsDouble(x);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}
void arity(Py_ssize_t have, Py_ssize_t need) {
  if (have == need) return;
  PyErr_Format(PyExc_TypeError, "%zd arguments, %zd are needed", have, need);
  throw Refused{};
}

// (k_cache, v_cache, q, k, v, positions, slots, inv_freq, pair_axis, interleaved, q_norm, k_norm,
//  eps, k_scale, v_scale, q_out, err_out, stream) -> status
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 18);
    static const char* const names[18] = {"k_cache", "v_cache", "q", "k", "v", "positions", "slots", "inv_freq", "pair_axis",
                                          "interleaved", "q_norm", "k_norm", "eps", "k_scale", "v_scale", "q_out", "err_out",
                                          "stream"};
    const c10::DeviceIndex device = place(a, n, names);
    const pmoe_kv_desc d = cache(a[0], a[1], a[13], a[14]);
    const at::Tensor& tq = tensor(a[2], "q", at::kBFloat16, at::kBFloat16, 3);
    const int64_t T = tq.size(0), q_heads = tq.size(1);
    if (T > INT32_MAX || q_heads > INT32_MAX) refuse("q: too large");
    const Heads q(a[2], "q", T, q_heads, d.head_dim), k(a[3], "k", T, d.kv_heads, d.head_dim),
        v(a[4], "v", T, d.kv_heads, d.head_dim);
    int64_t axes = 1, pairs = 0;
    if (a[5] != Py_None) {
      const at::Tensor& t = tensor(a[5], "positions", at::kInt, at::kInt);
      if (t.dim() == 2) axes = t.size(0);
    }
    if (a[7] != Py_None) pairs = tensor(a[7], "inv_freq", at::kFloat, at::kFloat).numel();
    if (axes > 64 || pairs > 4096) refuse("positions, inv_freq: too large");
    const int interleaved = PyObject_IsTrue(a[9]);
    if (interleaved < 0) throw Refused{};
    const float eps = (float)real(a[12]);
    const auto* pos = vec<int32_t>(a[5], at::kInt, axes * T, "positions");
    const auto* slots = vec<int32_t>(a[6], at::kInt, T, "slots");
    const auto* freq = vec<float>(a[7], at::kFloat, pairs, "inv_freq");
    const auto* axis = vec<int32_t>(a[8], at::kInt, pairs, "pair_axis");
    const auto* qn = vec(a[10], at::kBFloat16, d.head_dim, "q_norm");
    const auto* kn = vec(a[11], at::kBFloat16, d.head_dim, "k_norm");
    auto* out = vec(a[15], at::kBFloat16, T * q_heads * d.head_dim, "q_out");
    auto* err = vec<int32_t>(a[16], at::kInt, 1, "err_out");
    const cudaStream_t stream = raw_stream(a[17], device);
    const OnDevice on(device);
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = f_append(&d, q.p, q.stride, k.p, k.stride, v.p, v.stride, (int)T, (int)q_heads, pos, (int)axes, axis, freq,
                 2 * (int)pairs, interleaved, qn, kn, eps, slots, out, err, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(r);
  });
}

// (k_cache, v_cache, q, prefix_pages, prefix_len, page_table, suffix_len, max_suffix, scale,
//  row_seq, k_scale, v_scale, out, lse_out, scratch, err_out, stream) -> status
PyObject* prefix_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 17);
    static const char* const names[17] = {"k_cache", "v_cache", "q", "prefix_pages", "prefix_len", "page_table", "suffix_len",
                                          "max_suffix", "scale", "row_seq", "k_scale", "v_scale", "out", "lse_out", "scratch",
                                          "err_out", "stream"};
    const c10::DeviceIndex device = place(a, n, names);
    const pmoe_kv_desc d = cache(a[0], a[1], a[10], a[11]);
    const at::Tensor& tq = tensor(a[2], "q", at::kBFloat16, at::kBFloat16, 3);
    const int64_t T = tq.size(0), q_heads = tq.size(1);
    const long long prefix = integer(a[4], "prefix_len"), suffix = integer(a[7], "max_suffix");
    const double scale = a[8] == Py_None ? 1.0 / std::sqrt((double)d.head_dim) : real(a[8]);
    if (T > INT32_MAX || q_heads > INT32_MAX) refuse("q: too large");
    const Heads q(a[2], "q", T, q_heads, d.head_dim);
    const int32_t *pages = nullptr, *table = nullptr, *lens = nullptr;
    int64_t sequences = 0, width = 0;
    if (prefix > 0 && a[3] != Py_None) {
      const int64_t have = tensor(a[3], "prefix_pages", at::kInt, at::kInt).numel();
      pages = vec<int32_t>(a[3], at::kInt, have, "prefix_pages");
      if (have * d.page_size < prefix) refuse("prefix_pages: %lld for %lld keys", (long long)have, prefix);
    }
    if (suffix > 0 && a[5] != Py_None) {
      const at::Tensor& t = tensor(a[5], "page_table", at::kInt, at::kInt, 2);
      sequences = t.size(0), width = t.size(1);
      table = vec<int32_t>(a[5], at::kInt, sequences * width, "page_table");
      lens = vec<int32_t>(a[6], at::kInt, T, "suffix_len");
      if (sequences > INT32_MAX || width > INT32_MAX) refuse("page_table: too large");
    }
    const auto* seq = vec<int32_t>(a[9], at::kInt, T, "row_seq");
    auto* out = vec(a[12], at::kBFloat16, T * q_heads * d.head_dim, "out");
    auto* lse = vec<float>(a[13], at::kFloat, T * q_heads, "lse_out");
    auto* err = vec<int32_t>(a[15], at::kInt, 1, "err_out");
    const cudaStream_t stream = raw_stream(a[16], device);
    const OnDevice on(device);
    void *work = nullptr, *own = nullptr;  // scratch, and what of it was taken here
    int64_t bytes;
    if (a[14] != Py_None) {
      bytes = tensor(a[14], "scratch", at::kByte, at::kByte).numel();
      work = vec(a[14], at::kByte, bytes, "scratch");
    } else {
      pmoe_attention_plan_desc p;
      f_plan(&d, (int)T, (int)q_heads, (int)prefix, (int)suffix, 0, &p);  // (0 bytes where the call refuses)
      bytes = (int64_t)p.scratch_bytes;
      if (bytes > 0) work = own = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(bytes, stream);
    }
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = f_attention(&d, q.p, q.stride, (int)T, (int)q_heads, (float)scale, pages, (int)prefix, table, (int)width,
                    (int)sequences, seq, lens, (int)suffix, out, lse, work, (size_t)bytes, err, stream);
    Py_END_ALLOW_THREADS
    // what reuses the block on this stream runs after the launches
    if (own != nullptr) c10::cuda::CUDACachingAllocator::raw_delete(own);
    return PyLong_FromLong(r);
  });
}

// (logits, u, temperature, top_k, top_p, min_p, ids_out, logprob_out, stream) -> status
PyObject* sample_tokens(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 9);
    static const char* const names[9] = {"logits", "u", "temperature", "top_k", "top_p", "min_p", "ids_out", "logprob_out",
                                         "stream"};
    const c10::DeviceIndex device = place(a, n, names);
    const at::Tensor& x = tensor(a[0], "logits", at::kFloat, at::kBFloat16, 2);
    const int64_t T = x.size(0), V = x.size(1);
    if (T > INT32_MAX || V > INT32_MAX) refuse("logits: too large");
    if (V > 1 && x.stride(1) != 1) refuse("logits: rows are not contiguous");
    if (a[1] == Py_None) refuse("u: needed");
    const auto* u = vec<float>(a[1], at::kFloat, T, "u");
    const auto* temp = vec<float>(a[2], at::kFloat, T, "temperature");
    const auto* k = vec<int32_t>(a[3], at::kInt, T, "top_k");
    const auto* p = vec<float>(a[4], at::kFloat, T, "top_p");
    const auto* m = vec<float>(a[5], at::kFloat, T, "min_p");
    auto* ids = vec<int32_t>(a[6], at::kInt, T, "ids_out");
    auto* lp = vec<float>(a[7], at::kFloat, T, "logprob_out");
    const cudaStream_t stream = raw_stream(a[8], device);
    const int64_t row = T > 1 ? x.stride(0) : V;
    const void* logits = x.data_ptr();
    const int bf16 = x.scalar_type() == at::kBFloat16;
    const OnDevice on(device);
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = f_sample(logits, bf16, (int)T, (int)V, row, temp, k, p, m, u, ids, lp, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(r);
  });
}

// [T][width] with contiguous rows, some stride apart.
struct Rows {
  void* p = nullptr;
  int64_t width = 0, stride = 0;
  Rows(PyObject* x, const char* name, at::ScalarType type, at::ScalarType other, int64_t T) {
    if (x == Py_None) return;
    const at::Tensor& t = tensor(x, name, type, other, 2);
    if (T >= 0 && t.size(0) != T) refuse("%s: %lld rows, %lld are needed", name, (long long)t.size(0), (long long)T);
    width = t.size(1);
    if (width > INT32_MAX || t.size(0) > INT32_MAX) refuse("%s: too large", name);
    if (width > 1 && t.stride(1) != 1) refuse("%s: rows are not contiguous", name);
    stride = t.size(0) > 1 ? t.stride(0) : width;  // a single row has no stride
    p = t.data_ptr();
  }
};

int32_t* ints(PyObject* x, int64_t n, const char* name) {
  if (x == Py_None) refuse("%s: needed", name);
  return vec<int32_t>(x, at::kInt, n, name);
}

// (page_table, free_pages, free_count, lens, new_len, T, page_size, num_pages, lens_out, free_count_out,
//  q_start, positions, slots, row_seq, row_len, err_out, stream) -> status
PyObject* batch_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 17);
    static const char* const names[17] = {"page_table", "free_pages", "free_count", "lens", "new_len", "T", "page_size",
                                          "num_pages", "lens_out", "free_count_out", "q_start", "positions", "slots",
                                          "row_seq", "row_len", "err_out", "stream"};
    const c10::DeviceIndex device = place(a, n, names);
    const at::Tensor& table = tensor(a[0], "page_table", at::kInt, at::kInt, 2);
    const int64_t R = table.size(0), width = table.size(1);
    if (R > INT32_MAX || width > INT32_MAX) refuse("page_table: too large");
    auto* pt = ints(a[0], R * width, "page_table");
    const int64_t capacity = tensor(a[1], "free_pages", at::kInt, at::kInt).numel();
    if (capacity > INT32_MAX) refuse("free_pages: too large");
    auto* free_pages = ints(a[1], capacity, "free_pages");
    const auto *count = ints(a[2], 1, "free_count"), *lens = ints(a[3], R, "lens"), *new_len = ints(a[4], R, "new_len");
    const long long T = integer(a[5], "T"), page = integer(a[6], "page_size"), pages = integer(a[7], "num_pages");
    auto *lens_out = ints(a[8], R, "lens_out"), *count_out = ints(a[9], 1, "free_count_out"),
         *start = ints(a[10], R + 1, "q_start"), *positions = ints(a[11], T, "positions"), *slots = ints(a[12], T, "slots"),
         *row_seq = ints(a[13], T, "row_seq"), *row_len = vec<int32_t>(a[14], at::kInt, T, "row_len"),
         *err = vec<int32_t>(a[15], at::kInt, 1, "err_out");
    const cudaStream_t stream = raw_stream(a[16], device);
    const OnDevice on(device);
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = f_tables(pt, (int)width, (int)page, (int)pages, free_pages, (int)capacity, count, lens, new_len, (int)R, (int)T,
                 lens_out, count_out, start, positions, slots, row_seq, row_len, err, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(r);
  });
}

// (k_cache, v_cache, q, q_start, kv_len, page_table, window, sinks, scale, k_scale, v_scale, out, lse_out,
//  scratch, err_out, stream) -> status
PyObject* chunk_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 16);
    static const char* const names[16] = {"k_cache", "v_cache", "q", "q_start", "kv_len", "page_table", "window", "sinks",
                                          "scale", "k_scale", "v_scale", "out", "lse_out", "scratch", "err_out", "stream"};
    const c10::DeviceIndex device = place(a, n, names);
    const pmoe_kv_desc d = cache(a[0], a[1], a[9], a[10]);
    const at::Tensor& tq = tensor(a[2], "q", at::kBFloat16, at::kBFloat16, 3);
    const int64_t T = tq.size(0), q_heads = tq.size(1);
    if (T > INT32_MAX || q_heads > INT32_MAX) refuse("q: too large");
    const Heads q(a[2], "q", T, q_heads, d.head_dim);
    const at::Tensor& table = tensor(a[5], "page_table", at::kInt, at::kInt, 2);
    const int64_t R = table.size(0), width = table.size(1);
    if (R > INT32_MAX || width > INT32_MAX) refuse("page_table: too large");
    const auto *pt = ints(a[5], R * width, "page_table"), *start = ints(a[3], R + 1, "q_start"), *lens = ints(a[4], R, "kv_len");
    const long long window = integer(a[6], "window"), sinks = integer(a[7], "sinks");
    const double scale = a[8] == Py_None ? 1.0 / std::sqrt((double)d.head_dim) : real(a[8]);
    auto* out = vec(a[11], at::kBFloat16, T * q_heads * d.head_dim, "out");
    auto* lse = vec<float>(a[12], at::kFloat, T * q_heads, "lse_out");
    auto* err = vec<int32_t>(a[14], at::kInt, 1, "err_out");
    const cudaStream_t stream = raw_stream(a[15], device);
    const OnDevice on(device);
    void *work = nullptr, *own = nullptr;  // scratch, and what of it was taken here
    int64_t bytes;
    if (a[13] != Py_None) {
      bytes = tensor(a[13], "scratch", at::kByte, at::kByte).numel();
      work = vec(a[13], at::kByte, bytes, "scratch");
    } else {
      bytes = (int64_t)f_chunk_bytes(&d, (int)T, (int)q_heads, (int)R);  // (0 where the call refuses)
      if (bytes > 0) work = own = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(bytes, stream);
    }
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = f_chunk(&d, q.p, q.stride, (int)T, (int)q_heads, (float)scale, start, lens, (int)R, pt, (int)width, (int)window,
                (int)sinks, out, lse, work, (size_t)bytes, err, stream);
    Py_END_ALLOW_THREADS
    // what reuses the block on this stream runs after the launches
    if (own != nullptr) c10::cuda::CUDACachingAllocator::raw_delete(own);
    return PyLong_FromLong(r);
  });
}

// (logits, bias, top_k, scoring, groups, top_groups, group_top, renormalize, scale, ids_out, w_out, stream)
// -> status
PyObject* router_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 12);
    static const char* const names[12] = {"logits", "bias", "top_k", "scoring", "groups", "top_groups", "group_top",
                                          "renormalize", "scale", "ids_out", "w_out", "stream"};
    const c10::DeviceIndex device = place(a, n, names);
    const Rows x(a[0], "logits", at::kFloat, at::kBFloat16, -1);
    const at::Tensor& t = THPVariable_Unpack(a[0]);
    const int64_t T = t.size(0);
    const auto* bias = vec<float>(a[1], at::kFloat, x.width, "bias");
    const long long k = integer(a[2], "top_k"), scoring = integer(a[3], "scoring"), groups = integer(a[4], "groups"),
                    top_groups = integer(a[5], "top_groups"), group_top = integer(a[6], "group_top");
    const int renorm = PyObject_IsTrue(a[7]);
    if (renorm < 0) throw Refused{};
    const float scale = (float)real(a[8]);
    auto* ids = ints(a[9], T * k, "ids_out");
    if (a[10] == Py_None) refuse("w_out: needed");
    auto* w = vec<float>(a[10], at::kFloat, T * k, "w_out");
    const cudaStream_t stream = raw_stream(a[11], device);
    const int bf16 = t.scalar_type() == at::kBFloat16;
    const OnDevice on(device);
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = f_select(x.p, bf16, (int)T, (int)x.width, x.stride, (int)k, (int)scoring, bias, (int)groups, (int)top_groups,
                 (int)group_top, renorm, scale, ids, w, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(r);
  });
}

// (logits, history, prompt_len, history_len, repetition, frequency, presence, bias_ids, bias, mask, out,
//  err_out, stream) -> status
PyObject* adjust_logits(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    arity(n, 13);
    static const char* const names[13] = {"logits", "history", "prompt_len", "history_len", "repetition", "frequency",
                                          "presence", "bias_ids", "bias", "mask", "out", "err_out", "stream"};
    const c10::DeviceIndex device = place(a, n, names);
    const Rows x(a[0], "logits", at::kFloat, at::kBFloat16, -1);
    const at::Tensor& t = THPVariable_Unpack(a[0]);
    const int64_t T = t.size(0);
    const Rows history(a[1], "history", at::kInt, at::kInt, T);
    if (a[1] != Py_None && a[3] == Py_None) refuse("history_len: needed with a history");
    const auto *prompt = vec<int32_t>(a[2], at::kInt, T, "prompt_len"), *len = vec<int32_t>(a[3], at::kInt, T, "history_len");
    const auto *rep = vec<float>(a[4], at::kFloat, T, "repetition"), *freq = vec<float>(a[5], at::kFloat, T, "frequency"),
               *pres = vec<float>(a[6], at::kFloat, T, "presence");
    int64_t biases = 0;
    const int32_t* bias_ids = nullptr;
    const float* bias = nullptr;
    if (a[7] != Py_None || a[8] != Py_None) {
      if (a[7] == Py_None || a[8] == Py_None) refuse("bias_ids, bias: one without the other");
      const Rows ids(a[7], "bias_ids", at::kInt, at::kInt, T);
      biases = ids.width;
      bias_ids = vec<int32_t>(a[7], at::kInt, T * biases, "bias_ids");
      const Rows values(a[8], "bias", at::kFloat, at::kFloat, T);
      bias = vec<float>(a[8], at::kFloat, T * biases, "bias");
    }
    const Rows mask(a[9], "mask", at::kInt, at::kInt, T);
    if (a[9] != Py_None && mask.width < (x.width + 31) / 32)
      refuse("mask: %lld words a row for %lld tokens", (long long)mask.width, (long long)x.width);
    if (a[10] == Py_None) refuse("out: needed");
    const Rows out(a[10], "out", at::kFloat, at::kBFloat16, T);
    if (out.width != x.width) refuse("out: %lld tokens, %lld are needed", (long long)out.width, (long long)x.width);
    auto* err = vec<int32_t>(a[11], at::kInt, 1, "err_out");
    const cudaStream_t stream = raw_stream(a[12], device);
    const int bf16 = t.scalar_type() == at::kBFloat16, out_bf16 = THPVariable_Unpack(a[10]).scalar_type() == at::kBFloat16;
    const int64_t mask_stride = T > 1 ? mask.stride : mask.width;
    const OnDevice on(device);
    int r;
    Py_BEGIN_ALLOW_THREADS
    r = f_adjust(x.p, bf16, (int)T, (int)x.width, x.stride, static_cast<const int32_t*>(history.p), history.stride,
                 (int)history.width, prompt, len, rep, freq, pres, bias_ids, bias, (int)biases,
                 static_cast<const uint32_t*>(mask.p), mask_stride, out.p, out_bf16, out.stride, err, stream);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(r);
  });
}

// setup(the library's entry points, in the order below)
PyObject* setup(PyObject*, PyObject* args) {
  unsigned long long f[9];
  if (!PyArg_ParseTuple(args, "(KKKKKKKKK)", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &f[6], &f[7], &f[8])) return nullptr;
  f_append = reinterpret_cast<decltype(f_append)>((uintptr_t)f[0]);
  f_attention = reinterpret_cast<decltype(f_attention)>((uintptr_t)f[1]);
  f_plan = reinterpret_cast<decltype(f_plan)>((uintptr_t)f[2]);
  f_sample = reinterpret_cast<decltype(f_sample)>((uintptr_t)f[3]);
  f_tables = reinterpret_cast<decltype(f_tables)>((uintptr_t)f[4]);
  f_chunk = reinterpret_cast<decltype(f_chunk)>((uintptr_t)f[5]);
  f_chunk_bytes = reinterpret_cast<decltype(f_chunk_bytes)>((uintptr_t)f[6]);
  f_select = reinterpret_cast<decltype(f_select)>((uintptr_t)f[7]);
  f_adjust = reinterpret_cast<decltype(f_adjust)>((uintptr_t)f[8]);
  Py_RETURN_NONE;
}

PyCFunction fast(PyObject* (*f)(PyObject*, PyObject* const*, Py_ssize_t)) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}
PyMethodDef methods[] = {{"setup", setup, METH_VARARGS, "entry points"},
                         {"kv_append", fast(kv_append), METH_FASTCALL, "moe_kv_append"},
                         {"prefix_attention", fast(prefix_attention), METH_FASTCALL, "moe_prefix_attention"},
                         {"sample_tokens", fast(sample_tokens), METH_FASTCALL, "moe_sample_tokens"},
                         {"batch_tables", fast(batch_tables), METH_FASTCALL, "moe_batch_tables"},
                         {"chunk_attention", fast(chunk_attention), METH_FASTCALL, "moe_chunk_attention"},
                         {"router_select", fast(router_select), METH_FASTCALL, "moe_router_select"},
                         {"adjust_logits", fast(adjust_logits), METH_FASTCALL, "moe_adjust_logits"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "binding of the serving-step calls", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) {
  n_cuda_stream = PyUnicode_InternFromString("cuda_stream");
  n_device_index = PyUnicode_InternFromString("device_index");
  return n_cuda_stream == nullptr || n_device_index == nullptr ? nullptr : PyModule_Create(&module);
}
