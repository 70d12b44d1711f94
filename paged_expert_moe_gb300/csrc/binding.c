/* Python binding of the calls of a decode step (moe_kv_append, moe_prefix_attention,
 * moe_sample_tokens): argument checks and marshalling only, as _lib.py does for the others
 * through ctypes. Their kernels take a few microseconds; checking a dozen tensors attribute
 * by attribute in Python and passing two dozen arguments through ctypes takes longer than
 * the launch (11.5 us a call of moe_kv_append, of which the library's part is 3.6).
 *
 * The library's entry points and torch's dtypes come in through setup(); nothing of torch is
 * included or linked. Tensors are used through their public attributes.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/pagedmoe.h"

typedef int (*append_fn)(const pmoe_kv_desc*, const void*, int64_t, const void*, int64_t, const void*, int64_t, int, int,
                         const int32_t*, int, const int32_t*, const float*, int, int, const void*, const void*, float,
                         const int32_t*, void*, int32_t*, void*);
typedef int (*attention_fn)(const pmoe_kv_desc*, const void*, int64_t, int, int, float, const int32_t*, int, const int32_t*,
                            int, int, const int32_t*, const int32_t*, int, void*, float*, void*, size_t, int32_t*, void*);
typedef size_t (*scratch_fn)(const pmoe_kv_desc*, int, int, int, int);
typedef int (*sample_fn)(const void*, int, int, int, int64_t, const float*, const int32_t*, const float*, const float*,
                         const float*, int32_t*, float*, void*);

static append_fn f_append;
static attention_fn f_attention;
static scratch_fn f_scratch;
static sample_fn f_sample;
/* torch.bfloat16, float8_e4m3fn, float32, int32, uint8; current raw stream; raw alloc, delete */
static PyObject *t_bf16, *t_e4m3, *t_f32, *t_i32, *t_u8, *p_stream, *p_alloc, *p_delete;
static PyObject *n_data_ptr, *n_dtype, *n_is_cuda, *n_numel, *n_contiguous, *n_shape, *n_stride, *n_device, *n_cuda_stream;

#define REFUSE(...)                                \
  do {                                             \
    PyErr_Format(PyExc_AssertionError, __VA_ARGS__); \
    return -1;                                     \
  } while (0)

/* A tensor's attribute or method result as a number; -1 with an error set. */
static long long as_number(PyObject* v) {
  if (v == NULL) return -1;
  const long long n = PyLong_AsLongLong(v);
  Py_DECREF(v);
  return n;
}

static int is_true(PyObject* v) {
  const int r = v == Py_True;
  Py_XDECREF(v);
  return r;
}

/* dtype (one of two; `other` may be NULL) and place of x: 0 or 1 for which of them, -1 refused. */
static int check_kind(PyObject* x, PyObject* dtype, PyObject* other, const char* name) {
  PyObject* d = PyObject_GetAttr(x, n_dtype);
  if (d == NULL) return -1;
  const int which = d == dtype ? 0 : other != NULL && d == other ? 1 : -1;
  if (which < 0) PyErr_Format(PyExc_AssertionError, "%s: dtype %S", name, d);
  Py_DECREF(d);
  if (which < 0) return -1;
  PyObject* c = PyObject_GetAttr(x, n_is_cuda);
  if (c == NULL) return -1;
  if (!is_true(c)) REFUSE("%s: not a CUDA tensor", name);
  return which;
}

static int address(PyObject* x, void** out) {
  const long long p = as_number(PyObject_CallMethodNoArgs(x, n_data_ptr));
  if (p == -1 && PyErr_Occurred()) return -1;
  *out = (void*)(uintptr_t)p;
  return 0;
}

/* The address of a contiguous tensor of n elements; NULL for None. */
static int vec(PyObject* x, PyObject* dtype, long long n, const char* name, void** out) {
  *out = NULL;
  if (x == Py_None) return 0;
  if (check_kind(x, dtype, NULL, name) < 0) return -1;
  const long long have = as_number(PyObject_CallMethodNoArgs(x, n_numel));
  if (have == -1 && PyErr_Occurred()) return -1;
  if (have != n) REFUSE("%s: %lld elements, %lld are needed", name, have, n);
  PyObject* c = PyObject_CallMethodNoArgs(x, n_contiguous);
  if (c == NULL) return -1;
  if (!is_true(c)) REFUSE("%s: not contiguous", name);
  return address(x, out);
}

/* The n numbers of a tensor's shape (method == 0) or stride. */
static int numbers(PyObject* x, int method, int n, const char* name, long long* out) {
  PyObject* t = method ? PyObject_CallMethodNoArgs(x, n_stride) : PyObject_GetAttr(x, n_shape);
  if (t == NULL) return -1;
  if (!PyTuple_Check(t) || PyTuple_GET_SIZE(t) != n) {
    Py_DECREF(t);
    REFUSE("%s: %d dimensions are needed", name, n);
  }
  for (int i = 0; i < n; ++i) out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
  Py_DECREF(t);
  return PyErr_Occurred() ? -1 : 0;
}

/* A paged cache: two tensors [pages, kv_heads, page_size, head_dim] of one type and strides,
 * contiguous but for the page stride. */
static int cache(PyObject* k, PyObject* v, PyObject* ks, PyObject* vs, pmoe_kv_desc* d) {
  long long a[4], b[4], s[4], t[4];
  const int kind = check_kind(k, t_bf16, t_e4m3, "k_cache");
  if (kind < 0) return -1;
  if (check_kind(v, kind == 0 ? t_bf16 : t_e4m3, NULL, "v_cache") < 0) return -1;
  if (numbers(k, 0, 4, "k_cache", a) || numbers(v, 0, 4, "v_cache", b) || numbers(k, 1, 4, "k_cache", s) ||
      numbers(v, 1, 4, "v_cache", t))
    return -1;
  for (int i = 0; i < 4; ++i)
    if (a[i] != b[i] || s[i] != t[i] || a[i] > INT32_MAX) REFUSE("k_cache and v_cache: different or too large");
  if (s[3] != 1 || s[2] != a[3] || s[1] != a[2] * a[3]) REFUSE("k_cache, v_cache: pages are not contiguous");
  d->num_pages = (int32_t)a[0], d->kv_heads = (int32_t)a[1], d->page_size = (int32_t)a[2], d->head_dim = (int32_t)a[3];
  d->page_stride = s[0];
  d->dtype = kind == 0 ? PMOE_KV_BF16 : PMOE_KV_E4M3;
  void *p = NULL, *q = NULL;
  if (kind == 1) {
    if (ks == Py_None || vs == Py_None) REFUSE("k_scale, v_scale: needed with an e4m3 cache");
    if (vec(ks, t_f32, a[1], "k_scale", &p) || vec(vs, t_f32, a[1], "v_scale", &q)) return -1;
  }
  d->k_scale = p, d->v_scale = q;
  if (address(k, &p) || address(v, &q)) return -1;
  d->k = p, d->v = q;
  return 0;
}

/* bf16 [T, heads, dim] with contiguous heads; *stride: elements from token to token. */
static int heads(PyObject* x, long long T, long long n, long long dim, const char* name, void** p, int64_t* stride) {
  long long a[3], s[3];
  if (check_kind(x, t_bf16, NULL, name) < 0 || numbers(x, 0, 3, name, a) || numbers(x, 1, 3, name, s)) return -1;
  if (a[0] != T || a[1] != n || a[2] != dim) REFUSE("%s: [%lld, %lld, %lld] is needed", name, T, n, dim);
  if ((s[2] != 1 && dim > 1) || (s[1] != dim && n > 1)) REFUSE("%s: heads are not contiguous", name);
  *stride = T > 1 ? s[0] : n * dim; /* one token has no stride of its own */
  return address(x, p);
}

/* The raw handle of `stream`, or of the current stream of x's device for None. */
static int raw_stream(PyObject* stream, PyObject* x, void** out) {
  PyObject* v;
  if (stream == Py_None) {
    PyObject* dev = PyObject_CallMethodNoArgs(x, n_device);
    if (dev == NULL) return -1;
    v = PyObject_CallOneArg(p_stream, dev);
    Py_DECREF(dev);
  } else {
    v = PyObject_GetAttr(stream, n_cuda_stream);
  }
  const long long s = as_number(v);
  if (s == -1 && PyErr_Occurred()) return -1;
  *out = (void*)(uintptr_t)s;
  return 0;
}

static int arity(Py_ssize_t have, Py_ssize_t need) {
  if (have == need) return 0;
  PyErr_Format(PyExc_TypeError, "%zd arguments, %zd are needed", have, need);
  return -1;
}

/* (k_cache, v_cache, q, k, v, positions, slots, inv_freq, pair_axis, interleaved, q_norm,
 *  k_norm, eps, k_scale, v_scale, q_out, err_out, stream) -> status */
static PyObject* kv_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  pmoe_kv_desc d;
  long long qs[3];
  if (arity(n, 18) || cache(a[0], a[1], a[13], a[14], &d) || numbers(a[2], 0, 3, "q", qs)) return NULL;
  const long long T = qs[0];
  if (T > INT32_MAX || qs[1] > INT32_MAX) return PyErr_Format(PyExc_AssertionError, "q: too large");
  void *q, *k, *v, *pos, *slots, *freq, *axis, *qn, *kn, *out, *err, *stream;
  int64_t q_stride, k_stride, v_stride;
  if (heads(a[2], T, qs[1], d.head_dim, "q", &q, &q_stride) || heads(a[3], T, d.kv_heads, d.head_dim, "k", &k, &k_stride) ||
      heads(a[4], T, d.kv_heads, d.head_dim, "v", &v, &v_stride))
    return NULL;
  long long axes = 1, pairs = 0;
  if (a[5] != Py_None) {
    PyObject* shape = PyObject_GetAttr(a[5], n_shape);
    if (shape == NULL) return NULL;
    if (PyTuple_Check(shape) && PyTuple_GET_SIZE(shape) == 2) axes = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 0));
    Py_DECREF(shape);
  }
  if (a[7] != Py_None) pairs = as_number(PyObject_CallMethodNoArgs(a[7], n_numel));
  if (PyErr_Occurred()) return NULL;
  if (axes > 64 || pairs > 4096) return PyErr_Format(PyExc_AssertionError, "positions, inv_freq: too large");
  const int interleaved = PyObject_IsTrue(a[9]);
  const double eps = PyFloat_AsDouble(a[12]);
  if (PyErr_Occurred()) return NULL;
  if (vec(a[5], t_i32, axes * T, "positions", &pos) || vec(a[6], t_i32, T, "slots", &slots) ||
      vec(a[7], t_f32, pairs, "inv_freq", &freq) || vec(a[8], t_i32, pairs, "pair_axis", &axis) ||
      vec(a[10], t_bf16, d.head_dim, "q_norm", &qn) || vec(a[11], t_bf16, d.head_dim, "k_norm", &kn) ||
      vec(a[15], t_bf16, T * qs[1] * d.head_dim, "q_out", &out) || vec(a[16], t_i32, 1, "err_out", &err) ||
      raw_stream(a[17], a[2], &stream))
    return NULL;
  int r;
  Py_BEGIN_ALLOW_THREADS
  r = f_append(&d, q, q_stride, k, k_stride, v, v_stride, (int)T, (int)qs[1], pos, (int)axes, axis, freq, 2 * (int)pairs,
               interleaved, qn, kn, (float)eps, slots, out, err, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(r);
}

/* (k_cache, v_cache, q, prefix_pages, prefix_len, page_table, suffix_len, max_suffix, scale,
 *  row_seq, k_scale, v_scale, out, lse_out, scratch, err_out, stream) -> status */
static PyObject* prefix_attention(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  pmoe_kv_desc d;
  long long qs[3];
  if (arity(n, 17) || cache(a[0], a[1], a[10], a[11], &d) || numbers(a[2], 0, 3, "q", qs)) return NULL;
  const long long T = qs[0], prefix = PyLong_AsLongLong(a[4]), suffix = PyLong_AsLongLong(a[7]);
  const double scale = PyFloat_AsDouble(a[8]);
  if (PyErr_Occurred()) return NULL;
  if (T > INT32_MAX || qs[1] > INT32_MAX || prefix > INT32_MAX || suffix > INT32_MAX || prefix < INT32_MIN || suffix < INT32_MIN)
    return PyErr_Format(PyExc_AssertionError, "q, prefix_len, max_suffix: too large");
  void *q, *pages = NULL, *table = NULL, *lens = NULL, *seq, *out, *lse, *work = NULL, *err, *stream;
  int64_t q_stride;
  long long shape[2] = {0, 0}, nbytes = 0;
  if (heads(a[2], T, qs[1], d.head_dim, "q", &q, &q_stride)) return NULL;
  if (prefix > 0) {
    const long long have = as_number(PyObject_CallMethodNoArgs(a[3], n_numel));
    if (PyErr_Occurred() || vec(a[3], t_i32, have, "prefix_pages", &pages)) return NULL;
    if (have * d.page_size < prefix) return PyErr_Format(PyExc_AssertionError, "prefix_pages: %lld for %lld keys", have, prefix);
  }
  if (suffix > 0) {
    if (numbers(a[5], 0, 2, "page_table", shape) || vec(a[5], t_i32, shape[0] * shape[1], "page_table", &table) ||
        vec(a[6], t_i32, T, "suffix_len", &lens))
      return NULL;
    if (shape[0] > INT32_MAX || shape[1] > INT32_MAX) return PyErr_Format(PyExc_AssertionError, "page_table: too large");
  }
  if (vec(a[9], t_i32, T, "row_seq", &seq) || vec(a[12], t_bf16, T * qs[1] * d.head_dim, "out", &out) ||
      vec(a[13], t_f32, T * qs[1], "lse_out", &lse) || vec(a[15], t_i32, 1, "err_out", &err) || raw_stream(a[16], a[2], &stream))
    return NULL;
  PyObject* own = NULL; /* the address of scratch taken here */
  if (a[14] != Py_None) {
    nbytes = as_number(PyObject_CallMethodNoArgs(a[14], n_numel));
    if (PyErr_Occurred() || vec(a[14], t_u8, nbytes, "scratch", &work)) return NULL;
  } else {
    nbytes = (long long)f_scratch(&d, (int)T, (int)qs[1], (int)prefix, (int)suffix);
    if (nbytes > 0) {
      PyObject* args[2] = {PyLong_FromLongLong(nbytes), PyLong_FromUnsignedLongLong((uintptr_t)stream)};
      if (args[0] != NULL && args[1] != NULL) own = PyObject_Vectorcall(p_alloc, args, 2, NULL);
      Py_XDECREF(args[0]);
      Py_XDECREF(args[1]);
      if (own == NULL) return NULL;
      work = (void*)(uintptr_t)PyLong_AsUnsignedLongLong(own);
    }
  }
  int r;
  Py_BEGIN_ALLOW_THREADS
  r = f_attention(&d, q, q_stride, (int)T, (int)qs[1], (float)scale, pages, (int)prefix, table, (int)shape[1], (int)shape[0],
                  seq, lens, (int)suffix, out, lse, work, (size_t)nbytes, err, stream);
  Py_END_ALLOW_THREADS
  if (own != NULL) {
    /* what reuses the block on this stream runs after the launches */
    PyObject* none = PyObject_CallOneArg(p_delete, own);
    Py_DECREF(own);
    if (none == NULL) return NULL;
    Py_DECREF(none);
  }
  return PyLong_FromLong(r);
}

/* (logits, u, temperature, top_k, top_p, min_p, ids_out, logprob_out, stream) -> status */
static PyObject* sample_tokens(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (arity(n, 9)) return NULL;
  long long shape[2], stride[2];
  const int kind = check_kind(a[0], t_f32, t_bf16, "logits");
  if (kind < 0 || numbers(a[0], 0, 2, "logits", shape) || numbers(a[0], 1, 2, "logits", stride)) return NULL;
  const long long T = shape[0], V = shape[1];
  if (T > INT32_MAX || V > INT32_MAX) return PyErr_Format(PyExc_AssertionError, "logits: too large");
  if (V > 1 && stride[1] != 1) return PyErr_Format(PyExc_AssertionError, "logits: rows are not contiguous");
  if (a[1] == Py_None) return PyErr_Format(PyExc_AssertionError, "u: needed");
  void *x, *u, *temp, *k, *p, *m, *ids, *lp, *stream;
  if (address(a[0], &x) || vec(a[1], t_f32, T, "u", &u) || vec(a[2], t_f32, T, "temperature", &temp) ||
      vec(a[3], t_i32, T, "top_k", &k) || vec(a[4], t_f32, T, "top_p", &p) || vec(a[5], t_f32, T, "min_p", &m) ||
      vec(a[6], t_i32, T, "ids_out", &ids) || vec(a[7], t_f32, T, "logprob_out", &lp) || raw_stream(a[8], a[0], &stream))
    return NULL;
  int r;
  Py_BEGIN_ALLOW_THREADS
  r = f_sample(x, kind, (int)T, (int)V, T > 1 ? stride[0] : V, temp, k, p, m, u, ids, lp, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(r);
}

/* setup((append, attention, scratch, sample addresses), (bf16, e4m3, f32, i32, u8 dtypes),
 *       current raw stream, raw alloc, raw delete) */
static PyObject* setup(PyObject* self, PyObject* args) {
  (void)self;
  unsigned long long f[4];
  PyObject *t[5], *s, *al, *de;
  if (!PyArg_ParseTuple(args, "(KKKK)(OOOOO)OOO", &f[0], &f[1], &f[2], &f[3], &t[0], &t[1], &t[2], &t[3], &t[4], &s, &al, &de))
    return NULL;
  f_append = (append_fn)(uintptr_t)f[0];
  f_attention = (attention_fn)(uintptr_t)f[1];
  f_scratch = (scratch_fn)(uintptr_t)f[2];
  f_sample = (sample_fn)(uintptr_t)f[3];
  PyObject** slot[8] = {&t_bf16, &t_e4m3, &t_f32, &t_i32, &t_u8, &p_stream, &p_alloc, &p_delete};
  PyObject* value[8] = {t[0], t[1], t[2], t[3], t[4], s, al, de};
  for (int i = 0; i < 8; ++i) {
    Py_INCREF(value[i]);
    Py_XSETREF(*slot[i], value[i]);
  }
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"setup", setup, METH_VARARGS, "entry points and dtypes"},
    {"kv_append", (PyCFunction)(void (*)(void))kv_append, METH_FASTCALL, "moe_kv_append"},
    {"prefix_attention", (PyCFunction)(void (*)(void))prefix_attention, METH_FASTCALL, "moe_prefix_attention"},
    {"sample_tokens", (PyCFunction)(void (*)(void))sample_tokens, METH_FASTCALL, "moe_sample_tokens"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "binding of the decode-step calls", -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
  PyObject** slot[9] = {&n_data_ptr, &n_dtype, &n_is_cuda, &n_numel, &n_contiguous, &n_shape, &n_stride, &n_device, &n_cuda_stream};
  const char* name[9] = {"data_ptr", "dtype", "is_cuda", "numel", "is_contiguous", "shape", "stride", "get_device", "cuda_stream"};
  for (int i = 0; i < 9; ++i)
    if ((*slot[i] = PyUnicode_InternFromString(name[i])) == NULL) return NULL;
  return PyModule_Create(&module);
}
