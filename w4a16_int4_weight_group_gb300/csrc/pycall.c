/*
 * CPython entry points for the prepared-layer call and the serving operators of libw4a16.so: convert
 * their arguments and call them through function pointers that the Python binding resolves once from
 * the library (ctypes) and hands over with bind() and bind_serving(). Argument marshalling only:
 * no computation happens here. It exists because a ctypes call converts its arguments through
 * per-argument Python objects, which costs more host time per call than the small decode kernels
 * take on the GPU.
 *
 *   bind(address)                                    address of w4a16_layer_gemm
 *   layer_gemm(layer, a, out, m, ws, ws_bytes, stream) -> status (int)
 *     layer, a, out, ws, stream: integers (addresses; None or 0 for a null pointer);
 *     m: int64; ws_bytes: size_t. The GIL is released around the call.
 *
 *   bind_capture(address), capture_id(stream) -> int  w4a16_stream_capture_id
 *
 *   bind_serving(rope, kv_write, kv_read, tree_attention_fill, token_logprobs)   addresses of the five
 *   rope, kv_write, kv_read, tree_attention, token_logprobs -> status (int): flat arguments, the fields of
 *     w4a16_rope_t (positions, table, table_rows, rot_dim, interleaved; positions 0: no rope) and of
 *     w4a16_kv_cache_t (data, num_pages, kv_heads, head_dim, page_size, bits) in the place of the structures. The GIL is
 *     released around each: a launch waits while the stream's queue is full.
 *
 *   bind_step(lora, verify_drafts, kv_fork, kv_reserve, kv_free, kv_copy, kv_compact)   addresses of the seven
 *   lora, verify_drafts, kv_fork, kv_reserve, kv_free, kv_copy, kv_compact -> status (int): the same way.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <limits.h>
#include <stddef.h>
#include <stdint.h>

#include "w4a16.h"

typedef int (*layer_gemm_fn)(void *layer, const void *a, void *out, int64_t m, void *workspace,
                             size_t workspace_bytes, void *stream);
static layer_gemm_fn g_layer_gemm = NULL;

static void *as_ptr(PyObject *o) {
  if (o == Py_None) return NULL;
  return PyLong_AsVoidPtr(o);
}

static PyObject *bind(PyObject *self, PyObject *arg) {
  (void)self;
  void *p = PyLong_AsVoidPtr(arg);
  if (p == NULL) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: null function address");
    return NULL;
  }
  g_layer_gemm = (layer_gemm_fn)p;
  Py_RETURN_NONE;
}

static PyObject *layer_gemm(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  (void)self;
  if (nargs != 7) {
    PyErr_SetString(PyExc_TypeError, "layer_gemm takes 7 arguments (layer, a, out, m, ws, ws_bytes, stream)");
    return NULL;
  }
  if (g_layer_gemm == NULL) {
    PyErr_SetString(PyExc_RuntimeError, "layer_gemm: bind() was not called");
    return NULL;
  }
  void *layer = as_ptr(args[0]);
  const void *a = as_ptr(args[1]);
  void *out = as_ptr(args[2]);
  const long long m = PyLong_AsLongLong(args[3]);
  void *ws = as_ptr(args[4]);
  const size_t ws_bytes = args[5] == Py_None ? 0 : PyLong_AsSize_t(args[5]);
  void *stream = as_ptr(args[6]);
  if (PyErr_Occurred()) return NULL;
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = g_layer_gemm(layer, a, out, (int64_t)m, ws, ws_bytes, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

static uint64_t (*g_capture_id)(w4a16_stream_t) = NULL;

static PyObject *bind_capture(PyObject *self, PyObject *arg) {
  (void)self;
  void *p = PyLong_AsVoidPtr(arg);
  if (p == NULL) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind_capture: null function address");
    return NULL;
  }
  *(void **)&g_capture_id = p;
  Py_RETURN_NONE;
}
static PyObject *capture_id(PyObject *self, PyObject *arg) {
  (void)self;
  if (g_capture_id == NULL) {
    PyErr_SetString(PyExc_RuntimeError, "capture_id: bind_capture() was not called");
    return NULL;
  }
  void *stream = as_ptr(arg);
  if (PyErr_Occurred()) return NULL;
  return PyLong_FromUnsignedLongLong(g_capture_id((w4a16_stream_t)stream));
}

/* Integer arguments (None counts as 0) of a call that takes `want` of them; argument `f` (if not negative)
 * is a float. 0 on success. */
static int take(const char *name, PyObject *const *args, Py_ssize_t nargs, int want, int f, int64_t *v, double *d) {
  if (nargs != want) {
    PyErr_Format(PyExc_TypeError, "%s takes %d arguments (got %zd)", name, want, nargs);
    return -1;
  }
  for (int i = 0; i < want; ++i) {
    if (i == f) *d = PyFloat_AsDouble(args[i]);
    else v[i] = args[i] == Py_None ? 0 : PyLong_AsLongLong(args[i]);
  }
  return PyErr_Occurred() ? -1 : 0;
}
/* An argument of the C type int: one outside its range becomes the nearest end, which the library's checks refuse (cut to
 * 32 bits it could be another, valid number). */
static int to_int(int64_t x) { return x > INT_MAX ? INT_MAX : x < INT_MIN ? INT_MIN : (int)x; }
#define PTR(i) ((void *)(uintptr_t)v[i])
#define I32(i) to_int(v[i])

static w4a16_status (*g_rope)(const w4a16_rope_t *, const void *, int64_t, int64_t, void *, int64_t, int64_t, int64_t, int, int,
                              w4a16_dtype, w4a16_stream_t);
static w4a16_status (*g_kv_write)(const w4a16_kv_cache_t *, const void *, int64_t, int64_t, const void *, int64_t, int64_t,
                                  const int64_t *, int64_t, const w4a16_rope_t *, const void *, int64_t, int64_t, int, void *,
                                  w4a16_dtype, w4a16_stream_t);
static w4a16_status (*g_kv_read)(const w4a16_kv_cache_t *, const int64_t *, int64_t, void *, void *, w4a16_dtype, w4a16_stream_t);
static w4a16_status (*g_tree_attention)(const w4a16_kv_cache_t *, const void *, int64_t, int64_t, int, int64_t, const int32_t *, int64_t,
                                        int, const int32_t *, const int32_t *, int64_t, const uint64_t *, float, void *, float *,
                                        int, w4a16_dtype, void *, size_t, w4a16_stream_t);
static w4a16_status (*g_token_logprobs)(const void *, int64_t, int64_t, int64_t, w4a16_dtype, const int64_t *, int, int, float *,
                                        float *, int64_t *, float *, w4a16_stream_t);

static PyObject *bind_serving(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  (void)self;
  int64_t v[5];
  if (take("bind_serving", args, nargs, 5, -1, v, NULL)) return NULL;
  for (int i = 0; i < 5; ++i)
    if (!v[i]) {
      PyErr_SetString(PyExc_ValueError, "bind_serving: null function address");
      return NULL;
    }
  *(void **)&g_rope = PTR(0);
  *(void **)&g_kv_write = PTR(1);
  *(void **)&g_kv_read = PTR(2);
  *(void **)&g_tree_attention = PTR(3);
  *(void **)&g_token_logprobs = PTR(4);
  Py_RETURN_NONE;
}
static int unbound(const void *fn) {
  if (fn == NULL) PyErr_SetString(PyExc_RuntimeError, "bind_serving() was not called");
  return fn == NULL;
}
static w4a16_rope_t rope_at(const int64_t *v) {
  const w4a16_rope_t r = {(const int64_t *)(uintptr_t)v[0], (const float *)(uintptr_t)v[1], v[2], I32(3), I32(4)};
  return r;
}
static w4a16_kv_cache_t cache_at(const int64_t *v) {
  const w4a16_kv_cache_t c = {(void *)(uintptr_t)v[0], v[1], I32(2), I32(3), I32(4), I32(5)};
  return c;
}

/* rope[5], x, token stride, head stride, out, token stride, head stride, tokens, heads, head_dim, dtype, stream */
static PyObject *rope(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  (void)self;
  int64_t v[16];
  if (unbound(*(void **)&g_rope) || take("rope", args, nargs, 16, -1, v, NULL)) return NULL;
  const w4a16_rope_t r = rope_at(v);
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = g_rope(&r, PTR(5), v[6], v[7], PTR(8), v[9], v[10], v[11], I32(12), I32(13), (w4a16_dtype)I32(14), PTR(15));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}
/* cache[6], k, strides[2], v, strides[2], slots, tokens, rope[5], q, strides[2], q_heads, q_out, dtype, stream */
static PyObject *kv_write(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  (void)self;
  int64_t v[26];
  if (unbound(*(void **)&g_kv_write) || take("kv_write", args, nargs, 26, -1, v, NULL)) return NULL;
  const w4a16_kv_cache_t c = cache_at(v);
  const w4a16_rope_t r = rope_at(v + 14);
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = g_kv_write(&c, PTR(6), v[7], v[8], PTR(9), v[10], v[11], PTR(12), v[13], v[14] ? &r : NULL, PTR(19), v[20], v[21], I32(22),
                  PTR(23), (w4a16_dtype)I32(24), PTR(25));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}
/* cache[6], slots, tokens, k_out, v_out, dtype, stream */
static PyObject *kv_read(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  (void)self;
  int64_t v[12];
  if (unbound(*(void **)&g_kv_read) || take("kv_read", args, nargs, 12, -1, v, NULL)) return NULL;
  const w4a16_kv_cache_t c = cache_at(v);
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = g_kv_read(&c, PTR(6), v[7], PTR(8), PTR(9), (w4a16_dtype)I32(10), PTR(11));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}
/* cache[6], q, strides[2], q_heads, total_q, q_start, batch, max_q, kv_lens, page_table, max_pages, tree_mask, scale, out,
 * lse, fill, dtype, workspace, bytes, stream */
static PyObject *tree_attention(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  (void)self;
  int64_t v[26];
  double scale = 0.0;
  if (unbound(*(void **)&g_tree_attention) || take("tree_attention", args, nargs, 26, 18, v, &scale)) return NULL;
  const w4a16_kv_cache_t c = cache_at(v);
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = g_tree_attention(&c, PTR(6), v[7], v[8], I32(9), v[10], PTR(11), v[12], I32(13), PTR(14), PTR(15), v[16], PTR(17), (float)scale,
                        PTR(19), PTR(20), I32(21), (w4a16_dtype)I32(22), PTR(23), (size_t)v[24], PTR(25));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}
/* logits, row_stride, rows, vocab, dtype, tokens, n_tokens, top_k, logprobs, entropy, top_ids, top_logprobs, stream */
static PyObject *token_logprobs(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  (void)self;
  int64_t v[13];
  if (unbound(*(void **)&g_token_logprobs) || take("token_logprobs", args, nargs, 13, -1, v, NULL)) return NULL;
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = g_token_logprobs(PTR(0), v[1], v[2], v[3], (w4a16_dtype)I32(4), PTR(5), I32(6), I32(7), PTR(8), PTR(9), PTR(10), PTR(11), PTR(12));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

static w4a16_status (*g_lora)(const void *, int64_t, const void *, const void *, const int32_t *, const float *, const void *, int64_t, void *,
                              int64_t, int64_t, int64_t, int64_t, int, int64_t, w4a16_dtype, void *, size_t, w4a16_stream_t);
static w4a16_status (*g_verify)(const void *, int64_t, int64_t, int64_t, w4a16_dtype, const int64_t *, const int32_t *, int64_t, int,
                                const uint64_t *, const float *, const float *, int64_t, const float *, int64_t, const float *, int32_t *,
                                int32_t *, int64_t *, float *, void *, size_t, w4a16_stream_t);
static w4a16_status (*g_kv_fork)(int32_t *, int64_t, int, const int32_t *, int64_t, const int32_t *, int64_t, const int32_t *, int64_t, int32_t *,
                                 int32_t *, w4a16_stream_t);
static w4a16_status (*g_kv_reserve)(int32_t *, int64_t, int, int32_t *, int64_t, const int32_t *, const int32_t *, int64_t, int32_t *, int32_t *,
                                    w4a16_stream_t);
static w4a16_status (*g_kv_free)(int32_t *, int64_t, int, int32_t *, int64_t, const int32_t *, const int32_t *, int64_t, w4a16_stream_t);
static w4a16_status (*g_kv_copy)(const w4a16_kv_cache_t *, int64_t, const int32_t *, int64_t, w4a16_stream_t);
static w4a16_status (*g_kv_compact)(const w4a16_kv_cache_t *, int64_t, const int32_t *, int64_t, const int32_t *, const int32_t *, int64_t,
                                    const int32_t *, int, int32_t *, w4a16_stream_t);

static PyObject *bind_step(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  (void)self;
  int64_t v[7];
  if (take("bind_step", args, nargs, 7, -1, v, NULL)) return NULL;
  for (int i = 0; i < 7; ++i)
    if (!v[i]) {
      PyErr_SetString(PyExc_ValueError, "bind_step: null function address");
      return NULL;
    }
  *(void **)&g_lora = PTR(0);
  *(void **)&g_verify = PTR(1);
  *(void **)&g_kv_fork = PTR(2);
  *(void **)&g_kv_reserve = PTR(3);
  *(void **)&g_kv_free = PTR(4);
  *(void **)&g_kv_copy = PTR(5);
  *(void **)&g_kv_compact = PTR(6);
  Py_RETURN_NONE;
}
static int step_unbound(const void *fn) {
  if (fn == NULL) PyErr_SetString(PyExc_RuntimeError, "bind_step() was not called");
  return fn == NULL;
}

/* the arguments of the C functions in their order, a cache as its six fields */
static PyObject *lora(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  (void)self;
  int64_t v[19];
  if (step_unbound(*(void **)&g_lora) || take("lora", args, nargs, 19, -1, v, NULL)) return NULL;
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = g_lora(PTR(0), v[1], PTR(2), PTR(3), PTR(4), PTR(5), PTR(6), v[7], PTR(8), v[9], v[10], v[11], v[12], I32(13), v[14], (w4a16_dtype)I32(15),
              PTR(16), (size_t)v[17], PTR(18));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}
static PyObject *verify_drafts(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  (void)self;
  int64_t v[23];
  if (step_unbound(*(void **)&g_verify) || take("verify_drafts", args, nargs, 23, -1, v, NULL)) return NULL;
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = g_verify(PTR(0), v[1], v[2], v[3], (w4a16_dtype)I32(4), PTR(5), PTR(6), v[7], I32(8), PTR(9), PTR(10), PTR(11), v[12], PTR(13), v[14],
                PTR(15), PTR(16), PTR(17), PTR(18), PTR(19), PTR(20), (size_t)v[21], PTR(22));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}
static PyObject *kv_fork(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  (void)self;
  int64_t v[12];
  if (step_unbound(*(void **)&g_kv_fork) || take("kv_fork", args, nargs, 12, -1, v, NULL)) return NULL;
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = g_kv_fork(PTR(0), v[1], I32(2), PTR(3), v[4], PTR(5), v[6], PTR(7), v[8], PTR(9), PTR(10), PTR(11));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}
static PyObject *kv_reserve(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  (void)self;
  int64_t v[11];
  if (step_unbound(*(void **)&g_kv_reserve) || take("kv_reserve", args, nargs, 11, -1, v, NULL)) return NULL;
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = g_kv_reserve(PTR(0), v[1], I32(2), PTR(3), v[4], PTR(5), PTR(6), v[7], PTR(8), PTR(9), PTR(10));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}
static PyObject *kv_free(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  (void)self;
  int64_t v[9];
  if (step_unbound(*(void **)&g_kv_free) || take("kv_free", args, nargs, 9, -1, v, NULL)) return NULL;
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = g_kv_free(PTR(0), v[1], I32(2), PTR(3), v[4], PTR(5), PTR(6), v[7], PTR(8));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}
static PyObject *kv_copy(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  (void)self;
  int64_t v[10];
  if (step_unbound(*(void **)&g_kv_copy) || take("kv_copy", args, nargs, 10, -1, v, NULL)) return NULL;
  const w4a16_kv_cache_t c = cache_at(v);
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = g_kv_copy(&c, v[6], PTR(7), v[8], PTR(9));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}
static PyObject *kv_compact(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  (void)self;
  int64_t v[16];
  if (step_unbound(*(void **)&g_kv_compact) || take("kv_compact", args, nargs, 16, -1, v, NULL)) return NULL;
  const w4a16_kv_cache_t c = cache_at(v);
  int st;
  Py_BEGIN_ALLOW_THREADS
  st = g_kv_compact(&c, v[6], PTR(7), v[8], PTR(9), PTR(10), v[11], PTR(12), I32(13), PTR(14), PTR(15));
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(st);
}

#define FAST(f) (PyCFunction)(void (*)(void))f, METH_FASTCALL
static PyMethodDef kMethods[] = {
    {"bind", (PyCFunction)bind, METH_O, "bind(address of w4a16_layer_gemm)"},
    {"layer_gemm", (PyCFunction)(void (*)(void))layer_gemm, METH_FASTCALL,
     "layer_gemm(layer, a, out, m, ws, ws_bytes, stream) -> status"},
    {"bind_capture", (PyCFunction)bind_capture, METH_O, "bind_capture(address of w4a16_stream_capture_id)"},
    {"capture_id", (PyCFunction)capture_id, METH_O, "capture_id(stream) -> number of its capture, 0 for none"},
    {"bind_serving", FAST(bind_serving), "bind_serving(rope, kv_write, kv_read, tree_attention_fill, token_logprobs)"},
    {"rope", FAST(rope), "w4a16_rope, flat arguments -> status"},
    {"kv_write", FAST(kv_write), "w4a16_kv_write, flat arguments -> status"},
    {"kv_read", FAST(kv_read), "w4a16_kv_read, flat arguments -> status"},
    {"tree_attention", FAST(tree_attention), "w4a16_tree_attention_fill, flat arguments -> status"},
    {"token_logprobs", FAST(token_logprobs), "w4a16_token_logprobs, flat arguments -> status"},
    {"bind_step", FAST(bind_step), "bind_step(lora, verify_drafts, kv_fork, kv_reserve, kv_free, kv_copy, kv_compact)"},
    {"lora", FAST(lora), "w4a16_lora -> status"},
    {"verify_drafts", FAST(verify_drafts), "w4a16_verify_drafts -> status"},
    {"kv_fork", FAST(kv_fork), "w4a16_kv_fork -> status"},
    {"kv_reserve", FAST(kv_reserve), "w4a16_kv_reserve -> status"},
    {"kv_free", FAST(kv_free), "w4a16_kv_free -> status"},
    {"kv_copy", FAST(kv_copy), "w4a16_kv_copy, flat arguments -> status"},
    {"kv_compact", FAST(kv_compact), "w4a16_kv_compact, flat arguments -> status"},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_w4a16_call",
                                     "Argument marshalling for the calls of libw4a16.so.", -1, kMethods,
                                     NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__w4a16_call(void) { return PyModule_Create(&kModule); }
