/*
 * The calls of the operators around a step of many users for tensors that need no words: checks of the tensors, allocation of the
 * outputs and the call of the C entry point in one step of C++. It exists because reading a tensor's dtype, shape, strides,
 * device and address from Python takes longer than the smallest of these calls run on the GPU (seven tensors of w4a16_lora:
 * 6 of 10 us). No computation happens here.
 *
 * Every function returns its outputs, or None where the call is not an ordinary one: a tensor that is none (or of a subclass), is
 * elsewhere, or has another dtype or layout than it should; sizes that do not fit; a call that needs a workspace, or
 * that the library refuses. The binding then makes the call itself, with its checks and messages.
 *
 *   bind(lora, verify_drafts, kv_fork, kv_reserve, kv_free, kv_copy, kv_compact, lora_workspace_size)   addresses
 */
#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>

#include "w4a16.h"

namespace {

decltype(&w4a16_lora) g_lora;
decltype(&w4a16_verify_drafts) g_verify;
decltype(&w4a16_kv_fork) g_fork;
decltype(&w4a16_kv_reserve) g_reserve;
decltype(&w4a16_kv_free) g_free;
decltype(&w4a16_kv_copy) g_copy;
decltype(&w4a16_kv_compact) g_compact;
decltype(&w4a16_lora_workspace_size) g_lora_workspace;

using at::ScalarType;

const at::Tensor *tensor(PyObject *o) { return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr; }

// The device of an ordinary call: the tensor's, when that is the current one; -1 otherwise
int device_of(const at::Tensor *t) {
  if (!t || !t->is_cuda()) return -1;
  const int dev = t->get_device();
  return dev == c10::cuda::current_device() ? dev : -1;
}
// A contiguous tensor of this type, shape and device
bool is(const at::Tensor *t, int dev, ScalarType type, std::initializer_list<int64_t> shape) {
  return t && t->is_cuda() && t->get_device() == dev && t->scalar_type() == type && t->sizes() == c10::IntArrayRef(shape) && t->is_contiguous();
}
// The same or None; the address (null for None) in *p
bool is_or_none(PyObject *o, int dev, ScalarType type, std::initializer_list<int64_t> shape, const void **p) {
  *p = nullptr;
  if (o == Py_None) return true;
  const at::Tensor *t = tensor(o);
  if (!is(t, dev, type, shape)) return false;
  *p = t->const_data_ptr();
  return true;
}
// Contiguous rows
bool has_rows(const at::Tensor *t, int dev, ScalarType type, int64_t rows, int64_t cols) {
  return t && t->is_cuda() && t->get_device() == dev && t->scalar_type() == type && t->dim() == 2 && t->size(0) == rows && t->size(1) == cols &&
         (t->stride(1) == 1 || cols <= 1);
}
bool half_type(ScalarType t) { return t == ScalarType::Half || t == ScalarType::BFloat16; }
w4a16_dtype code(ScalarType t) { return t == ScalarType::Half ? W4A16_F16 : t == ScalarType::BFloat16 ? W4A16_BF16 : W4A16_F32; }
at::Tensor make(std::initializer_list<int64_t> shape, ScalarType type, const at::Tensor &like) {
  // (what at::empty comes to, without its dispatch)
  return at::detail::empty_cuda(c10::IntArrayRef(shape), type, like.device(), c10::nullopt);
}
w4a16_stream_t stream_of(int dev) {
  return reinterpret_cast<w4a16_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
}
template <class F>
w4a16_status call(F &&f) {  // without the GIL: a launch waits while the stream's queue is full
  w4a16_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  return st;
}
PyObject *none() { Py_RETURN_NONE; }
PyObject *tuple(std::initializer_list<at::Tensor> ts) {
  PyObject *out = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
  Py_ssize_t i = 0;
  for (const at::Tensor &t : ts) PyTuple_SET_ITEM(out, i++, THPVariable_Wrap(t));
  return out;
}
// No C++ exception leaves a function: what torch throws is left to the binding's own call
template <class F>
PyObject *guarded(F &&f) {
  try {
    return f();
  } catch (const std::exception &) {
    return none();
  }
}
bool integer(PyObject *o, int64_t *v) {
  if (!PyLong_CheckExact(o)) return false;
  int overflow = 0;
  *v = PyLong_AsLongLongAndOverflow(o, &overflow);
  return !overflow;
}

// x, a, b, ids, base, scales, out
PyObject *lora(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 7 || !g_lora) return none();
  return guarded([&]() -> PyObject * {
    const at::Tensor *x = tensor(args[0]), *a = tensor(args[1]), *b = tensor(args[2]), *ids = tensor(args[3]), *base = tensor(args[4]);
    const int dev = device_of(x);
    if (dev < 0 || !a || !b || !base || x->dim() != 2 || a->dim() != 3 || b->dim() != 3) return none();
    const ScalarType type = x->scalar_type();
    const int64_t T = x->size(0), K = x->size(1), L = a->size(0), r = a->size(1), N = b->size(1);
    const void *scales;
    if (!half_type(type) || r > 128 || !has_rows(x, dev, type, T, K) || !is(a, dev, type, {L, r, K}) || !is(b, dev, type, {L, N, r}) ||
        !is(ids, dev, ScalarType::Int, {T}) || !has_rows(base, dev, type, T, N) || !is_or_none(args[5], dev, ScalarType::Float, {L}, &scales))
      return none();
    if (T > 256 && g_lora_workspace(T, static_cast<int>(r), L) != 0) return none();
    at::Tensor out;
    if (args[6] == Py_None) {
      out = make({T, N}, type, *x);
    } else {
      const at::Tensor *given = tensor(args[6]);
      if (!has_rows(given, dev, type, T, N)) return none();
      out = *given;
    }
    const w4a16_stream_t s = stream_of(dev);
    const w4a16_status st = call([&] {
      return g_lora(x->const_data_ptr(), x->stride(0), a->const_data_ptr(), b->const_data_ptr(), static_cast<const int32_t *>(ids->const_data_ptr()),
                    static_cast<const float *>(scales), base->const_data_ptr(), base->stride(0), out.data_ptr(), out.stride(0), T, K, N,
                    static_cast<int>(r), L, code(type), nullptr, 0, s);
    });
    if (st != W4A16_OK) return none();
    if (args[6] == Py_None) return THPVariable_Wrap(out);
    Py_INCREF(args[6]);
    return args[6];
  });
}

// logits, tokens, uniforms, noise, q_start, tree_mask, draft_probs, temperature, max_q, workspace address, its bytes
PyObject *verify_drafts(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 11 || !g_verify) return none();
  return guarded([&]() -> PyObject * {
    const at::Tensor *logits = tensor(args[0]), *tokens = tensor(args[1]), *uniforms = tensor(args[2]), *noise = tensor(args[3]);
    const int dev = device_of(logits);
    int64_t m, ws, ws_bytes;
    if (dev < 0 || logits->dim() != 2 || !noise || noise->dim() != 2 || !integer(args[8], &m) || !integer(args[9], &ws) || !integer(args[10], &ws_bytes))
      return none();
    const ScalarType type = logits->scalar_type();
    const int64_t total = logits->size(0), V = logits->size(1), B = noise->size(0);
    const void *q_start, *mask, *temperature;
    if ((!half_type(type) && type != ScalarType::Float) || m < 1 || m > 64 || !has_rows(logits, dev, type, total, V) ||
        !has_rows(noise, dev, ScalarType::Float, B, V) || !is(tokens, dev, ScalarType::Long, {total}) || !is(uniforms, dev, ScalarType::Float, {total}) ||
        !is_or_none(args[4], dev, ScalarType::Int, {B + 1}, &q_start) || !is_or_none(args[5], dev, ScalarType::Long, {total}, &mask) ||
        !is_or_none(args[7], dev, ScalarType::Float, {B}, &temperature))
      return none();
    const void *draft = nullptr;
    int64_t draft_stride = 0;
    if (args[6] != Py_None) {
      const at::Tensor *d = tensor(args[6]);
      if (!has_rows(d, dev, ScalarType::Float, total, V)) return none();
      draft = d->const_data_ptr(), draft_stride = d->stride(0);
    }
    const at::Tensor accepted = make({B}, ScalarType::Int, *logits), path = make({B, m}, ScalarType::Int, *logits),
                     out = make({B, m}, ScalarType::Long, *logits), probs = make({B, m}, ScalarType::Float, *logits);
    const w4a16_stream_t s = stream_of(dev);
    const w4a16_status st = call([&] {
      return g_verify(logits->const_data_ptr(), logits->stride(0), total, V, code(type), static_cast<const int64_t *>(tokens->const_data_ptr()),
                      static_cast<const int32_t *>(q_start), B, static_cast<int>(m), static_cast<const uint64_t *>(mask),
                      static_cast<const float *>(uniforms->const_data_ptr()), static_cast<const float *>(noise->const_data_ptr()), noise->stride(0),
                      static_cast<const float *>(draft), draft_stride, static_cast<const float *>(temperature),
                      static_cast<int32_t *>(accepted.data_ptr()), static_cast<int32_t *>(path.data_ptr()), static_cast<int64_t *>(out.data_ptr()),
                      static_cast<float *>(probs.data_ptr()), reinterpret_cast<void *>(ws), static_cast<size_t>(ws_bytes), s);
    });
    return st == W4A16_OK ? tuple({accepted, path, out, probs}) : none();
  });
}

struct Table {
  int32_t *refs, *table;
  int64_t pages, batch, cols;
  const int32_t *lens;
  int dev, page_size;
};
// refs, page_table, kv_lens of args[0 .. 2] and the page size of args[at]
bool table_of(PyObject *const *args, int at, Table *t) {
  const at::Tensor *refs = tensor(args[0]), *table = tensor(args[1]), *lens = tensor(args[2]);
  t->dev = device_of(refs);
  int64_t page_size;
  if (t->dev < 0 || refs->dim() != 1 || !table || table->dim() != 2 || !integer(args[at], &page_size) || page_size < 1 || page_size > (1 << 20)) return false;
  t->pages = refs->size(0), t->batch = table->size(0), t->cols = table->size(1), t->page_size = static_cast<int>(page_size);
  if (!is(refs, t->dev, ScalarType::Int, {t->pages}) || !is(table, t->dev, ScalarType::Int, {t->batch, t->cols}) ||
      !is(lens, t->dev, ScalarType::Int, {t->batch}))
    return false;
  t->refs = static_cast<int32_t *>(refs->data_ptr()), t->table = static_cast<int32_t *>(table->data_ptr());
  t->lens = static_cast<const int32_t *>(lens->const_data_ptr());
  return true;
}

// refs, page_table, kv_lens, parents, page_size
PyObject *kv_fork(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 5 || !g_fork) return none();
  return guarded([&]() -> PyObject * {
    Table t;
    const at::Tensor *parents = tensor(args[3]);
    if (!table_of(args, 4, &t) || !parents || parents->dim() != 1) return none();
    const int64_t rows = parents->size(0);
    if (!is(parents, t.dev, ScalarType::Int, {rows})) return none();
    const at::Tensor table = make({rows, t.cols}, ScalarType::Int, *parents), lens = make({rows}, ScalarType::Int, *parents);
    const w4a16_stream_t s = stream_of(t.dev);
    const w4a16_status st = call([&] {
      return g_fork(t.refs, t.pages, t.page_size, t.table, t.cols, t.lens, t.batch, static_cast<const int32_t *>(parents->const_data_ptr()), rows,
                    static_cast<int32_t *>(table.data_ptr()), static_cast<int32_t *>(lens.data_ptr()), s);
    });
    return st == W4A16_OK ? tuple({table, lens}) : none();
  });
}
// refs, page_table, kv_lens, new_lens, page_size
PyObject *kv_reserve(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 5 || !g_reserve) return none();
  return guarded([&]() -> PyObject * {
    Table t;
    const at::Tensor *new_lens = tensor(args[3]);
    if (!table_of(args, 4, &t) || !is(new_lens, t.dev, ScalarType::Int, {t.batch})) return none();
    const at::Tensor held = make({t.batch}, ScalarType::Int, *new_lens), copies = make({t.batch, 2}, ScalarType::Int, *new_lens);
    const w4a16_stream_t s = stream_of(t.dev);
    const w4a16_status st = call([&] {
      return g_reserve(t.refs, t.pages, t.page_size, t.table, t.cols, t.lens, static_cast<const int32_t *>(new_lens->const_data_ptr()), t.batch,
                       static_cast<int32_t *>(held.data_ptr()), static_cast<int32_t *>(copies.data_ptr()), s);
    });
    return st == W4A16_OK ? tuple({held, copies}) : none();
  });
}
// refs, page_table, kv_lens, page_size, keep -> True
PyObject *kv_free(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 5 || !g_free) return none();
  return guarded([&]() -> PyObject * {
    Table t;
    const void *keep;
    if (!table_of(args, 3, &t) || !is_or_none(args[4], t.dev, ScalarType::Int, {t.batch}, &keep)) return none();
    const w4a16_stream_t s = stream_of(t.dev);
    const w4a16_status st = call([&] {
      return g_free(t.refs, t.pages, t.page_size, t.table, t.cols, t.lens, static_cast<const int32_t *>(keep), t.batch, s);
    });
    if (st != W4A16_OK) return none();
    Py_RETURN_TRUE;
  });
}

// A cache of one layer or a stack of them; head_dim 0: any that fits
bool cache_of(const at::Tensor *t, int64_t head_dim, int *dev, w4a16_kv_cache_t *c, int64_t *layers) {
  *dev = device_of(t);
  if (*dev < 0 || t->scalar_type() != ScalarType::Byte || !t->is_contiguous() || (t->dim() != 4 && t->dim() != 5)) return false;
  const int64_t d = t->dim();
  *layers = d == 5 ? t->size(0) : 1;
  const int64_t tile = t->size(d - 1), tiles = t->size(d - 2), heads = t->size(d - 3);
  if (tiles > (1 << 16) || heads > 1024) return false;
  *c = w4a16_kv_cache_t{t->data_ptr(), t->size(d - 4), static_cast<int32_t>(heads), 0, static_cast<int32_t>(tiles * 16), 0};
  for (int size : {64, 128, 256})
    for (int bits : {4, 8})
      if (c->bits == 0 && (head_dim == 0 || head_dim == size) && tile == 4 * size * bits + 128) c->head_dim = size, c->bits = bits;
  return c->bits != 0;
}
// cache, copies -> True
PyObject *kv_copy(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 2 || !g_copy) return none();
  return guarded([&]() -> PyObject * {
    int dev;
    w4a16_kv_cache_t c;
    int64_t layers;
    const at::Tensor *copies = tensor(args[1]);
    if (!cache_of(tensor(args[0]), 0, &dev, &c, &layers) || !copies || copies->dim() != 2) return none();
    const int64_t pairs = copies->size(0);
    if (!is(copies, dev, ScalarType::Int, {pairs, 2})) return none();
    const w4a16_stream_t s = stream_of(dev);
    if (call([&] { return g_copy(&c, layers, static_cast<const int32_t *>(copies->const_data_ptr()), pairs, s); }) != W4A16_OK) return none();
    Py_RETURN_TRUE;
  });
}
// cache, head_dim, page_table, kv_lens, path, q_start
PyObject *kv_compact(PyObject *, PyObject *const *args, Py_ssize_t n) {
  if (n != 6 || !g_compact) return none();
  return guarded([&]() -> PyObject * {
    int dev;
    w4a16_kv_cache_t c;
    int64_t layers, head_dim;
    const at::Tensor *table = tensor(args[2]), *lens = tensor(args[3]), *path = tensor(args[4]);
    if (!integer(args[1], &head_dim) || head_dim <= 0 || !cache_of(tensor(args[0]), head_dim, &dev, &c, &layers) || !table || table->dim() != 2 || !path ||
        path->dim() != 2)
      return none();
    const int64_t B = table->size(0), cols = table->size(1), m = path->size(1);
    const void *q_start;
    if (m > 64 || !is(table, dev, ScalarType::Int, {B, cols}) || !is(lens, dev, ScalarType::Int, {B}) || !is(path, dev, ScalarType::Int, {B, m}) ||
        !is_or_none(args[5], dev, ScalarType::Int, {B + 1}, &q_start))
      return none();
    const at::Tensor out = make({B}, ScalarType::Int, *lens);
    const w4a16_stream_t s = stream_of(dev);
    const w4a16_status st = call([&] {
      return g_compact(&c, layers, static_cast<const int32_t *>(table->const_data_ptr()), cols, static_cast<const int32_t *>(lens->const_data_ptr()),
                       static_cast<const int32_t *>(q_start), B, static_cast<const int32_t *>(path->const_data_ptr()), static_cast<int>(m),
                       static_cast<int32_t *>(out.data_ptr()), s);
    });
    return st == W4A16_OK ? THPVariable_Wrap(out) : none();
  });
}

PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
  void *p[8];
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "bind takes 8 addresses");
    return nullptr;
  }
  for (int i = 0; i < 8; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (!p[i]) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "bind: null function address");
      return nullptr;
    }
  }
  g_lora = reinterpret_cast<decltype(g_lora)>(p[0]);
  g_verify = reinterpret_cast<decltype(g_verify)>(p[1]);
  g_fork = reinterpret_cast<decltype(g_fork)>(p[2]);
  g_reserve = reinterpret_cast<decltype(g_reserve)>(p[3]);
  g_free = reinterpret_cast<decltype(g_free)>(p[4]);
  g_copy = reinterpret_cast<decltype(g_copy)>(p[5]);
  g_compact = reinterpret_cast<decltype(g_compact)>(p[6]);
  g_lora_workspace = reinterpret_cast<decltype(g_lora_workspace)>(p[7]);
  Py_RETURN_NONE;
}

#define FAST(f) #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef kMethods[] = {{FAST(bind), "bind(addresses)"},
                          {FAST(lora), "lora(x, a, b, ids, base, scales, out) -> out or None"},
                          {FAST(verify_drafts), "verify_drafts(.., max_q, workspace, bytes) -> outputs or None"},
                          {FAST(kv_fork), "kv_fork(refs, page_table, kv_lens, parents, page_size) -> outputs or None"},
                          {FAST(kv_reserve), "kv_reserve(refs, page_table, kv_lens, new_lens, page_size) -> outputs or None"},
                          {FAST(kv_free), "kv_free(refs, page_table, kv_lens, page_size, keep) -> True or None"},
                          {FAST(kv_copy), "kv_copy(cache, copies) -> True or None"},
                          {FAST(kv_compact), "kv_compact(cache, head_dim, page_table, kv_lens, path, q_start) -> new_lens or None"},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_w4a16_fast", "Ordinary calls of libw4a16.so on tensors.", -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// built_for: the torch whose headers this was compiled with, which the binding compares with the one that runs before it makes a call
PyMODINIT_FUNC PyInit__w4a16_fast(void) {
  PyObject *m = PyModule_Create(&kModule);
  if (m && PyModule_AddStringConstant(m, "built_for", W4A16_BUILT_FOR) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
