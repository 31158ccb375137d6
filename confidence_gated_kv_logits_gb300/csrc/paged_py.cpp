// Fast path of the Python binding (paged.py): checks tensor arguments and calls
// the C ABI of include/confkv_paged.h.  For a single token the checks and the
// launch are a call's whole cost: reading a tensor's type, device, shape,
// strides and address from Python takes about 0.5 us, here a few nanoseconds.
// Nothing is computed, copied or converted; a call returns the C ABI's code,
// and raises ValueError for a tensor of the wrong kind.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>
#include <initializer_list>
#include <new>

#include "../../include/confkv_paged.h"

namespace {

// What paged.py keeps beside a handle (its address is a Python integer there).
struct Object {
  confkv_paged* kv;           // BeamSelect: any non-null address
  void* ws;                   // BeamSelect: scratch
  size_t ws_bytes;
  cudaStream_t home;          // stream that the scratch was made on
  int64_t sizes[4];           // PagedKV: heads, kv_heads, head_dim; BeamSelect: batch, beams, vocab, keep
  int device;
  int dtype;                  // CONFKV_FP16, BF16, FP32
  int away;                   // a call ran on another stream
};

at::ScalarType type_of(int code) {
  return code == CONFKV_FP16 ? at::kHalf : code == CONFKV_BF16 ? at::kBFloat16 : at::kFloat;
}

// Raises ValueError with what was wanted and what came.
bool wrong(const char* name, const char* want, PyObject* got) {
  PyObject* shape = PyObject_GetAttrString(got, "shape");
  PyObject* dtype = PyObject_GetAttrString(got, "dtype");
  PyObject* dev = PyObject_GetAttrString(got, "device");
  PyErr_Clear();
  PyErr_Format(PyExc_ValueError, "%s: want %s, got %S %S on %S", name, want, dtype ? dtype : Py_None,
               shape ? shape : Py_None, dev ? dev : Py_None);
  Py_XDECREF(shape);
  Py_XDECREF(dtype);
  Py_XDECREF(dev);
  return false;
}

const at::Tensor* tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_ValueError, "%s: want a tensor, got %R", name, reinterpret_cast<PyObject*>(Py_TYPE(o)));
    return nullptr;
  }
  return &THPVariable_Unpack(o);
}

// dense memory on the object's device that holds the values as they are
bool plain(const Object* ob, const at::Tensor& t) {
  return t.is_cuda() && t.layout() == at::kStrided && !t.is_nested() && !t.is_neg() && t.get_device() == ob->device;
}

// a contiguous tensor of the given type and shape on the object's device
bool dense(const Object* ob, PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape,
           void** out) {
  const at::Tensor* t = tensor(o, name);
  if (!t) return false;
  bool ok = t->scalar_type() == type && plain(ob, *t) &&
            t->dim() == static_cast<int64_t>(shape.size()) && t->is_contiguous();
  if (ok) {
    int i = 0;
    for (const int64_t n : shape) ok = ok && t->size(i++) == n;
  }
  if (!ok) return wrong(name, "a contiguous tensor of the documented type and shape on the object's device", o);
  *out = t->data_ptr();
  return true;
}

// [rows, heads, head_dim] of the cache's type with dense rows
bool rows_of(const Object* ob, PyObject* o, const char* name, int64_t rows, int64_t heads, void** out, int64_t* stride) {
  const at::Tensor* t = tensor(o, name);
  if (!t) return false;
  const int64_t d = ob->sizes[2];
  if (t->scalar_type() != type_of(ob->dtype) || !plain(ob, *t) || t->dim() != 3 ||
      t->size(0) != rows || t->size(1) != heads || t->size(2) != d || t->stride(2) != 1 ||
      (heads > 1 && t->stride(1) != d))
    return wrong(name, "[rows, heads, head_dim] of the cache's type on its device, rows dense", o);
  *out = t->data_ptr();
  *stride = rows > 1 ? t->stride(0) : heads * d;
  return true;
}

bool rows_count(PyObject* o, const char* name, int64_t* rows) {
  const at::Tensor* t = tensor(o, name);
  if (!t) return false;
  if (t->dim() < 1 || t->size(0) > INT32_MAX) return wrong(name, "[rows, ..]", o);
  *rows = t->size(0);
  return true;
}

// [rows, columns]
bool matrix(PyObject* o, const char* name, int64_t* rows, int64_t* cols) {
  const at::Tensor* t = tensor(o, name);
  if (!t) return false;
  if (t->dim() != 2 || t->size(0) > INT32_MAX || t->size(1) > INT32_MAX) return wrong(name, "two dimensions", o);
  *rows = t->size(0);
  *cols = t->size(1);
  return true;
}

bool stream_of(Object* ob, PyObject* o, void** out) {
  cudaStream_t s;
  if (o == Py_None) {
    s = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(ob->device)).stream();
  } else {
    PyObject* v = PyObject_GetAttrString(o, "cuda_stream");
    if (!v) return false;
    s = static_cast<cudaStream_t>(PyLong_AsVoidPtr(v));
    Py_DECREF(v);
    if (PyErr_Occurred()) return false;
  }
  if (s != ob->home) ob->away = 1;
  *out = s;
  return true;
}

template <typename T>
T* pointer(PyObject* o) {
  return static_cast<T*>(PyLong_AsVoidPtr(o));
}
bool integer(PyObject* o, int* out) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) return false;
  if (v < INT32_MIN || v > INT32_MAX) {
    PyErr_SetString(PyExc_ValueError, "an integer argument does not fit 32 bits");
    return false;
  }
  *out = static_cast<int>(v);
  return true;
}
bool count(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%zd arguments, want %zd", n, want);
  return false;
}
bool ready(const Object* ob) {
  if (ob && ob->kv) return true;
  PyErr_SetString(PyExc_ValueError, "the handle is closed");    // (in the place of what reading None raised)
  return false;
}

// What both appends take of layer, k, v, q, q_out, .., inv_freq, interleaved, stream.
struct Append {
  int layer, rotary = 0, interleaved;
  int64_t rows, ks, vs, qs = 0, os = 0;
  void *k, *v, *q = nullptr, *out = nullptr, *pos = nullptr, *inv = nullptr, *s;
};
bool append_of(Object* ob, PyObject* const* a, PyObject* inv_freq, PyObject* interleaved, Append* x) {
  if (!integer(a[0], &x->layer) || !rows_count(a[1], "k", &x->rows) ||
      !rows_of(ob, a[1], "k", x->rows, ob->sizes[1], &x->k, &x->ks) || !rows_of(ob, a[2], "v", x->rows, ob->sizes[1], &x->v, &x->vs))
    return false;
  if (a[3] != Py_None || a[4] != Py_None) {
    if (a[3] == Py_None || a[4] == Py_None) {
      PyErr_SetString(PyExc_ValueError, "q and q_out go together");
      return false;
    }
    if (!rows_of(ob, a[3], "q", x->rows, ob->sizes[0], &x->q, &x->qs) ||
        !rows_of(ob, a[4], "q_out", x->rows, ob->sizes[0], &x->out, &x->os))
      return false;
  }
  if (inv_freq != Py_None) {
    int64_t half;
    if (!rows_count(inv_freq, "inv_freq", &half) || !dense(ob, inv_freq, "inv_freq", at::kFloat, {half}, &x->inv)) return false;
    x->rotary = half > 4096 ? 8192 : static_cast<int>(2 * half);
  }
  x->interleaved = PyObject_IsTrue(interleaved);
  return x->interleaved >= 0;
}

// object, batch, layer, k, v, q, q_out, positions, inv_freq, interleaved, stream
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 11)) return nullptr;
  Object* ob = pointer<Object>(a[0]);
  const confkv_paged_batch* batch = pointer<confkv_paged_batch>(a[1]);
  Append x;
  if (!ready(ob) || !append_of(ob, a + 2, a[8], a[9], &x) ||
      (a[7] != Py_None && !dense(ob, a[7], "positions", at::kInt, {x.rows}, &x.pos)) || !stream_of(ob, a[10], &x.s))
    return nullptr;
  return PyLong_FromLong(confkv_paged_append(ob->kv, batch, x.layer, static_cast<int>(x.rows), x.k, x.ks, x.v, x.vs, x.q, x.qs,
                                             x.out, x.os, static_cast<int32_t*>(x.pos), static_cast<float*>(x.inv), x.rotary,
                                             x.interleaved, x.s));
}

// weights [head_dim], fp32 or of the cache's type, both alike
bool weights(Object* ob, PyObject* o, const char* name, int* type, const void** out) {
  if (o == Py_None) return true;
  const at::Tensor* t = tensor(o, name);
  if (!t) return false;
  const int mine = t->scalar_type() == at::kFloat ? CONFKV_FP32 : ob->dtype;
  void* at;
  if (!dense(ob, o, name, type_of(mine), {ob->sizes[2]}, &at)) return false;
  if (*type >= 0 && *type != mine) {
    PyErr_SetString(PyExc_ValueError, "q_norm and k_norm differ in type");
    return false;
  }
  *type = mine;
  *out = at;
  return true;
}

// object, batch, layer, k, v, q, q_out, positions, inv_freq, interleaved, q_norm, k_norm, eps, axis, stream
PyObject* append_normed(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 15)) return nullptr;
  Object* ob = pointer<Object>(a[0]);
  const confkv_paged_batch* batch = pointer<confkv_paged_batch>(a[1]);
  Append x;
  confkv_paged_norm norm = {};
  int type = -1;
  if (!ready(ob)) return nullptr;
  const double eps = PyFloat_AsDouble(a[12]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  if (!append_of(ob, a + 2, a[8], a[9], &x) || !weights(ob, a[10], "q_norm", &type, &norm.q_norm) ||
      !weights(ob, a[11], "k_norm", &type, &norm.k_norm))
    return nullptr;
  if (a[13] != Py_None) {
    void* axis;
    int64_t rows = x.rows, axes = 0;
    if (!dense(ob, a[13], "axis", at::kInt, {x.rotary / 2}, &axis)) return nullptr;
    if (a[7] == Py_None) {
      PyErr_SetString(PyExc_ValueError, "axis needs positions [rows, axes]");
      return nullptr;
    }
    if (!matrix(a[7], "positions", &rows, &axes) || !dense(ob, a[7], "positions", at::kInt, {x.rows, axes}, &x.pos)) return nullptr;
    norm.axis = static_cast<int32_t*>(axis);
    norm.axes = static_cast<int>(axes);
  } else if (a[7] != Py_None && !dense(ob, a[7], "positions", at::kInt, {x.rows}, &x.pos)) {
    return nullptr;
  }
  if (!stream_of(ob, a[14], &x.s)) return nullptr;
  norm.norm_dtype = type < 0 ? CONFKV_FP32 : type;
  norm.eps = static_cast<float>(eps);
  return PyLong_FromLong(confkv_paged_append_normed(ob->kv, batch, x.layer, static_cast<int>(x.rows), x.k, x.ks, x.v, x.vs, x.q,
                                                    x.qs, x.out, x.os, static_cast<int32_t*>(x.pos), static_cast<float*>(x.inv),
                                                    x.rotary, x.interleaved, &norm, x.s));
}

// The scale of an attention: 0 for the default.
bool scale_of(PyObject* o, float* out) {
  const double scale = PyFloat_AsDouble(o);
  if (scale == -1.0 && PyErr_Occurred()) return false;
  if (scale != 0.0 && static_cast<float>(scale) == 0.0f) {      // 0 would mean the default
    PyErr_SetString(PyExc_ValueError, "scale is zero in 32 bits");
    return false;
  }
  *out = static_cast<float>(scale);
  return true;
}
bool mask_fits(int mask_rows, int64_t rows) {
  if (mask_rows < 0 || mask_rows >= rows) return true;
  PyErr_Format(PyExc_ValueError, "the batch's mask has %d rows, q has %lld", mask_rows, static_cast<long long>(rows));
  return false;
}

// What both attends take of mask rows (-1: no mask), layer, q, out, lse, scale.
struct Attend {
  int mask_rows, layer;
  int64_t rows, qs;
  void *q, *out, *lse = nullptr, *s;
  float scale;
};
bool attend_of(Object* ob, PyObject* const* a, Attend* x) {
  return scale_of(a[5], &x->scale) && integer(a[0], &x->mask_rows) && integer(a[1], &x->layer) && rows_count(a[2], "q", &x->rows) &&
         rows_of(ob, a[2], "q", x->rows, ob->sizes[0], &x->q, &x->qs) &&
         dense(ob, a[3], "out", type_of(ob->dtype), {x->rows, ob->sizes[0], ob->sizes[2]}, &x->out) &&
         mask_fits(x->mask_rows, x->rows) &&
         (a[4] == Py_None || dense(ob, a[4], "lse", at::kFloat, {x->rows, ob->sizes[0]}, &x->lse));
}

// object, batch, mask rows (-1: no mask), layer, q, out, lse, scale, stream
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 9)) return nullptr;
  Object* ob = pointer<Object>(a[0]);
  const confkv_paged_batch* batch = pointer<confkv_paged_batch>(a[1]);
  Attend x;
  if (!ready(ob) || !attend_of(ob, a + 2, &x) || !stream_of(ob, a[8], &x.s)) return nullptr;
  return PyLong_FromLong(confkv_paged_attend(ob->kv, batch, x.layer, static_cast<int>(x.rows), x.q, x.qs, x.out,
                                             static_cast<float*>(x.lse), x.scale, x.s));
}

// object, batch, prefix, mask rows (-1: no mask), layer, q, out, lse, scale, stream
PyObject* attend_shared(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 10)) return nullptr;
  Object* ob = pointer<Object>(a[0]);
  const confkv_paged_batch* batch = pointer<confkv_paged_batch>(a[1]);
  const confkv_paged_prefix* prefix = pointer<confkv_paged_prefix>(a[2]);
  Attend x;
  if (!ready(ob) || !attend_of(ob, a + 3, &x) || !stream_of(ob, a[9], &x.s)) return nullptr;
  return PyLong_FromLong(confkv_paged_attend_shared(ob->kv, batch, prefix, x.layer, static_cast<int>(x.rows), x.q, x.qs, x.out,
                                                    static_cast<float*>(x.lse), x.scale, x.s));
}

// a contiguous tensor of the given type, [.., cap] behind `shape`
bool table_of(Object* ob, PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape, int64_t* cap,
              void** out) {
  const at::Tensor* t = tensor(o, name);
  if (!t) return false;
  bool ok = t->scalar_type() == type && plain(ob, *t) && t->dim() == static_cast<int64_t>(shape.size()) + 1 && t->is_contiguous();
  if (ok) {
    int i = 0;
    for (const int64_t n : shape) ok = ok && t->size(i++) == n;
    ok = ok && t->size(i) <= INT32_MAX && (*cap < 0 || *cap == t->size(i));
    if (ok) *cap = t->size(i);
  }
  if (!ok) return wrong(name, "a contiguous tensor of the documented type and shape on the object's device", o);
  *out = t->data_ptr();
  return true;
}

// object, batch, sequences, mask rows, layer, q, lse, mass, mass_out, pos, positions, decay, gain, scale, stream
PyObject* weigh(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 15)) return nullptr;
  Object* ob = pointer<Object>(a[0]);
  const confkv_paged_batch* batch = pointer<confkv_paged_batch>(a[1]);
  int B, mask_rows, layer;
  int64_t rows, qs, cap = -1;
  void *q, *lse, *mass, *out, *pos = nullptr, *positions = nullptr, *s;
  float scale;
  if (!ready(ob)) return nullptr;
  const double decay = PyFloat_AsDouble(a[11]);
  if (decay == -1.0 && PyErr_Occurred()) return nullptr;
  const double gain = PyFloat_AsDouble(a[12]);
  if (gain == -1.0 && PyErr_Occurred()) return nullptr;
  const int64_t H = ob->sizes[1];
  if (!scale_of(a[13], &scale) || !integer(a[2], &B) || !integer(a[3], &mask_rows) || !integer(a[4], &layer) ||
      !rows_count(a[5], "q", &rows) || !rows_of(ob, a[5], "q", rows, ob->sizes[0], &q, &qs) || !mask_fits(mask_rows, rows) ||
      !dense(ob, a[6], "lse", at::kFloat, {rows, ob->sizes[0]}, &lse) ||
      !table_of(ob, a[7], "mass", at::kFloat, {B, H}, &cap, &mass) || !table_of(ob, a[8], "mass_out", at::kFloat, {B, H}, &cap, &out) ||
      (a[9] != Py_None && !table_of(ob, a[9], "pos", at::kInt, {B, H}, &cap, &pos)) ||
      (a[10] != Py_None && !dense(ob, a[10], "positions", at::kInt, {rows}, &positions)) || !stream_of(ob, a[14], &s))
    return nullptr;
  return PyLong_FromLong(confkv_paged_weigh(ob->kv, batch, layer, static_cast<int>(rows), q, qs, static_cast<float*>(lse),
                                            static_cast<float*>(mass), static_cast<float*>(out), static_cast<int32_t*>(pos),
                                            static_cast<int>(cap), static_cast<int32_t*>(positions), static_cast<float>(decay),
                                            static_cast<float>(gain), scale, s));
}

// object, layers, page_table, length, mass, pos, keep, mass_out, pos_out, new_len, protect, first, stream
PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 13)) return nullptr;
  Object* ob = pointer<Object>(a[0]);
  int layers, protect;
  int64_t B, blocks, cap = -1;
  void *table, *len, *mass, *pos, *keep, *mo, *po, *out, *first = nullptr, *s;
  if (!ready(ob) || !integer(a[1], &layers) || !matrix(a[2], "page_table", &B, &blocks) ||
      !dense(ob, a[2], "page_table", at::kInt, {B, blocks}, &table))
    return nullptr;
  const at::Tensor* t = tensor(a[3], "length");
  if (!t) return nullptr;
  const int per_layer = t->dim() == 2;
  auto lengths = [&](PyObject* o, const char* name, void** p) {
    return per_layer ? dense(ob, o, name, at::kInt, {layers, B}, p) : dense(ob, o, name, at::kInt, {B}, p);
  };
  const int64_t H = ob->sizes[1];
  if (!lengths(a[3], "length", &len) || !table_of(ob, a[4], "mass", at::kFloat, {layers, B, H}, &cap, &mass) ||
      !table_of(ob, a[5], "pos", at::kInt, {layers, B, H}, &cap, &pos) || !lengths(a[6], "keep", &keep) ||
      !table_of(ob, a[7], "mass_out", at::kFloat, {layers, B, H}, &cap, &mo) ||
      !table_of(ob, a[8], "pos_out", at::kInt, {layers, B, H}, &cap, &po) || !lengths(a[9], "new_len", &out) ||
      !integer(a[10], &protect) || (a[11] != Py_None && !dense(ob, a[11], "first", at::kInt, {B}, &first)) || !stream_of(ob, a[12], &s))
    return nullptr;
  return PyLong_FromLong(confkv_paged_evict(ob->kv, static_cast<int>(B), static_cast<int>(blocks), static_cast<int32_t*>(table),
                                            static_cast<int32_t*>(len), per_layer, static_cast<float*>(mass),
                                            static_cast<int32_t*>(pos), static_cast<int>(cap), static_cast<int32_t*>(keep),
                                            static_cast<int32_t*>(first), protect, static_cast<float*>(mo),
                                            static_cast<int32_t*>(po), static_cast<int32_t*>(out), s));
}

// object, page_table, ctx_len, path, path_len, new_len, stream
PyObject* commit(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 7)) return nullptr;
  Object* ob = pointer<Object>(a[0]);
  int64_t B, blocks, pb, cap;
  void *table, *ctx, *path, *len, *out, *s;
  if (!ready(ob) || !matrix(a[1], "page_table", &B, &blocks) || !matrix(a[3], "path", &pb, &cap) ||
      !dense(ob, a[1], "page_table", at::kInt, {B, blocks}, &table) || !dense(ob, a[2], "ctx_len", at::kInt, {B}, &ctx) ||
      !dense(ob, a[3], "path", at::kInt, {B, cap}, &path) || !dense(ob, a[4], "path_len", at::kInt, {B}, &len) ||
      !dense(ob, a[5], "new_len", at::kInt, {B}, &out) || !stream_of(ob, a[6], &s))
    return nullptr;
  return PyLong_FromLong(confkv_paged_commit(ob->kv, static_cast<int>(B), static_cast<int>(blocks),
                                             static_cast<int32_t*>(table), static_cast<int32_t*>(ctx),
                                             static_cast<int32_t*>(path), static_cast<int>(cap),
                                             static_cast<int32_t*>(len), static_cast<int32_t*>(out), s));
}

// object, parent, beams, table_in, len_in, tail_pages, table_out, len_out, stream
PyObject* fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 9)) return nullptr;
  Object* ob = pointer<Object>(a[0]);
  int beams;
  int64_t rows, blocks;
  void *parent, *tin, *lin, *tail, *tout, *lout, *s;
  if (!ready(ob) || !integer(a[2], &beams) || !matrix(a[3], "table_in", &rows, &blocks)) return nullptr;
  const at::Tensor* p = tensor(a[1], "parent");
  if (!p) return nullptr;
  if (p->dim() == 2 && beams > 0 && p->size(1) == beams && p->numel() == rows) {
    if (!dense(ob, a[1], "parent", at::kInt, {rows / beams, beams}, &parent)) return nullptr;
  } else if (!dense(ob, a[1], "parent", at::kInt, {rows}, &parent)) {
    return nullptr;
  }
  if (!dense(ob, a[3], "table_in", at::kInt, {rows, blocks}, &tin) || !dense(ob, a[4], "len_in", at::kInt, {rows}, &lin) ||
      !dense(ob, a[5], "tail_pages", at::kInt, {rows}, &tail) ||
      !dense(ob, a[6], "table_out", at::kInt, {rows, blocks}, &tout) ||
      !dense(ob, a[7], "len_out", at::kInt, {rows}, &lout) || !stream_of(ob, a[8], &s))
    return nullptr;
  return PyLong_FromLong(confkv_paged_fork(ob->kv, static_cast<int>(rows), beams, static_cast<int>(blocks),
                                           static_cast<int32_t*>(parent), static_cast<int32_t*>(tin),
                                           static_cast<int32_t*>(lin), static_cast<int32_t*>(tail),
                                           static_cast<int32_t*>(tout), static_cast<int32_t*>(lout), s));
}

// object, logits, scores, finished, pad_token, score_out, parent_out, token_out, flags_out, stream
PyObject* select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 10)) return nullptr;
  Object* ob = pointer<Object>(a[0]);
  if (!ready(ob)) return nullptr;
  const int64_t B = ob->sizes[0], W = ob->sizes[1], V = ob->sizes[2], K = ob->sizes[3];
  const at::Tensor* z = tensor(a[1], "logits");
  if (!z) return nullptr;
  int64_t stride = V;
  bool ok = z->scalar_type() == type_of(ob->dtype) && plain(ob, *z) && z->dim() == 3 &&
            z->size(0) == B && z->size(1) == W && z->size(2) == V;
  if (ok && !z->is_contiguous()) {
    stride = W > 1 ? z->stride(1) : z->stride(0);
    ok = z->stride(2) == 1 && (B == 1 || W == 1 || z->stride(0) == W * stride) && stride >= V;
  }
  if (!ok) {
    wrong("logits", "[batch, beams, vocab] of the object's type on its device, rows dense and evenly spaced", a[1]);
    return nullptr;
  }
  int pad;
  void *scores, *fin = nullptr, *so, *po, *to, *flags = nullptr, *s;
  if (!dense(ob, a[2], "scores", at::kFloat, {B, W}, &scores) || !integer(a[4], &pad) ||
      !dense(ob, a[5], "score_out", at::kFloat, {B, K}, &so) || !dense(ob, a[6], "parent_out", at::kInt, {B, K}, &po) ||
      !dense(ob, a[7], "token_out", at::kInt, {B, K}, &to))
    return nullptr;
  if (a[3] != Py_None) {
    const at::Tensor* f = tensor(a[3], "finished");
    if (!f || !dense(ob, a[3], "finished", f->scalar_type() == at::kByte ? at::kByte : at::kBool, {B, W}, &fin)) return nullptr;
  }
  if (a[8] != Py_None && !dense(ob, a[8], "flags_out", at::kInt, {B, W}, &flags)) return nullptr;
  if (!stream_of(ob, a[9], &s)) return nullptr;
  return PyLong_FromLong(confkv_beam_select(z->data_ptr(), ob->dtype, stride, static_cast<int>(B), static_cast<int>(W),
                                            static_cast<int>(V), static_cast<int>(K), static_cast<float*>(scores),
                                            static_cast<uint8_t*>(fin), pad, static_cast<float*>(so),
                                            static_cast<int32_t*>(po), static_cast<int32_t*>(to),
                                            static_cast<int32_t*>(flags), ob->ws, ob->ws_bytes, ob->device, s));
}

// handle, workspace, its bytes, home stream, four sizes, device, type code -> the object's address
PyObject* make(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count(n, 10)) return nullptr;
  Object* ob = new (std::nothrow) Object();
  if (!ob) return PyErr_NoMemory();
  ob->kv = pointer<confkv_paged>(a[0]);
  ob->ws = pointer<void>(a[1]);
  ob->ws_bytes = PyLong_AsSize_t(a[2]);
  ob->home = static_cast<cudaStream_t>(pointer<void>(a[3]));
  for (int i = 0; i < 4; ++i) ob->sizes[i] = PyLong_AsLongLong(a[4 + i]);
  if (!integer(a[8], &ob->device) || !integer(a[9], &ob->dtype) || PyErr_Occurred()) {
    delete ob;
    return nullptr;
  }
  return PyLong_FromVoidPtr(ob);
}

// object -> whether a call ran on another stream than the scratch's; the object ends
PyObject* release(PyObject*, PyObject* o) {
  Object* ob = pointer<Object>(o);
  if (PyErr_Occurred()) return nullptr;
  const int away = ob ? ob->away : 0;
  delete ob;
  return PyBool_FromLong(away);
}

// torch throws at tensors without plain memory (sparse, nested, meta): no exception
// may pass a C entry.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* safe(PyObject* self, PyObject* const* a, Py_ssize_t n) noexcept {
  try {
    return F(self, a, n);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_ValueError, "a tensor cannot be read");
  }
  return nullptr;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(safe<f>))
PyMethodDef kMethods[] = {{"append", FAST(append), METH_FASTCALL, nullptr},
                          {"append_normed", FAST(append_normed), METH_FASTCALL, nullptr},
                          {"attend", FAST(attend), METH_FASTCALL, nullptr},
                          {"attend_shared", FAST(attend_shared), METH_FASTCALL, nullptr},
                          {"weigh", FAST(weigh), METH_FASTCALL, nullptr},
                          {"evict", FAST(evict), METH_FASTCALL, nullptr},
                          {"commit", FAST(commit), METH_FASTCALL, nullptr},
                          {"fork", FAST(fork), METH_FASTCALL, nullptr},
                          {"select", FAST(select), METH_FASTCALL, nullptr},
                          {"make", FAST(make), METH_FASTCALL, nullptr},
                          {"release", release, METH_O, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_paged_ops", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_ops() { return PyModule_Create(&kModule); }
