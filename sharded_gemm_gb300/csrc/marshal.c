/* marshal.c -- the Python side of the attention-side entry points: checks that
 * the tensors it is given can be described to the C ABI and calls the library.
 *
 * These calls stand between kernels of a few microseconds, several per layer of
 * a decode step.  Marshalled in Python one took about 20 us; here it takes about
 * as long as the launch.  Nothing is kept between calls.
 *
 * Every function takes the library function's address first and allocates the
 * outputs that are None.  It returns them, or the library's error code as an int.
 * With address 0 it calls nothing and returns (outputs, the tuple of arguments
 * that it would have passed, pointer arrays as bytes), for prepare(). */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "../../include/tp_api.h"

#define MOST_RANKS 64

static PyObject *s_shape, *s_stride, *s_dtype, *s_get_device, *s_data_ptr, *s_cuda_stream;
/* set by init() */
static PyObject *t_f32, *t_bf16, *t_f16, *t_i32, *t_i64, *raw_stream, *torch_empty;
static PyObject *empty_names; /* ("dtype", "device") */

static int dtype_code(PyObject *dtype) {
  return dtype == t_bf16 ? TP_BF16 : dtype == t_f16 ? TP_F16 : dtype == t_f32 ? TP_F32 : -1;
}

typedef struct {
  uint64_t ptr;
  int nd;
  int64_t shape[6], stride[6];
  PyObject *dtype; /* a singleton: no reference kept */
  long dev;
} Info;

static int ints(PyObject *tuple, int64_t *to, int *n, const char *name) {
  if (!tuple) return -1;
  if (!PyTuple_Check(tuple) || PyTuple_GET_SIZE(tuple) > 6) {
    PyErr_Format(PyExc_ValueError, "%s has too many dimensions", name);
    Py_DECREF(tuple);
    return -1;
  }
  *n = (int)PyTuple_GET_SIZE(tuple);
  for (int i = 0; i < *n; ++i) to[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
  Py_DECREF(tuple);
  return PyErr_Occurred() ? -1 : 0;
}

static int whole(PyObject *v, int64_t *to) {
  if (!v) return -1;
  *to = (int64_t)PyLong_AsUnsignedLongLongMask(v);
  Py_DECREF(v);
  return PyErr_Occurred() ? -1 : 0;
}

static int info_of(PyObject *t, Info *o, const char *name) {
  int nd;
  int64_t v;
  if (ints(PyObject_GetAttr(t, s_shape), o->shape, &o->nd, name)) return -1;
  if (ints(PyObject_CallMethodNoArgs(t, s_stride), o->stride, &nd, name)) return -1;
  PyObject *d = PyObject_GetAttr(t, s_dtype);
  if (!d) return -1;
  o->dtype = d;
  Py_DECREF(d);
  if (whole(PyObject_CallMethodNoArgs(t, s_get_device), &v)) return -1;
  o->dev = (long)v;
  if (whole(PyObject_CallMethodNoArgs(t, s_data_ptr), &v)) return -1;
  o->ptr = (uint64_t)v;
  if (o->dev < 0) {
    PyErr_Format(PyExc_ValueError, "%s must be a CUDA tensor", name);
    return -1;
  }
  return 0;
}

/* A per-rank argument: a list of N tensors, or one tensor whose first dimension
 * is the ranks. */
typedef struct {
  int n, dt;
  uint64_t ptr[MOST_RANKS];
  int64_t shape[5], stride[5];
  PyObject *dtype;
  long dev;
} Ranks;

static int ranks_of(PyObject *x, Ranks *o, int dim, const char *name) {
  Info f;
  int first = 0;
  if (PyList_Check(x) || PyTuple_Check(x)) {
    const Py_ssize_t n = PySequence_Fast_GET_SIZE(x);
    if (n < 1) {
      PyErr_Format(PyExc_ValueError, "%s: no ranks", name);
      return -1;
    }
    if (info_of(PySequence_Fast_GET_ITEM(x, 0), &f, name)) return -1;
    o->n = (int)n;
    o->ptr[0] = f.ptr;
    for (Py_ssize_t i = 1; i < n && i < MOST_RANKS; ++i) {
      Info g;
      if (info_of(PySequence_Fast_GET_ITEM(x, i), &g, name)) return -1;
      int same = g.nd == f.nd && g.dtype == f.dtype && g.dev == f.dev;
      for (int d = 0; same && d < f.nd; ++d) same = g.shape[d] == f.shape[d] && g.stride[d] == f.stride[d];
      if (!same) {
        PyErr_Format(PyExc_ValueError, "%s: all ranks need one shape, stride, dtype and device", name);
        return -1;
      }
      o->ptr[i] = g.ptr;
    }
  } else {
    if (info_of(x, &f, name)) return -1;
    first = 1;
  }
  if (f.nd != dim + first) {
    PyErr_Format(PyExc_ValueError, "%s: each rank's tensor must be %d-D", name, dim);
    return -1;
  }
  o->dt = dtype_code(f.dtype);
  if (o->dt < 0) {
    PyErr_Format(PyExc_TypeError, "%s: unsupported dtype %S", name, f.dtype);
    return -1;
  }
  if (first) {
    o->n = f.shape[0] > 1 << 20 ? 1 << 20 : (int)f.shape[0];
    const uint64_t step = (uint64_t)f.stride[0] * (o->dt == TP_F32 ? 4 : 2);
    for (int i = 0; i < o->n && i < MOST_RANKS; ++i) o->ptr[i] = f.ptr + i * step;
  }
  for (int d = 0; d < dim; ++d) o->shape[d] = f.shape[first + d], o->stride[d] = f.stride[first + d];
  o->dtype = f.dtype;
  o->dev = f.dev;
  return 0;
}

/* Row stride of a per-rank matrix. */
static int ld_of(const Ranks *o, int64_t *ld, const char *name) {
  if (o->stride[1] != 1 && o->shape[1] > 1) {
    PyErr_Format(PyExc_ValueError, "%s must have unit column stride", name);
    return -1;
  }
  *ld = o->shape[0] > 1 ? o->stride[0] : o->shape[1];
  return 0;
}

/* Device pointer of a contiguous 1-D parameter array (None: 0). */
static int param_of(PyObject *t, uint64_t *ptr, PyObject *dtype, int64_t n, long dev, const char *name) {
  *ptr = 0;
  if (t == Py_None) return 0;
  Info f;
  if (info_of(t, &f, name)) return -1;
  if (f.dtype != dtype) {
    PyErr_Format(PyExc_TypeError, "%s must be %S", name, dtype);
    return -1;
  }
  if (f.dev != dev) {
    PyErr_Format(PyExc_ValueError, "%s must be on device %ld", name, dev);
    return -1;
  }
  if (f.nd != 1 || f.shape[0] != n || (n > 1 && f.stride[0] != 1)) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous with %lld elements", name, (long long)n);
    return -1;
  }
  *ptr = f.ptr;
  return 0;
}

static int stream_of(PyObject *stream, long dev, uint64_t *to) {
  int64_t v;
  PyObject *s;
  if (stream == Py_None) {
    PyObject *d = PyLong_FromLong(dev);
    s = d ? PyObject_CallOneArg(raw_stream, d) : NULL;
    Py_XDECREF(d);
  } else if (PyLong_Check(stream)) {
    s = Py_NewRef(stream);
  } else {
    s = PyObject_GetAttr(stream, s_cuda_stream);
  }
  if (whole(s, &v)) return -1;
  *to = (uint64_t)v;
  return 0;
}

typedef struct {
  Ranks k, v;
  int64_t pages, ld;
  int Hk, page, D;
} Cache;

static int cache_of(PyObject *k, PyObject *v, Cache *c) {
  if (ranks_of(k, &c->k, 4, "k_cache") || ranks_of(v, &c->v, 4, "v_cache")) return -1;
  int same = c->k.n == c->v.n && c->k.dtype == c->v.dtype && c->k.dev == c->v.dev;
  for (int d = 0; d < 4; ++d) same = same && c->k.shape[d] == c->v.shape[d] && c->k.stride[d] == c->v.stride[d];
  if (!same) {
    PyErr_SetString(PyExc_ValueError, "k_cache and v_cache need the same ranks, shape, strides, dtype and device");
    return -1;
  }
  const int64_t P = c->k.shape[0], Hk = c->k.shape[1], page = c->k.shape[2], D = c->k.shape[3];
  if (Hk > 1 << 20 || page > 1 << 20 || D > 1 << 20) {
    PyErr_SetString(PyExc_ValueError, "the cache's pages are too large");
    return -1;
  }
  if ((c->k.stride[3] != 1 && D > 1) || (c->k.stride[2] != D && page > 1) || (c->k.stride[1] != page * D && Hk > 1)) {
    PyErr_SetString(PyExc_ValueError, "the heads, rows and values of a cache page must be contiguous");
    return -1;
  }
  c->pages = P, c->Hk = (int)Hk, c->page = (int)page, c->D = (int)D;
  c->ld = P > 1 ? c->k.stride[0] : Hk * page * D;
  return 0;
}

/* The heads of D in `cols` columns. */
static int heads_of(int64_t cols, int D, int *heads, const char *name) {
  if (D < 1 || cols % D || cols / D > 1 << 20) {
    PyErr_Format(PyExc_ValueError, "%s: %lld columns are not whole heads of %d", name, (long long)cols, D);
    return -1;
  }
  *heads = (int)(cols / D);
  return 0;
}

/* torch.empty(shape, dtype=dtype, device=dev): a new reference. */
static PyObject *new_tensor(int nd, const int64_t *shape, PyObject *dtype, long dev) {
  PyObject *size = PyTuple_New(nd), *device = PyLong_FromLong(dev), *t = NULL;
  int ok = size && device;
  for (int d = 0; ok && d < nd; ++d) {
    PyObject *n = PyLong_FromLongLong(shape[d]);
    if (n) PyTuple_SET_ITEM(size, d, n);
    else ok = 0;
  }
  if (ok) {
    PyObject *args[3] = {size, dtype, device};
    t = PyObject_Vectorcall(torch_empty, args, 1, empty_names);
  }
  Py_XDECREF(size);
  Py_XDECREF(device);
  return t;
}
/* The per-rank output `given`, or where it is None a new (n, rows, cols) tensor:
 * a new reference in *keep, described in *o. */
static int output_of(PyObject *given, int n, int64_t rows, int64_t cols, PyObject *dtype, long dev, PyObject **keep,
                     Ranks *o) {
  if (given == Py_None) {
    const int64_t shape[3] = {n, rows, cols};
    *keep = new_tensor(3, shape, dtype, dev);
  } else {
    *keep = Py_NewRef(given);
  }
  if (!*keep) return -1;
  if (ranks_of(*keep, o, 2, "out")) {
    Py_CLEAR(*keep);
    return -1;
  }
  return 0;
}
/* What a function returns: its outputs (a new reference, taken), or the error code. */
static PyObject *answer(PyObject *out, int rc) {
  if (rc == TP_OK) return out;
  Py_DECREF(out);
  return PyLong_FromLong(rc);
}

static PyObject *bytes_of(const Ranks *o) {
  return PyBytes_FromStringAndSize((const char *)o->ptr, 8 * (o->n < MOST_RANKS ? o->n : MOST_RANKS));
}

#define P(x) ((void *)(uintptr_t)(x))
#define A(r) ((void *const *)(uintptr_t)(r).ptr)
#define CA(r) ((const void *const *)(uintptr_t)(r).ptr)

/* append(fn, qkv, k_cache, v_cache, slots, positions, rope, q_norm, k_norm, eps, interleaved, out, stream) */
static PyObject *m_append(PyObject *self, PyObject *const *a, Py_ssize_t na) {
  if (na != 13) return PyErr_Format(PyExc_TypeError, "append takes 13 arguments");
  void *fn = PyLong_AsVoidPtr(a[0]);
  Cache c;
  Ranks x, out;
  int64_t ld, ldq, rows = 0, rot = 0;
  int H, Hq, inter, rc;
  double eps;
  uint64_t slots, positions, rope = 0, qn, kn, stream;
  PyObject *keep = NULL;
  if (cache_of(a[2], a[3], &c) || ranks_of(a[1], &x, 2, "qkv")) return NULL;
  if (x.n != c.k.n || x.dev != c.k.dev) {
    PyErr_SetString(PyExc_ValueError, "qkv and the caches need the same ranks on one device");
    return NULL;
  }
  if (ld_of(&x, &ld, "qkv") || heads_of(x.shape[1], c.D, &H, "qkv")) return NULL;
  Hq = H - 2 * c.Hk;
  const int64_t T = x.shape[0];
  if (Hq < 1)
    return PyErr_Format(PyExc_ValueError, "qkv holds no query heads besides 2 * %d key and value heads", c.Hk);
  if (output_of(a[11], c.k.n, T, (int64_t)Hq * c.D, c.k.dtype, c.k.dev, &keep, &out)) return NULL;
  if (ld_of(&out, &ldq, "out")) goto fail;
  if (out.n != c.k.n || out.shape[0] != T || out.shape[1] != (int64_t)Hq * c.D || out.dtype != c.k.dtype ||
      out.dev != c.k.dev) {
    PyErr_SetString(PyExc_ValueError, "out must be (T, Hq * D) per rank in the cache's dtype");
    goto fail;
  }
  if (a[6] != Py_None) {
    Info f;
    if (info_of(a[6], &f, "rope")) goto fail;
    if (f.dtype != t_f32 || f.nd != 2 || f.dev != c.k.dev || (f.shape[1] > 1 && f.stride[1] != 1) ||
        (f.shape[0] > 1 && f.stride[0] != f.shape[1]) || f.shape[1] > 1 << 20) {
      PyErr_SetString(PyExc_ValueError,
                      "rope must be a contiguous float32 (positions, rope_dim) tensor on the caches' device");
      goto fail;
    }
    if (a[5] == Py_None) {
      PyErr_SetString(PyExc_ValueError, "rope needs positions");
      goto fail;
    }
    rope = f.ptr, rows = f.shape[0], rot = f.shape[1];
  }
  eps = PyFloat_AsDouble(a[9]);
  inter = PyObject_IsTrue(a[10]);
  if (PyErr_Occurred() || param_of(a[4], &slots, t_i64, T, c.k.dev, "slots") ||
      param_of(a[5], &positions, t_i32, T, c.k.dev, "positions") ||
      param_of(a[7], &qn, t_f32, c.D, c.k.dev, "q_norm") || param_of(a[8], &kn, t_f32, c.D, c.k.dev, "k_norm") ||
      stream_of(a[12], c.k.dev, &stream))
    goto fail;
  if (!fn)
    return Py_BuildValue("N(iNLLiiiiKKdKLiiKKNLNNLiLiK)", keep, x.n, bytes_of(&x), T, ld, x.dt, Hq, c.Hk, c.D, qn, kn,
                         eps, rope, rows, (int)rot, inter, positions, slots, bytes_of(&out), ldq, bytes_of(&c.k),
                         bytes_of(&c.v), c.pages, c.page, c.ld, c.k.dt, stream);
  Py_BEGIN_ALLOW_THREADS;
  rc = ((__typeof__(&tp_qkv_append))fn)(x.n, CA(x), T, ld, (tp_dtype)x.dt, Hq, c.Hk, c.D, P(qn), P(kn), (float)eps,
                                        P(rope), rows, (int)rot, inter, P(positions), P(slots), A(out), ldq, A(c.k),
                                        A(c.v), c.pages, c.page, c.ld, (tp_dtype)c.k.dt, P(stream));
  Py_END_ALLOW_THREADS;
  return answer(keep, rc);
fail:
  Py_XDECREF(keep);
  return NULL;
}

/* What both attentions share. */
typedef struct {
  Cache c;
  Ranks q, out;
  int64_t T, ldq, ldo, B, width, ldt;
  int Hq;
  uint64_t table;
  PyObject *keep;
} Attn;

/* On success o->keep is a new reference to the output. */
static int attn_of(PyObject *q, PyObject *k, PyObject *v, PyObject *table, PyObject *out, Attn *o) {
  Info f;
  o->keep = NULL;
  if (cache_of(k, v, &o->c) || ranks_of(q, &o->q, 2, "q")) return -1;
  if (o->q.n != o->c.k.n || o->q.dev != o->c.k.dev) {
    PyErr_SetString(PyExc_ValueError, "q and the caches need the same ranks on one device");
    return -1;
  }
  if (o->q.dtype != o->c.k.dtype) {
    PyErr_SetString(PyExc_TypeError, "q must have the caches' dtype");
    return -1;
  }
  if (ld_of(&o->q, &o->ldq, "q") || heads_of(o->q.shape[1], o->c.D, &o->Hq, "q") || info_of(table, &f, "block_table"))
    return -1;
  if (f.dtype != t_i32 || f.nd != 2 || f.dev != o->c.k.dev) {
    PyErr_SetString(PyExc_ValueError, "block_table must be a 2-D int32 tensor on the caches' device");
    return -1;
  }
  if (f.shape[1] > 1 && f.stride[1] != 1) {
    PyErr_SetString(PyExc_ValueError, "block_table must have unit column stride");
    return -1;
  }
  if (output_of(out, o->q.n, o->q.shape[0], o->q.shape[1], o->q.dtype, o->q.dev, &o->keep, &o->out)) return -1;
  if (o->out.n != o->q.n || o->out.shape[0] != o->q.shape[0] || o->out.shape[1] != o->q.shape[1] ||
      o->out.dtype != o->q.dtype || o->out.dev != o->q.dev) {
    PyErr_SetString(PyExc_ValueError, "out must have q's shape per rank and its dtype");
    Py_CLEAR(o->keep);
    return -1;
  }
  if (ld_of(&o->out, &o->ldo, "out")) {
    Py_CLEAR(o->keep);
    return -1;
  }
  o->T = o->q.shape[0], o->B = f.shape[0], o->width = f.shape[1];
  o->ldt = f.shape[0] > 1 ? f.stride[0] : f.shape[1];
  o->table = f.ptr;
  return 0;
}

/* scale (None: 1 / sqrt(D)), softcap, window */
static int scores_of(PyObject *const *a, int D, double *scale, double *cap, int *window) {
  *scale = a[0] == Py_None ? 1.0 / __builtin_sqrt((double)D) : PyFloat_AsDouble(a[0]);
  *cap = PyFloat_AsDouble(a[1]);
  const long w = PyLong_AsLong(a[2]);
  *window = w > 0x7fffffff ? 0x7fffffff : w < -1 ? -1 : (int)w;
  return PyErr_Occurred() ? -1 : 0;
}

/* decode(fn, q, k_cache, v_cache, block_table, seq_lens, scale, softcap, window, out, stream) */
static PyObject *m_decode(PyObject *self, PyObject *const *a, Py_ssize_t na) {
  if (na != 11) return PyErr_Format(PyExc_TypeError, "decode takes 11 arguments");
  void *fn = PyLong_AsVoidPtr(a[0]);
  Attn o;
  uint64_t lens, stream;
  double scale, cap;
  int window;
  if (attn_of(a[1], a[2], a[3], a[4], a[9], &o)) return NULL;
  if (o.B != o.T) {
    PyErr_SetString(PyExc_ValueError, "block_table needs one row per sequence");
    Py_DECREF(o.keep);
    return NULL;
  }
  if (param_of(a[5], &lens, t_i32, o.B, o.c.k.dev, "seq_lens") || scores_of(a + 6, o.c.D, &scale, &cap, &window) ||
      stream_of(a[10], o.c.k.dev, &stream)) {
    Py_DECREF(o.keep);
    return NULL;
  }
  const Cache *c = &o.c;
  if (!fn)
    return Py_BuildValue("N(iNLLiiiNNLiLKLLKddiiNLK)", o.keep, o.q.n, bytes_of(&o.q), o.T, o.ldq, o.Hq, c->Hk, c->D,
                         bytes_of(&c->k), bytes_of(&c->v), c->pages, c->page, c->ld, o.table, o.width, o.ldt, lens,
                         scale, cap, window, c->k.dt, bytes_of(&o.out), o.ldo, stream);
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = ((__typeof__(&tp_paged_decode))fn)(o.q.n, CA(o.q), o.T, o.ldq, o.Hq, c->Hk, c->D, A(c->k), A(c->v), c->pages,
                                          c->page, c->ld, P(o.table), o.width, o.ldt, P(lens), (float)scale, (float)cap,
                                          window, (tp_dtype)c->k.dt, A(o.out), o.ldo, P(stream));
  Py_END_ALLOW_THREADS;
  return answer(o.keep, rc);
}

/* prefill(fn, q, k_cache, v_cache, block_table, cu_seqlens, seq_lens, prefix_lens, scale, softcap, window, out, stream) */
static PyObject *m_prefill(PyObject *self, PyObject *const *a, Py_ssize_t na) {
  if (na != 13) return PyErr_Format(PyExc_TypeError, "prefill takes 13 arguments");
  void *fn = PyLong_AsVoidPtr(a[0]);
  Attn o;
  uint64_t cu, lens, prefix, stream;
  double scale, cap;
  int window;
  if (attn_of(a[1], a[2], a[3], a[4], a[11], &o)) return NULL;
  if (param_of(a[5], &cu, t_i32, o.B + 1, o.c.k.dev, "cu_seqlens") ||
      param_of(a[6], &lens, t_i32, o.B, o.c.k.dev, "seq_lens") ||
      param_of(a[7], &prefix, t_i32, o.B, o.c.k.dev, "prefix_lens") ||
      scores_of(a + 8, o.c.D, &scale, &cap, &window) || stream_of(a[12], o.c.k.dev, &stream)) {
    Py_DECREF(o.keep);
    return NULL;
  }
  const Cache *c = &o.c;
  if (!fn)
    return Py_BuildValue("N(iNLLiiiNNLiLKLLLKKKddiiNLK)", o.keep, o.q.n, bytes_of(&o.q), o.T, o.ldq, o.Hq, c->Hk, c->D,
                         bytes_of(&c->k), bytes_of(&c->v), c->pages, c->page, c->ld, o.table, o.B, o.width, o.ldt, cu,
                         lens, prefix, scale, cap, window, c->k.dt, bytes_of(&o.out), o.ldo, stream);
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = ((__typeof__(&tp_paged_prefill))fn)(o.q.n, CA(o.q), o.T, o.ldq, o.Hq, c->Hk, c->D, A(c->k), A(c->v), c->pages,
                                           c->page, c->ld, P(o.table), o.B, o.width, o.ldt, P(cu), P(lens), P(prefix),
                                           (float)scale, (float)cap, window, (tp_dtype)c->k.dt, A(o.out), o.ldo,
                                           P(stream));
  Py_END_ALLOW_THREADS;
  return answer(o.keep, rc);
}

/* sample(fn, logits, u, temperature, top_k, top_p, min_p, tokens, logprobs, stream) -> (tokens, logprobs) */
static PyObject *m_sample(PyObject *self, PyObject *const *a, Py_ssize_t na) {
  if (na != 10) return PyErr_Format(PyExc_TypeError, "sample takes 10 arguments");
  void *fn = PyLong_AsVoidPtr(a[0]);
  Info f;
  uint64_t u, t, k, p, m, tokens, logprobs, stream;
  if (info_of(a[1], &f, "logits")) return NULL;
  const int dt = dtype_code(f.dtype);
  if (dt < 0) return PyErr_Format(PyExc_TypeError, "logits: unsupported dtype %S", f.dtype);
  if (f.nd != 2 || (f.shape[1] > 1 && f.stride[1] != 1))
    return PyErr_Format(PyExc_ValueError, "logits must be 2-D with unit column stride");
  const int64_t B = f.shape[0], V = f.shape[1], ld = B > 1 ? f.stride[0] : V;
  if (param_of(a[2], &u, t_f32, B, f.dev, "u") || param_of(a[3], &t, t_f32, B, f.dev, "temperature") ||
      param_of(a[4], &k, t_i32, B, f.dev, "top_k") || param_of(a[5], &p, t_f32, B, f.dev, "top_p") ||
      param_of(a[6], &m, t_f32, B, f.dev, "min_p") || stream_of(a[9], f.dev, &stream))
    return NULL;
  PyObject *tk = a[7] == Py_None ? new_tensor(1, &B, t_i64, f.dev) : Py_NewRef(a[7]);
  PyObject *lp = !tk ? NULL : a[8] == Py_None ? new_tensor(1, &B, t_f32, f.dev) : Py_NewRef(a[8]);
  PyObject *out = lp ? PyTuple_Pack(2, tk, lp) : NULL;
  Py_XDECREF(tk); /* the tuple keeps them */
  Py_XDECREF(lp);
  if (!out) return NULL;
  if (param_of(PyTuple_GET_ITEM(out, 0), &tokens, t_i64, B, f.dev, "tokens") ||
      param_of(PyTuple_GET_ITEM(out, 1), &logprobs, t_f32, B, f.dev, "logprobs")) {
    Py_DECREF(out);
    return NULL;
  }
  if (!fn)
    return Py_BuildValue("N(KLLLiKKKKKKKK)", out, f.ptr, B, V, ld, dt, u, t, k, p, m, tokens, logprobs, stream);
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = ((__typeof__(&tp_sample))fn)(P(f.ptr), B, V, ld, (tp_dtype)dt, P(u), P(t), P(k), P(p), P(m), P(tokens),
                                    P(logprobs), P(stream));
  Py_END_ALLOW_THREADS;
  return answer(out, rc);
}

/* ---- the operators that serve many requests at once */

/* A 2-D int32 matrix: pointer, rows, columns and row stride. */
static int table_of(PyObject *t, long dev, uint64_t *ptr, int64_t *rows, int64_t *cols, int64_t *ld, const char *name) {
  Info f;
  if (info_of(t, &f, name)) return -1;
  if (f.dtype != t_i32 || f.nd != 2 || f.dev != dev || (f.shape[0] > 0 && f.shape[1] > 1 && f.stride[1] != 1)) {
    PyErr_Format(PyExc_ValueError, "%s must be a 2-D int32 tensor with unit column stride on device %ld", name, dev);
    return -1;
  }
  *ptr = f.ptr, *rows = f.shape[0], *cols = f.shape[1], *ld = f.shape[0] > 1 ? f.stride[0] : f.shape[1];
  return 0;
}

static int length_of(PyObject *t, int64_t *n, long *dev, const char *name) {
  Info f;
  if (info_of(t, &f, name)) return -1;
  if (f.nd != 1) {
    PyErr_Format(PyExc_ValueError, "%s must be 1-D", name);
    return -1;
  }
  *n = f.shape[0], *dev = f.dev;
  return 0;
}

/* The tensor `given`, or where it is None a new one of n values: a new reference. */
static PyObject *vector_or_new(PyObject *given, int64_t n, PyObject *dtype, long dev) {
  return given == Py_None ? new_tensor(1, &n, dtype, dev) : Py_NewRef(given);
}

/* plan(fn, counts, seq_lens, owned, block_table, free_pages, free_count, page, tokens, rejected, out, stream) -> the
 * seven outputs: lengths, pages, free count, missing, offsets, positions, slots */
static PyObject *m_plan(PyObject *self, PyObject *const *a, Py_ssize_t na) {
  if (na != 12) return PyErr_Format(PyExc_TypeError, "plan takes 12 arguments");
  void *fn = PyLong_AsVoidPtr(a[0]);
  int64_t B, rows, width, ld, pages;
  long dev, pool_dev;
  uint64_t counts, lens, owned, table, pool, free_n, rejected, stream, to[7];
  if (length_of(a[1], &B, &dev, "counts") || param_of(a[1], &counts, t_i32, B, dev, "counts") ||
      param_of(a[2], &lens, t_i32, B, dev, "seq_lens") || param_of(a[3], &owned, t_i32, B, dev, "owned") ||
      table_of(a[4], dev, &table, &rows, &width, &ld, "block_table"))
    return NULL;
  if (rows != B) return PyErr_Format(PyExc_ValueError, "block_table needs one row per sequence");
  if (length_of(a[5], &pages, &pool_dev, "free_pages") || param_of(a[5], &pool, t_i32, pages, dev, "free_pages") ||
      param_of(a[6], &free_n, t_i32, 1, dev, "free_count") || param_of(a[9], &rejected, t_i32, B, dev, "rejected") ||
      stream_of(a[11], dev, &stream))
    return NULL;
  const long page = PyLong_AsLong(a[7]);
  const int64_t T = PyLong_AsLongLong(a[8]);
  if (PyErr_Occurred()) return NULL;
  if (T < 0 || T > 0x7fffffff) return PyErr_Format(PyExc_ValueError, "tokens must be in 0..2^31 - 1");
  if (page != (int)page) return PyErr_Format(PyExc_ValueError, "page must be a power of two in 16..256");
  if (a[10] != Py_None && (!(PyTuple_Check(a[10]) || PyList_Check(a[10])) || PySequence_Fast_GET_SIZE(a[10]) != 7))
    return PyErr_Format(PyExc_ValueError, "out must be the seven outputs");
  static const char *const names[7] = {"out.seq_lens",   "out.owned",     "out.free_count", "out.missing",
                                       "out.cu_seqlens", "out.positions", "out.slots"};
  const int64_t sizes[7] = {B, B, 1, 1, B + 1, T, T};
  PyObject *out = PyTuple_New(7);
  if (!out) return NULL;
  for (int i = 0; i < 7; ++i) {
    PyObject *dtype = i == 6 ? t_i64 : t_i32;
    PyObject *t = a[10] == Py_None ? new_tensor(1, &sizes[i], dtype, dev) : Py_NewRef(PySequence_Fast_GET_ITEM(a[10], i));
    if (!t) goto fail;
    PyTuple_SET_ITEM(out, i, t);
    if (t == Py_None) {
      PyErr_Format(PyExc_ValueError, "%s is None", names[i]);
      goto fail;
    }
    if (param_of(t, &to[i], dtype, sizes[i], dev, names[i])) goto fail;
  }
  if (!fn)
    return Py_BuildValue("N(LKKKKKLLKLKiLKKKKKKKK)", out, B, counts, rejected, lens, owned, table, width, ld, pool, pages,
                         free_n, (int)page, T, to[0], to[1], to[2], to[3], to[4], to[5], to[6], stream);
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = ((__typeof__(&tp_paged_plan))fn)(B, P(counts), P(rejected), P(lens), P(owned), P(table), width, ld, P(pool), pages,
                                        P(free_n), (int)page, T, P(to[0]), P(to[1]), P(to[2]), P(to[3]), P(to[4]),
                                        P(to[5]), P(to[6]), P(stream));
  Py_END_ALLOW_THREADS;
  return answer(out, rc);
fail:
  Py_DECREF(out);
  return NULL;
}

static int64_t group_ints(int64_t T, int64_t n) { return 4 + 4 * (T < n + 1 ? T : n + 1) + T; }

/* groups(fn, adapters, tokens, n, cu_seqlens, out, stream) -> the plan */
static PyObject *m_groups(PyObject *self, PyObject *const *a, Py_ssize_t na) {
  if (na != 7) return PyErr_Format(PyExc_TypeError, "groups takes 7 arguments");
  void *fn = PyLong_AsVoidPtr(a[0]);
  int64_t B;
  long dev;
  uint64_t ids, cu, plan, stream;
  const int64_t T = PyLong_AsLongLong(a[2]), n = PyLong_AsLongLong(a[3]);
  if (PyErr_Occurred()) return NULL;
  if (T < 0 || T > 0x7fffffff || n < 1 || n > 0x7fffffff)
    return PyErr_Format(PyExc_ValueError, "tokens must be in 0..2^31 - 1, n in 1..2^31 - 1");
  if (length_of(a[1], &B, &dev, "adapters") || param_of(a[1], &ids, t_i32, B, dev, "adapters") ||
      param_of(a[4], &cu, t_i32, B + 1, dev, "cu_seqlens") || stream_of(a[6], dev, &stream))
    return NULL;
  PyObject *out = vector_or_new(a[5], group_ints(T, n), t_i32, dev);
  if (!out) return NULL;
  if (param_of(out, &plan, t_i32, group_ints(T, n), dev, "out")) {
    Py_DECREF(out);
    return NULL;
  }
  if (!fn) return Py_BuildValue("N(LKKLLKK)", out, B, ids, cu, T, n, plan, stream);
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = ((__typeof__(&tp_lora_plan))fn)(B, P(ids), P(cu), T, n, P(plan), P(stream));
  Py_END_ALLOW_THREADS;
  return answer(out, rc);
}

/* A pool of adapters (n, rows, cols): contiguous, in x's 16-bit dtype. */
static int pool_of(const Ranks *o, PyObject *dtype, long dev, const char *name) {
  if (o->dtype != dtype || o->dev != dev || dtype == t_f32) {
    PyErr_Format(PyExc_ValueError, "%s must have x's 16-bit dtype and its device", name);
    return -1;
  }
  if ((o->shape[2] > 1 && o->stride[2] != 1) || (o->shape[1] > 1 && o->stride[1] != o->shape[2]) ||
      (o->shape[0] > 1 && o->stride[0] != o->shape[1] * o->shape[2])) {
    PyErr_Format(PyExc_ValueError, "%s must be contiguous", name);
    return -1;
  }
  return 0;
}

/* An argument that is one tensor, as a list of one. */
static int one_of(PyObject *t, Ranks *o, int dim, const char *name) {
  if (PyList_Check(t) || PyTuple_Check(t)) {
    PyErr_Format(PyExc_ValueError, "%s must be one tensor", name);
    return -1;
  }
  PyObject *list = PyTuple_Pack(1, t);
  if (!list) return -1;
  const int rc = ranks_of(list, o, dim, name);
  Py_DECREF(list);
  return rc;
}

/* lora(fn, column, x, a, b, plan, workspace, y, scales, out, stream) -> out; workspace(T, R, device, stream) gives a
 * step of many tokens its memory */
static PyObject *m_lora(PyObject *self, PyObject *const *a, Py_ssize_t na) {
  if (na != 11) return PyErr_Format(PyExc_TypeError, "lora takes 11 arguments");
  void *fn = PyLong_AsVoidPtr(a[0]);
  const int column = PyObject_IsTrue(a[1]);
  Ranks x, A_, B_, y, out;
  int64_t ldx, ldy, ldo, size;
  uint64_t plan, room = 0, scales, stream;
  int64_t floats;
  long dev;
  PyObject *to = a[9] == Py_None ? a[7] : a[9];
  if (column ? one_of(a[2], &x, 2, "x") || one_of(a[3], &A_, 3, "a") || ranks_of(a[4], &B_, 3, "b") ||
                   ranks_of(a[7], &y, 2, "y") || ranks_of(to, &out, 2, "out")
             : ranks_of(a[2], &x, 2, "x") || ranks_of(a[3], &A_, 3, "a") || one_of(a[4], &B_, 3, "b") ||
                   one_of(a[7], &y, 2, "y") || one_of(to, &out, 2, "out"))
    return NULL;
  if (pool_of(&A_, x.dtype, x.dev, "a") || pool_of(&B_, x.dtype, x.dev, "b")) return NULL;
  if (A_.n != x.n || B_.n != y.n) {
    PyErr_SetString(PyExc_ValueError, column ? "b and y need the same ranks" : "x and a need the same ranks");
    return NULL;
  }
  const int64_t T = x.shape[0], K = x.shape[1], n = A_.shape[0], R = A_.shape[1], O = B_.shape[1];
  if (A_.shape[2] != K || B_.shape[0] != n || B_.shape[2] != R || y.shape[0] != T || y.shape[1] != O || y.dev != x.dev) {
    PyErr_SetString(PyExc_ValueError, "per rank x (T, K), a (n, R, K), b (n, O, R), y (T, O): the shapes do not fit");
    return NULL;
  }
  if (out.n != y.n || out.shape[0] != T || out.shape[1] != O || out.dtype != y.dtype || out.dev != y.dev) {
    PyErr_SetString(PyExc_ValueError, "out must have y's ranks, shape, dtype and device");
    return NULL;
  }
  if (R > 1 << 20 || ld_of(&x, &ldx, "x") || ld_of(&y, &ldy, "y") || ld_of(&out, &ldo, "out")) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "the adapters' rank is too large");
    return NULL;
  }
  if (length_of(a[5], &size, &dev, "plan") || param_of(a[5], &plan, t_i32, size, x.dev, "plan") ||
      param_of(a[8], &scales, t_f32, n, x.dev, "scales") || stream_of(a[10], x.dev, &stream))
    return NULL;
  PyObject *keep = Py_NewRef(to), *mem = NULL;
  if (T > (R <= 64 ? 1024 : 512)) {  /* few_tokens() of serve.cuh */
    mem = PyObject_CallFunction(a[6], "LLlO", T, R, x.dev, a[10]);
    if (!mem || length_of(mem, &floats, &dev, "workspace") || param_of(mem, &room, t_f32, floats, x.dev, "workspace")) {
      Py_XDECREF(mem);
      Py_DECREF(keep);
      return NULL;
    }
  }
  if (!fn) {  // whoever made the memory keeps it
    Py_XDECREF(mem);
    if (column)
      return Py_BuildValue("N(iKLLLKNLiLKKLKiNLNLiK)", keep, y.n, x.ptr[0], T, K, ldx, A_.ptr[0], bytes_of(&B_), n, (int)R,
                           O * y.n, scales, plan, size, room, x.dt, bytes_of(&y), ldy, bytes_of(&out), ldo, y.dt, stream);
    return Py_BuildValue("N(iNLLLNKLiLKKLKiKLKLiK)", keep, x.n, bytes_of(&x), T, K * x.n, ldx, bytes_of(&A_), B_.ptr[0], n,
                         (int)R, O, scales, plan, size, room, x.dt, y.ptr[0], ldy, out.ptr[0], ldo, y.dt, stream);
  }
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  if (column)
    rc = ((__typeof__(&tp_lora_all_to_sharded))fn)(y.n, P(x.ptr[0]), T, K, ldx, P(A_.ptr[0]), CA(B_), n, (int)R, O * y.n,
                                                   P(scales), P(plan), size, P(room), (tp_dtype)x.dt, CA(y), ldy, A(out), ldo,
                                                   (tp_dtype)y.dt, P(stream));
  else
    rc = ((__typeof__(&tp_lora_sharded_to_all))fn)(x.n, CA(x), T, K * x.n, ldx, CA(A_), P(B_.ptr[0]), n, (int)R, O,
                                                   P(scales), P(plan), size, P(room), (tp_dtype)x.dt, P(y.ptr[0]), ldy,
                                                   P(out.ptr[0]), ldo, (tp_dtype)y.dt, P(stream));
  Py_END_ALLOW_THREADS;
  Py_XDECREF(mem);
  return answer(keep, rc);
}

/* verify(fn, logits, drafts, cu_rows, u, draft_probs, temperature, top_k, top_p, min_p, tokens, logprobs, accepted,
 * rejected, stream) -> (tokens, logprobs, accepted, rejected) */
static PyObject *m_verify(PyObject *self, PyObject *const *a, Py_ssize_t na) {
  if (na != 15) return PyErr_Format(PyExc_TypeError, "verify takes 15 arguments");
  void *fn = PyLong_AsVoidPtr(a[0]);
  Info f, q;
  long dev;
  int64_t seqs, ldq = 0;
  uint64_t drafts, cu, u, t, k, p, m, stream, to[4];
  if (info_of(a[1], &f, "logits")) return NULL;
  const int dt = dtype_code(f.dtype);
  if (dt < 0) return PyErr_Format(PyExc_TypeError, "logits: unsupported dtype %S", f.dtype);
  if (f.nd != 2 || (f.shape[1] > 1 && f.stride[1] != 1))
    return PyErr_Format(PyExc_ValueError, "logits must be 2-D with unit column stride");
  const int64_t T = f.shape[0], V = f.shape[1], ld = T > 1 ? f.stride[0] : V;
  int q_dt = TP_F32;
  q.ptr = 0;
  if (a[5] != Py_None) {
    if (info_of(a[5], &q, "draft_probs")) return NULL;
    q_dt = dtype_code(q.dtype);
    if (q_dt < 0) return PyErr_Format(PyExc_TypeError, "draft_probs: unsupported dtype %S", q.dtype);
    if (q.nd != 2 || q.dev != f.dev || q.shape[0] != T || q.shape[1] != V || (V > 1 && q.stride[1] != 1))
      return PyErr_Format(PyExc_ValueError, "draft_probs must have logits' shape and device and unit column stride");
    ldq = T > 1 ? q.stride[0] : V;
  }
  if (length_of(a[3], &seqs, &dev, "cu_rows")) return NULL;
  if (--seqs < 0) return PyErr_Format(PyExc_ValueError, "cu_rows needs one value more than there are sequences");
  if (param_of(a[3], &cu, t_i32, seqs + 1, f.dev, "cu_rows") || param_of(a[2], &drafts, t_i64, T, f.dev, "drafts") ||
      param_of(a[4], &u, t_f32, T, f.dev, "u") || param_of(a[6], &t, t_f32, seqs, f.dev, "temperature") ||
      param_of(a[7], &k, t_i32, seqs, f.dev, "top_k") || param_of(a[8], &p, t_f32, seqs, f.dev, "top_p") ||
      param_of(a[9], &m, t_f32, seqs, f.dev, "min_p") || stream_of(a[14], f.dev, &stream))
    return NULL;
  static const char *const names[4] = {"tokens", "logprobs", "accepted", "rejected"};
  PyObject *const types[4] = {t_i64, t_f32, t_i32, t_i32};
  PyObject *out = PyTuple_New(4);
  if (!out) return NULL;
  for (int i = 0; i < 4; ++i) {
    const int64_t n = i < 2 ? T : seqs;
    PyObject *v = vector_or_new(a[10 + i], n, types[i], f.dev);
    if (!v) goto fail;
    PyTuple_SET_ITEM(out, i, v);
    if (param_of(v, &to[i], types[i], n, f.dev, names[i])) goto fail;
  }
  if (!fn)
    return Py_BuildValue("N(KLLLiKKLiLKKKKKKKKKKK)", out, f.ptr, T, V, ld, dt, drafts, q.ptr, ldq, q_dt, seqs, cu, u, t, k,
                         p, m, to[0], to[1], to[2], to[3], stream);
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = ((__typeof__(&tp_verify))fn)(P(f.ptr), T, V, ld, (tp_dtype)dt, P(drafts), P(q.ptr), ldq, (tp_dtype)q_dt, seqs,
                                    P(cu), P(u), P(t), P(k), P(p), P(m), P(to[0]), P(to[1]), P(to[2]), P(to[3]),
                                    P(stream));
  Py_END_ALLOW_THREADS;
  return answer(out, rc);
fail:
  Py_DECREF(out);
  return NULL;
}

/* init(float32, bfloat16, float16, int32, int64, current raw stream of a device index, torch.empty) */
static PyObject *m_init(PyObject *self, PyObject *args) {
  PyObject **to[7] = {&t_f32, &t_bf16, &t_f16, &t_i32, &t_i64, &raw_stream, &torch_empty}, *v[7];
  if (!PyArg_ParseTuple(args, "OOOOOOO", &v[0], &v[1], &v[2], &v[3], &v[4], &v[5], &v[6])) return NULL;
  for (int i = 0; i < 7; ++i) Py_XSETREF(*to[i], Py_NewRef(v[i]));
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {{"init", m_init, METH_VARARGS, NULL},
                                {"append", (PyCFunction)(void (*)(void))m_append, METH_FASTCALL, NULL},
                                {"decode", (PyCFunction)(void (*)(void))m_decode, METH_FASTCALL, NULL},
                                {"prefill", (PyCFunction)(void (*)(void))m_prefill, METH_FASTCALL, NULL},
                                {"sample", (PyCFunction)(void (*)(void))m_sample, METH_FASTCALL, NULL},
                                {"plan", (PyCFunction)(void (*)(void))m_plan, METH_FASTCALL, NULL},
                                {"groups", (PyCFunction)(void (*)(void))m_groups, METH_FASTCALL, NULL},
                                {"lora", (PyCFunction)(void (*)(void))m_lora, METH_FASTCALL, NULL},
                                {"verify", (PyCFunction)(void (*)(void))m_verify, METH_FASTCALL, NULL},
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__marshal(void) {
  struct {
    PyObject **to;
    const char *text;
  } names[] = {{&s_shape, "shape"},         {&s_stride, "stride"},     {&s_dtype, "dtype"},
               {&s_get_device, "get_device"}, {&s_data_ptr, "data_ptr"}, {&s_cuda_stream, "cuda_stream"}};
  for (unsigned i = 0; i < sizeof(names) / sizeof(names[0]); ++i) {
    *names[i].to = PyUnicode_InternFromString(names[i].text);
    if (!*names[i].to) return NULL;
  }
  empty_names = Py_BuildValue("(ss)", "dtype", "device");
  return empty_names ? PyModule_Create(&module) : NULL;
}
