// The short way from torch tensors to the calls whose GPU time is a few
// microseconds: a Python extension that checks and passes the arguments of
// pa_norm_rope_and_cache, pa_verify_tree, pa_decode_accumulate,
// pa_evict_select and pa_compact_kv and allocates their outputs and scratch.
//
// It takes regular calls only: plain tensors on the current device, of the
// documented types and shapes, on the current stream.  For anything else a
// function returns None with nothing done, and the caller goes the long way,
// which marshals the rare forms and words the refusals (ops.py); so what is
// accepted here must be accepted there, and the reverse is not needed.  A
// status of the C call other than PA_OK is returned as an int.
//
// Host time of a call (us, Grace host; the long way through ctypes and this
// one): norm_rope_and_cache 22.4 and 5.4, verify_tree with scratch and two
// launches 26.9 and 8.7, decode_accumulate 27.9 and 8.9, evict_select 20.4 and
// 5.9, compact_kv 9.9 and 3.0.  Of a short one the launch is 2 to 3 us and an
// allocation one.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>

#include "pa.h"

namespace {

// Addresses of the loaded libpa.so's functions (bind).
struct {
  decltype(&pa_norm_rope_and_cache) norm_rope;
  decltype(&pa_verify_tree_workspace_size) tree_workspace;
  decltype(&pa_verify_tree) verify_tree;
  decltype(&pa_decode_accumulate_workspace_size) accumulate_workspace;
  decltype(&pa_decode_accumulate) accumulate;
  decltype(&pa_evict_select) evict_select;
  decltype(&pa_compact_kv) compact;
} pa;

// One call's arguments: every function returns a value that may only be used
// while `ok`.
struct Call {
  bool ok = true;
  int64_t dev = -1;

  bool need(bool c) { return ok = ok && c; }

  const at::Tensor* tensor(PyObject* o) {
    if (!need(THPVariable_CheckExact(o))) return nullptr;
    const at::Tensor* t = &THPVariable_Unpack(o);
    return need(t->defined() && t->layout() == at::kStrided) ? t : nullptr;
  }
  // the tensor that names the device
  const at::Tensor* first(PyObject* o) {
    const at::Tensor* t = tensor(o);
    if (ok && need(t->is_cuda())) need((dev = t->get_device()) == c10::cuda::current_device());
    return t;
  }
  int size(const at::Tensor* t, int d) {
    if (!ok) return 0;
    const int64_t n = t->size(d);
    need(n <= INT_MAX);
    return (int)n;
  }
  void* here(const at::Tensor* t) {  // on the device, heads or elements apart as they may be
    return ok && need(t->is_cuda() && t->get_device() == dev) ? t->data_ptr() : nullptr;
  }
  void* ptr(const at::Tensor* t) { return ok && need(t->is_contiguous()) ? here(t) : nullptr; }
  void* ptr(PyObject* o, at::ScalarType type) {
    const at::Tensor* t = tensor(o);
    return ok && need(t->scalar_type() == type) ? ptr(t) : nullptr;
  }
  const int32_t* rows(PyObject* o, int n) {  // an int32 index tensor of n leading entries
    const at::Tensor* t = tensor(o);
    return ok && need(t->scalar_type() == at::kInt && t->dim() >= 1 && t->size(0) == n)
               ? static_cast<const int32_t*>(ptr(t))
               : nullptr;
  }
  const int32_t* rows_or_none(PyObject* o, int n) { return o == Py_None ? nullptr : rows(o, n); }
  int integer(PyObject* o) {
    if (!need(PyLong_CheckExact(o))) return 0;
    int over = 0;
    const long v = PyLong_AsLongAndOverflow(o, &over);
    need(!over && v >= INT_MIN && v <= INT_MAX);
    return (int)v;
  }
  float real(PyObject* o) {  // as the long way takes it: through a C double
    return need(PyFloat_Check(o)) ? (float)PyFloat_AS_DOUBLE(o) : 0.f;
  }
};

struct Caches {
  void *k = nullptr, *v = nullptr;
  int nb = 0, bs = 0, hkv = 0, d = 0;
  at::ScalarType type = at::kBFloat16;
  pa_dtype dtype = PA_BF16;
};

// two caches of one shape and type; `names_device`: the key cache does
Caches caches(Call& c, PyObject* ko, PyObject* vo, bool names_device) {
  Caches r;
  const at::Tensor* k = names_device ? c.first(ko) : c.tensor(ko);
  const at::Tensor* v = c.tensor(vo);
  if (!c.ok || !c.need(k->dim() == 4 && v->sizes() == k->sizes() && v->scalar_type() == k->scalar_type())) return r;
  r.type = k->scalar_type();
  c.need(r.type == at::kBFloat16 || r.type == at::kHalf);
  r.dtype = r.type == at::kHalf ? PA_FP16 : PA_BF16;
  r.nb = c.size(k, 0), r.bs = c.size(k, 1), r.hkv = c.size(k, 2), r.d = c.size(k, 3);
  r.k = c.ptr(k), r.v = c.ptr(v);
  return r;
}

struct Scores {
  float* p = nullptr;
  const int32_t* rows = nullptr;
  int num_rows = 0, length = 0;
};

// fp32 [rows][hkv][length], and the requests' rows
Scores scores(Call& c, const at::Tensor* t, int hkv, PyObject* rows, int num_seqs) {
  Scores s;
  if (!c.ok || !c.need(t->dim() == 3 && t->size(1) == hkv && t->scalar_type() == at::kFloat)) return s;
  s.num_rows = c.size(t, 0), s.length = c.size(t, 2);
  s.p = static_cast<float*>(c.ptr(t));
  if (rows != Py_None) s.rows = c.rows(rows, num_seqs);
  else c.need(s.num_rows >= num_seqs);
  return s;
}

pa_stream current_stream(int64_t dev) {
  return reinterpret_cast<pa_stream>(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
}

// Runs `f` (allocations and the C call) without the interpreter's lock; false
// if an allocation failed (the long way then raises what it raises).
template <typename F>
bool run(F&& f) {
  PyThreadState* s = PyEval_SaveThread();
  bool done = true;
  try {
    f();
  } catch (...) {
    done = false;
  }
  PyEval_RestoreThread(s);
  return done;
}

// A result's object; nullptr with an error set.  (The work is under way by
// then: no going the long way any more.)
PyObject* give(const at::Tensor& t) {
  try {
    return THPVariable_Wrap(t);
  } catch (...) {
    if (!PyErr_Occurred()) PyErr_NoMemory();
    return nullptr;
  }
}

// (q, k, v, positions, cos_sin, slot_mapping, k_cache, v_cache, q_weight, k_weight, eps, sections, interleaved, out)
PyObject* norm_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 14) Py_RETURN_NONE;
  Call c;
  const Caches kv = caches(c, a[6], a[7], true);
  const at::Tensor *q = c.tensor(a[0]), *k = c.tensor(a[1]), *v = c.tensor(a[2]);
  if (!c.ok || !c.need(q->dim() == 3 && k->dim() == 3 && v->dim() == 3 && q->size(2) == kv.d)) Py_RETURN_NONE;
  const int T = c.size(q, 0), hq = c.size(q, 1);
  auto stride = [&](const at::Tensor* t, int heads) -> int64_t {  // of the tokens, whose heads are contiguous
    const int64_t row = (int64_t)heads * kv.d;
    if (!c.need(t->scalar_type() == kv.type && t->size(0) == T && t->size(1) == heads && t->size(2) == kv.d)) return 0;
    int64_t s = row;
    if (!t->is_contiguous()) {
      c.need(t->stride(2) == 1 && (heads <= 1 || t->stride(1) == kv.d));
      if (T > 1) s = t->stride(0);
    }
    c.need(s >= row && s % 8 == 0);
    return s;
  };
  const int64_t qs = stride(q, hq), ks = stride(k, kv.hkv), vs = stride(v, kv.hkv);
  const at::Tensor *pos = c.tensor(a[3]), *table = c.tensor(a[4]);
  if (!c.ok || !c.need(pos->scalar_type() == at::kInt && (pos->dim() == 1 || pos->dim() == 2) &&
                       pos->size(pos->dim() - 1) == T && table->dim() == 2 && table->scalar_type() == at::kFloat))
    Py_RETURN_NONE;
  const int axes = pos->dim() == 1 ? 1 : c.size(pos, 0), max_pos = c.size(table, 0), rot = c.size(table, 1);
  c.need(axes >= 1 && axes <= 3);
  int32_t sec[3] = {0, 0, 0};
  if (a[11] == Py_None) {
    c.need(axes == 1);
  } else if (c.ok && c.need((PyTuple_CheckExact(a[11]) || PyList_CheckExact(a[11])) &&
                            PySequence_Fast_GET_SIZE(a[11]) == axes)) {
    int64_t sum = 0;
    for (int i = 0; i < axes; ++i) {
      sec[i] = c.integer(PySequence_Fast_GET_ITEM(a[11], i));
      c.need(sec[i] >= 0);
      sum += sec[i];
    }
    c.need(sum == rot / 2);
  }
  auto weight = [&](PyObject* o) -> const void* {
    if (o == Py_None) return nullptr;
    const at::Tensor* w = c.tensor(o);
    return c.ok && c.need(w->dim() == 1 && w->size(0) == kv.d && w->scalar_type() == kv.type) ? c.ptr(w) : nullptr;
  };
  const void *qw = weight(a[8]), *kw = weight(a[9]);
  const float eps = c.real(a[10]);
  c.need(PyBool_Check(a[12]));
  const int32_t* slots = c.rows(a[5], T);
  const void *qp = c.here(q), *kp = c.here(k), *vp = c.here(v), *pp = c.ptr(pos), *tp = c.ptr(table);
  at::Tensor out;
  if (a[13] != Py_None) {
    const at::Tensor* t = c.tensor(a[13]);
    if (c.ok && c.need(t->sizes() == q->sizes() && t->scalar_type() == kv.type) && c.ptr(t), c.ok) out = *t;
  }
  if (!c.ok) Py_RETURN_NONE;
  const bool mine = !out.defined();
  int st = PA_OK;
  if (!run([&] {
        if (mine) out = at::empty(q->sizes(), q->options());
        st = pa.norm_rope(qp, kp, vp, qs, ks, vs, qw, kw, eps, static_cast<const int32_t*>(pp), axes,
                          a[11] == Py_None ? nullptr : sec, static_cast<const float*>(tp), max_pos, rot,
                          a[12] == Py_True, slots, T, hq, out.data_ptr(), kv.k, kv.v, kv.nb, kv.bs, kv.hkv, kv.d,
                          kv.dtype, current_stream(c.dev));
      }))
    Py_RETURN_NONE;
  if (st != PA_OK) return PyLong_FromLong(st);
  return mine ? give(out) : Py_NewRef(a[13]);
}

// (q, q_start, tree_mask, context_lens, k_cache, v_cache, block_tables, scale, max_q_len, out, split_tokens)
PyObject* verify_tree(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 11) Py_RETURN_NONE;
  Call c;
  const at::Tensor* q = c.first(a[0]);
  const Caches kv = caches(c, a[4], a[5], false);
  const at::Tensor *lens = c.tensor(a[3]), *table = c.tensor(a[6]), *mask = c.tensor(a[2]);
  if (!c.ok || !c.need(q->dim() == 3 && q->size(2) == kv.d && q->scalar_type() == kv.type && lens->dim() >= 1 &&
                       table->dim() == 2 && mask->dim() >= 1 && mask->size(0) == q->size(0)))
    Py_RETURN_NONE;
  const int T = c.size(q, 0), hq = c.size(q, 1), R = c.size(lens, 0), maxblk = c.size(table, 1);
  c.need(R < INT_MAX);
  const int32_t *lp = c.rows(a[3], R), *sp = c.rows(a[1], c.ok ? R + 1 : 0), *tp = c.rows(a[6], R);
  const void *mp = c.ptr(a[2], at::kLong), *qp = c.ptr(q);
  const float scale = c.real(a[7]);
  const int max_q = c.integer(a[8]), split = c.integer(a[10]);
  at::Tensor out, ws;
  if (a[9] != Py_None) {
    const at::Tensor* t = c.tensor(a[9]);
    if (c.ok && c.need(t->sizes() == q->sizes() && t->scalar_type() == kv.type) && c.ptr(t), c.ok) out = *t;
  }
  if (!c.ok) Py_RETURN_NONE;
  const bool mine = !out.defined();
  int st = PA_OK;
  if (!run([&] {
        if (mine) out = at::empty(q->sizes(), q->options());
        const size_t bytes = pa.tree_workspace(R, T, max_q, hq, kv.hkv, kv.d, maxblk, kv.bs, split);
        if (bytes) ws = at::empty({(int64_t)bytes}, q->options().dtype(at::kByte));
        st = pa.verify_tree(qp, sp, static_cast<const uint64_t*>(mp), lp, kv.k, kv.v, tp, maxblk, R, T, max_q, hq,
                            kv.hkv, kv.d, kv.bs, kv.nb, scale, split, bytes ? ws.data_ptr() : nullptr, bytes,
                            out.data_ptr(), kv.dtype, current_stream(c.dev));
      }))
    Py_RETURN_NONE;
  if (st != PA_OK) return PyLong_FromLong(st);
  return mine ? give(out) : Py_NewRef(a[9]);
}

// (q, k_cache, v_cache, block_tables, context_lens, scale, scores, score_rows, scores_out, out, split_tokens)
PyObject* decode_accumulate(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 11) Py_RETURN_NONE;
  Call c;
  const at::Tensor* q = c.first(a[0]);
  const Caches kv = caches(c, a[1], a[2], false);
  const at::Tensor *table = c.tensor(a[3]), *st0 = c.tensor(a[6]);
  if (!c.ok || !c.need(q->dim() == 3 && q->size(2) == kv.d && q->scalar_type() == kv.type && table->dim() == 2))
    Py_RETURN_NONE;
  const int B = c.size(q, 0), hq = c.size(q, 1), maxblk = c.size(table, 1);
  const int32_t *tp = c.rows(a[3], B), *lp = c.rows(a[4], B);
  const void* qp = c.ptr(q);
  const Scores s = scores(c, st0, kv.hkv, a[7], B);
  float* so = s.p;
  PyObject* sout = a[6];
  if (a[8] != Py_None) {
    const at::Tensor* t = c.tensor(a[8]);
    if (c.ok && c.need(t->sizes() == st0->sizes() && t->scalar_type() == at::kFloat))
      so = static_cast<float*>(c.ptr(t));
    sout = a[8];
  }
  const float scale = c.real(a[5]);
  const int split = c.integer(a[10]);
  at::Tensor out, ws;
  if (a[9] != Py_None) {
    const at::Tensor* t = c.tensor(a[9]);
    if (c.ok && c.need(t->sizes() == q->sizes() && t->scalar_type() == kv.type) && c.ptr(t), c.ok) out = *t;
  }
  if (!c.ok) Py_RETURN_NONE;
  const bool mine = !out.defined();
  int st = PA_OK;
  if (!run([&] {
        if (mine) out = at::empty(q->sizes(), q->options());
        const size_t bytes = pa.accumulate_workspace(B, hq, kv.hkv, kv.d, maxblk, kv.bs, split);
        ws = at::empty({(int64_t)(bytes ? bytes : 1)}, q->options().dtype(at::kByte));
        st = pa.accumulate(qp, kv.k, kv.v, tp, maxblk, lp, B, hq, kv.hkv, kv.d, kv.bs, kv.nb, scale, split, s.p, s.rows,
                           s.num_rows, s.length, so, ws.data_ptr(), bytes ? bytes : 1, out.data_ptr(), kv.dtype,
                           current_stream(c.dev));
      }))
    Py_RETURN_NONE;
  if (st != PA_OK) return PyLong_FromLong(st);
  PyObject* o = mine ? give(out) : Py_NewRef(a[9]);
  if (!o) return nullptr;
  PyObject* r = PyTuple_Pack(2, o, sout);
  Py_DECREF(o);
  return r;
}

// (scores, context_lens, sink, heavy, recent, score_rows)
PyObject* evict_select(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6) Py_RETURN_NONE;
  Call c;
  const at::Tensor *t = c.first(a[0]), *lens = c.tensor(a[1]);
  if (!c.ok || !c.need(t->dim() == 3 && lens->dim() >= 1)) Py_RETURN_NONE;
  const int hkv = c.size(t, 1), B = c.size(lens, 0);
  const int32_t* lp = c.rows(a[1], B);
  const Scores s = scores(c, t, hkv, a[5], B);
  const int sink = c.integer(a[2]), heavy = c.integer(a[3]), recent = c.integer(a[4]);
  const int64_t budget = (int64_t)sink + heavy + recent;
  if (!c.need(sink >= 0 && heavy >= 0 && recent >= 0 && budget >= 1 && budget <= INT_MAX)) Py_RETURN_NONE;
  at::Tensor keep, keep_lens;
  int st = PA_OK;
  if (!run([&] {
        const auto opt = t->options().dtype(at::kInt);
        keep = at::empty({B, hkv, budget}, opt);
        keep_lens = at::empty({B}, opt);
        st = pa.evict_select(s.p, s.rows, s.num_rows, hkv, s.length, lp, B, sink, heavy, recent,
                             static_cast<int32_t*>(keep.data_ptr()), static_cast<int32_t*>(keep_lens.data_ptr()),
                             current_stream(c.dev));
      }))
    Py_RETURN_NONE;
  if (st != PA_OK) return PyLong_FromLong(st);
  PyObject *k = give(keep), *l = k ? give(keep_lens) : nullptr;
  PyObject* r = k && l ? PyTuple_Pack(2, k, l) : nullptr;
  Py_XDECREF(k);
  Py_XDECREF(l);
  return r;
}

// (k_cache, v_cache, block_tables, context_lens, keep, keep_lens, base, scores, score_rows) -> PA_OK's 0, a status
PyObject* compact_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 9) Py_RETURN_NONE;
  Call c;
  const Caches kv = caches(c, a[0], a[1], true);
  const at::Tensor *table = c.tensor(a[2]), *lens = c.tensor(a[3]), *keep = c.tensor(a[4]);
  if (!c.ok || !c.need(table->dim() == 2 && lens->dim() >= 1 && keep->dim() == 3 && keep->size(2) > 0)) Py_RETURN_NONE;
  const int B = c.size(lens, 0), maxblk = c.size(table, 1), heads = c.size(keep, 1), most = c.size(keep, 2);
  c.need(heads == 1 || heads == kv.hkv);
  const int32_t *tp = c.rows(a[2], B), *lp = c.rows(a[3], B), *kp = c.rows(a[4], B), *np = c.rows(a[5], B);
  const int32_t* bp = c.rows_or_none(a[6], B);
  Scores s;
  if (a[7] != Py_None) s = scores(c, c.tensor(a[7]), kv.hkv, a[8], B);
  if (!c.ok) Py_RETURN_NONE;
  int st = PA_OK;
  if (!run([&] {
        st = pa.compact(kv.k, kv.v, tp, maxblk, lp, kp, heads, most, np, bp, B, kv.nb, kv.bs, kv.hkv, kv.d, kv.dtype,
                        s.p, s.rows, s.num_rows, s.length, current_stream(c.dev));
      }))
    Py_RETURN_NONE;
  return PyLong_FromLong(st);
}

// (addresses in the order of `pa`)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  constexpr int N = sizeof(pa) / sizeof(void*);
  void* f[N];
  if (n != N) {
    PyErr_SetString(PyExc_TypeError, "bind takes one address per function");
    return nullptr;
  }
  for (int i = 0; i < N; ++i)
    if (!(f[i] = PyLong_AsVoidPtr(a[i]))) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  pa.norm_rope = reinterpret_cast<decltype(pa.norm_rope)>(f[0]);
  pa.tree_workspace = reinterpret_cast<decltype(pa.tree_workspace)>(f[1]);
  pa.verify_tree = reinterpret_cast<decltype(pa.verify_tree)>(f[2]);
  pa.accumulate_workspace = reinterpret_cast<decltype(pa.accumulate_workspace)>(f[3]);
  pa.accumulate = reinterpret_cast<decltype(pa.accumulate)>(f[4]);
  pa.evict_select = reinterpret_cast<decltype(pa.evict_select)>(f[5]);
  pa.compact = reinterpret_cast<decltype(pa.compact)>(f[6]);
  Py_RETURN_NONE;
}

// What a tensor's own checks throw (one without storage, a wrapper) is the long
// way's to refuse; nothing has been launched by then.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(self, a, n);
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

#define PA_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {PA_METHOD(bind),
                         PA_METHOD(norm_rope),
                         PA_METHOD(verify_tree),
                         PA_METHOD(decode_accumulate),
                         PA_METHOD(evict_select),
                         PA_METHOD(compact_kv),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the torch whose headers, and so whose tensors' layout, this was
// compiled with; it is used with that one alone (ops.py).
PyMODINIT_FUNC PyInit__marshal() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", PA_TORCH_VERSION) != 0) Py_CLEAR(m);
  return m;
}
