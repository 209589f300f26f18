// The short way from torch tensors to the calls whose GPU time is a few
// microseconds: a Python extension that checks and passes the arguments of
// pa_norm_rope_and_cache, pa_verify_tree, pa_decode_accumulate,
// pa_evict_select, pa_compact_kv, the calls of the 4-bit cache, pa_fork_blocks
// and pa_copy_pages and allocates their outputs and scratch.
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
// 5.9, compact_kv 9.9 and 3.0; this one alone: quantize_and_cache 2.6,
// dequantize_kv4 4.9, decode_kv4 4.6, fork_blocks 7, copy_pages 2.5.  Of a short
// one the launch is 2 to 3 us and an allocation one.
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
  decltype(&pa_quantize_and_cache) quantize;
  decltype(&pa_dequantize_kv4) dequantize;
  decltype(&pa_decode_kv4_workspace_size) decode4_workspace;
  decltype(&pa_decode_kv4) decode4;
  decltype(&pa_chunked_prefill_kv4_workspace_size) prefill4_workspace;
  decltype(&pa_chunked_prefill_kv4) prefill4;
  decltype(&pa_fork_blocks_workspace_size) fork_workspace;
  decltype(&pa_fork_blocks) fork;
  decltype(&pa_copy_pages) copy_pages;
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

// of the tokens of [T][heads][d], whose heads are contiguous
int64_t token_stride(Call& c, const at::Tensor* t, int T, int heads, int d, at::ScalarType type) {
  const int64_t row = (int64_t)heads * d;
  if (!c.need(t->scalar_type() == type && t->dim() == 3 && t->size(0) == T && t->size(1) == heads && t->size(2) == d))
    return 0;
  int64_t s = row;
  if (!t->is_contiguous()) {
    c.need(t->stride(2) == 1 && (heads <= 1 || t->stride(1) == d));
    if (T > 1) s = t->stride(0);
  }
  c.need(s >= row && s % 8 == 0);
  return s;
}

// two 4-bit caches of one shape, for heads of d elements
Caches kv4_caches(Call& c, PyObject* ko, PyObject* vo, int64_t d, bool names_device) {
  Caches r;
  const at::Tensor* k = names_device ? c.first(ko) : c.tensor(ko);
  const at::Tensor* v = c.tensor(vo);
  if (!c.ok || !c.need((d == 64 || d == 128) && k->dim() == 3 && v->sizes() == k->sizes() &&
                       k->scalar_type() == at::kByte && v->scalar_type() == at::kByte))
    return r;
  const int64_t bs = k->size(2) * 16 / (9 * d);
  c.need(bs * 9 * d == k->size(2) * 16 && (bs == 4 || bs == 8 || bs == 16 || bs == 32));
  r.nb = c.size(k, 0), r.bs = (int)bs, r.hkv = c.size(k, 1), r.d = (int)d;
  r.k = c.ptr(k), r.v = c.ptr(v);
  return r;
}

// the type of q and of what comes with it
pa_dtype half_type(Call& c, const at::Tensor* t) {
  if (!c.ok) return PA_BF16;
  c.need(t->scalar_type() == at::kBFloat16 || t->scalar_type() == at::kHalf);
  return t->scalar_type() == at::kHalf ? PA_FP16 : PA_BF16;
}

// `o` as the output of q's shape and type, or none
at::Tensor given(Call& c, PyObject* o, const at::Tensor* q) {
  if (o == Py_None) return {};
  const at::Tensor* t = c.tensor(o);
  if (c.ok && c.need(t->sizes() == q->sizes() && t->scalar_type() == q->scalar_type()) && c.ptr(t), c.ok) return *t;
  return {};
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

// A contiguous tensor of `all`'s memory, from its element `at` on: small outputs
// share one allocation, since at::empty is 1.2 of the microseconds that a call takes.
at::Tensor piece(const at::Tensor& all, int64_t at, c10::IntArrayRef shape) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
  t.unsafeGetTensorImpl()->set_storage_offset(at);
  t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return t;
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
  auto stride = [&](const at::Tensor* t, int heads) { return token_stride(c, t, T, heads, kv.d, kv.type); };
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

// (k, v, slot_mapping, k_cache, v_cache) -> PA_OK's 0, a status
PyObject* quantize_and_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) Py_RETURN_NONE;
  Call c;
  const at::Tensor *k = c.first(a[0]), *v = c.tensor(a[1]);
  if (!c.ok || !c.need(k->dim() == 3)) Py_RETURN_NONE;
  const pa_dtype dtype = half_type(c, k);
  const int T = c.size(k, 0);
  const Caches kv = kv4_caches(c, a[3], a[4], k->size(2), false);
  if (!c.ok) Py_RETURN_NONE;
  const int64_t ks = token_stride(c, k, T, kv.hkv, kv.d, k->scalar_type());
  const int64_t vs = token_stride(c, v, T, kv.hkv, kv.d, k->scalar_type());
  const int32_t* slots = c.rows(a[2], T);
  const void *kp = c.here(k), *vp = c.here(v);
  if (!c.ok) Py_RETURN_NONE;
  int st = PA_OK;
  if (!run([&] {
        st = pa.quantize(kp, vp, ks, vs, slots, T, kv.k, kv.v, kv.nb, kv.bs, kv.hkv, kv.d, dtype, current_stream(c.dev));
      }))
    Py_RETURN_NONE;
  return PyLong_FromLong(st);
}

// (k_cache, v_cache, slots, head_dim, pa_dtype)
PyObject* dequantize_kv4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) Py_RETURN_NONE;
  Call c;
  const int d = c.integer(a[3]), dtype = c.integer(a[4]);
  const Caches kv = kv4_caches(c, a[0], a[1], d, true);
  const at::Tensor* slots = c.tensor(a[2]);
  if (!c.ok || !c.need(slots->dim() == 1 && (dtype == PA_FP16 || dtype == PA_BF16))) Py_RETURN_NONE;
  const int T = c.size(slots, 0);
  const int32_t* sp = c.rows(a[2], T);
  if (!c.ok) Py_RETURN_NONE;
  at::Tensor k, v;
  int st = PA_OK;
  if (!run([&] {
        const auto opt = slots->options().dtype(dtype == PA_FP16 ? at::kHalf : at::kBFloat16);
        const int64_t n = (int64_t)T * kv.hkv * d;  // a multiple of 64
        if (n <= (1 << 18)) {
          const at::Tensor all = at::empty({2 * n}, opt);
          k = piece(all, 0, {T, kv.hkv, d});
          v = piece(all, n, {T, kv.hkv, d});
        } else {  // so large that one may be let go before the other
          k = at::empty({T, kv.hkv, d}, opt);
          v = at::empty({T, kv.hkv, d}, opt);
        }
        st = pa.dequantize(kv.k, kv.v, sp, T, kv.nb, kv.bs, kv.hkv, d, k.data_ptr(), v.data_ptr(), (pa_dtype)dtype,
                           current_stream(c.dev));
      }))
    Py_RETURN_NONE;
  if (st != PA_OK) return PyLong_FromLong(st);
  PyObject *ko = give(k), *vo = ko ? give(v) : nullptr;
  PyObject* r = ko && vo ? PyTuple_Pack(2, ko, vo) : nullptr;
  Py_XDECREF(ko);
  Py_XDECREF(vo);
  return r;
}

// (q, k_cache, v_cache, block_tables, context_lens, scale, out, split_tokens)
PyObject* decode_kv4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8) Py_RETURN_NONE;
  Call c;
  const at::Tensor *q = c.first(a[0]), *table = c.tensor(a[3]);
  if (!c.ok || !c.need((q->dim() == 3 || q->dim() == 4) && table->dim() == 2)) Py_RETURN_NONE;
  const pa_dtype dtype = half_type(c, q);
  const int last = (int)q->dim() - 1;
  const Caches kv = kv4_caches(c, a[1], a[2], q->size(last), false);
  const int B = c.size(q, 0), ql = last == 2 ? 1 : c.size(q, 1), hq = c.size(q, last - 1), maxblk = c.size(table, 1);
  const int32_t *tp = c.rows(a[3], B), *lp = c.rows(a[4], B);
  const void* qp = c.ptr(q);
  const float scale = c.real(a[5]);
  const int split = c.integer(a[7]);
  at::Tensor out = given(c, a[6], q), ws;
  if (!c.ok) Py_RETURN_NONE;
  const bool mine = !out.defined();
  int st = PA_OK;
  if (!run([&] {
        if (mine) out = at::empty(q->sizes(), q->options());
        const size_t bytes = pa.decode4_workspace(B, ql, hq, kv.hkv, kv.d, maxblk, kv.bs, split);
        if (bytes) ws = at::empty({(int64_t)bytes}, q->options().dtype(at::kByte));
        st = pa.decode4(qp, kv.k, kv.v, tp, maxblk, lp, B, ql, hq, kv.hkv, kv.d, kv.bs, kv.nb, scale, split,
                        bytes ? ws.data_ptr() : nullptr, bytes, out.data_ptr(), dtype, current_stream(c.dev));
      }))
    Py_RETURN_NONE;
  if (st != PA_OK) return PyLong_FromLong(st);
  return mine ? give(out) : Py_NewRef(a[6]);
}

// (q, q_start, context_lens, k_cache, v_cache, block_tables, scale, max_q_len, out, split_tokens)
PyObject* chunked_prefill_kv4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 10) Py_RETURN_NONE;
  Call c;
  const at::Tensor *q = c.first(a[0]), *lens = c.tensor(a[2]), *table = c.tensor(a[5]);
  if (!c.ok || !c.need(q->dim() == 3 && lens->dim() >= 1 && table->dim() == 2)) Py_RETURN_NONE;
  const pa_dtype dtype = half_type(c, q);
  const Caches kv = kv4_caches(c, a[3], a[4], q->size(2), false);
  const int T = c.size(q, 0), hq = c.size(q, 1), R = c.size(lens, 0), maxblk = c.size(table, 1);
  c.need(R < INT_MAX);
  const int32_t *lp = c.rows(a[2], R), *sp = c.rows(a[1], c.ok ? R + 1 : 0), *tp = c.rows(a[5], R);
  const void* qp = c.ptr(q);
  const float scale = c.real(a[6]);
  const int max_q = c.integer(a[7]), split = c.integer(a[9]);
  at::Tensor out = given(c, a[8], q), ws;
  if (!c.ok) Py_RETURN_NONE;
  const bool mine = !out.defined();
  int st = PA_OK;
  if (!run([&] {
        if (mine) out = at::empty(q->sizes(), q->options());
        const size_t bytes = pa.prefill4_workspace(R, T, max_q, hq, kv.hkv, kv.d, maxblk, kv.bs, split);
        if (bytes) ws = at::empty({(int64_t)bytes}, q->options().dtype(at::kByte));
        st = pa.prefill4(qp, sp, lp, kv.k, kv.v, tp, maxblk, R, T, max_q, hq, kv.hkv, kv.d, kv.bs, kv.nb, scale, split,
                         bytes ? ws.data_ptr() : nullptr, bytes, out.data_ptr(), dtype, current_stream(c.dev));
      }))
    Py_RETURN_NONE;
  if (st != PA_OK) return PyLong_FromLong(st);
  return mine ? give(out) : Py_NewRef(a[8]);
}

// (block_tables, context_lens, parents, num_blocks, block_size, grow, max_grow, pinned, max_blocks): grow a tensor and
// max_grow its bound, or grow a count and max_grow None; pinned and max_blocks may be None
PyObject* fork_blocks(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 9) Py_RETURN_NONE;
  Call c;
  const at::Tensor *table = c.first(a[0]), *lens = c.tensor(a[1]), *parents = c.tensor(a[2]);
  if (!c.ok || !c.need(table->dim() == 2 && lens->dim() >= 1 && parents->dim() >= 1)) Py_RETURN_NONE;
  const int B = c.size(lens, 0), R = c.size(parents, 0), maxblk = c.size(table, 1);
  const int32_t *tp = c.rows(a[0], B), *lp = c.rows(a[1], B), *pp = c.rows(a[2], R), *gp = nullptr;
  const int num_blocks = c.integer(a[3]), bs = c.integer(a[4]);
  int most = 0;
  if (a[6] == Py_None) {
    most = c.integer(a[5]);
  } else {
    gp = c.rows(a[5], R);
    most = c.integer(a[6]);
  }
  const uint8_t* pin = nullptr;
  if (a[7] != Py_None) {
    const at::Tensor* t = c.tensor(a[7]);
    if (c.ok && c.need(t->dim() == 1 && t->size(0) == num_blocks &&
                       (t->scalar_type() == at::kBool || t->scalar_type() == at::kByte)))
      pin = static_cast<const uint8_t*>(c.ptr(t));
  }
  const int width = a[8] == Py_None ? maxblk : c.integer(a[8]);
  if (!c.ok || !c.need(most >= 0 && width >= 1)) Py_RETURN_NONE;
  at::Tensor out[5], ws;
  int st = PA_OK;
  if (!run([&] {
        const auto opt = table->options();
        const std::initializer_list<int64_t> shapes[5] = {{R, width}, {R}, {R, 2}, {R, most}, {1}};
        int64_t at[6] = {0};
        for (int i = 0; i < 5; ++i) {
          int64_t n = 1;
          for (const int64_t x : shapes[i]) n *= x;
          at[i + 1] = at[i] + (n + 63) / 64 * 64;
        }
        const at::Tensor all = at::empty({at[5]}, opt);
        int32_t* p[5];
        for (int i = 0; i < 5; ++i) {
          out[i] = piece(all, at[i], shapes[i]);
          p[i] = static_cast<int32_t*>(all.data_ptr()) + at[i];
        }
        const size_t bytes = pa.fork_workspace(R, num_blocks);
        ws = at::empty({(int64_t)bytes}, opt.dtype(at::kByte));
        st = pa.fork(tp, maxblk, lp, B, pp, R, gp, most, pin, num_blocks, bs, p[0], width, p[1], p[2], p[3], p[4],
                     ws.data_ptr(), bytes, current_stream(c.dev));
      }))
    Py_RETURN_NONE;
  if (st != PA_OK) return PyLong_FromLong(st);
  PyObject* r = PyTuple_New(5);
  for (int i = 0; r && i < 5; ++i) {
    PyObject* o = give(out[i]);
    if (o) PyTuple_SET_ITEM(r, i, o);
    else Py_CLEAR(r);
  }
  return r;
}

// (list of caches, pairs) -> PA_OK's 0, a status
PyObject* copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 2 || !PyList_CheckExact(a[0])) Py_RETURN_NONE;
  const Py_ssize_t num = PyList_GET_SIZE(a[0]);
  constexpr Py_ssize_t kMost = 512;  // longer lists go the long way
  if (num < 1 || num > kMost) Py_RETURN_NONE;
  Call c;
  void* p[kMost];
  int nb = 0;
  int64_t bytes = 0;
  for (Py_ssize_t i = 0; i < num; ++i) {
    const at::Tensor* t = i ? c.tensor(PyList_GET_ITEM(a[0], i)) : c.first(PyList_GET_ITEM(a[0], i));
    if (!c.ok || !c.need(t->dim() >= 1)) Py_RETURN_NONE;
    const int64_t size = t->numel() * t->element_size();
    if (i == 0) nb = c.size(t, 0), bytes = size;
    c.need(nb > 0 && t->size(0) == nb && size == bytes);
    p[i] = c.ptr(t);
  }
  const at::Tensor* pairs = c.tensor(a[1]);
  if (!c.ok || !c.need(bytes / nb % 16 == 0 && pairs->dim() == 2 && pairs->size(1) == 2)) Py_RETURN_NONE;
  const int np = c.size(pairs, 0);
  const int32_t* pp = c.rows(a[1], np);
  if (!c.ok) Py_RETURN_NONE;
  int st = PA_OK;
  if (!run([&] { st = pa.copy_pages(p, (int)num, pp, np, nb, bytes / nb, current_stream(c.dev)); })) Py_RETURN_NONE;
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
  pa.quantize = reinterpret_cast<decltype(pa.quantize)>(f[7]);
  pa.dequantize = reinterpret_cast<decltype(pa.dequantize)>(f[8]);
  pa.decode4_workspace = reinterpret_cast<decltype(pa.decode4_workspace)>(f[9]);
  pa.decode4 = reinterpret_cast<decltype(pa.decode4)>(f[10]);
  pa.prefill4_workspace = reinterpret_cast<decltype(pa.prefill4_workspace)>(f[11]);
  pa.prefill4 = reinterpret_cast<decltype(pa.prefill4)>(f[12]);
  pa.fork_workspace = reinterpret_cast<decltype(pa.fork_workspace)>(f[13]);
  pa.fork = reinterpret_cast<decltype(pa.fork)>(f[14]);
  pa.copy_pages = reinterpret_cast<decltype(pa.copy_pages)>(f[15]);
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
                         PA_METHOD(quantize_and_cache),
                         PA_METHOD(dequantize_kv4),
                         PA_METHOD(decode_kv4),
                         PA_METHOD(chunked_prefill_kv4),
                         PA_METHOD(fork_blocks),
                         PA_METHOD(copy_pages),
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
