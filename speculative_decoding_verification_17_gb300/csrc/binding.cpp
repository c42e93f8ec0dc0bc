// binding.cpp — the checks and the marshalling of the calls on logits and on the paged cache, for
// Python (built into _build/_calls.so).
//
// Each function takes the Python call's arguments in order, checks them as the functions of
// __init__.py do, and calls the C ABI. It returns the call's status, or None when an argument
// does not fit: the Python side then repeats the checks one by one and raises. The C ABI's
// functions are handed over once by address (bind), so that both sides use one loaded library.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cmath>
#include <initializer_list>

#include <ATen/ATen.h>
#include <torch/csrc/autograd/python_variable.h>

#include "specverify_kv.h"
#include "specverify_logits.h"

namespace {

decltype(&logit_adjust) p_adjust;
decltype(&paged_attention) p_attention;
decltype(&paged_attention_workspace) p_workspace;
decltype(&attention_weight_sum) p_weights;
decltype(&kv_cache_evict) p_evict;

PyObject* none() { Py_RETURN_NONE; }

// A tensor argument; `none_ok` for one that may be missing.
struct Arg {
  const at::Tensor* t = nullptr;
  bool ok = true;
  Arg(PyObject* o, bool none_ok = false) {
    if (THPVariable_Check(o))
      t = &THPVariable_Unpack(o);
    else
      ok = none_ok && o == Py_None;
  }
  explicit operator bool() const { return t != nullptr; }
  // Whether it is missing, or contiguous on the device with this type and these sizes.
  bool fits(at::ScalarType type, const at::Device& dev, std::initializer_list<int64_t> sizes) const {
    if (!t) return ok;
    return t->scalar_type() == type && t->device() == dev &&
           t->sizes() == at::IntArrayRef(sizes.begin(), sizes.size()) && t->is_contiguous();
  }
  template <typename T>
  T* ptr() const {
    return t ? static_cast<T*>(t->data_ptr()) : nullptr;
  }
};

bool number(PyObject* o, double* x) {
  *x = PyFloat_AsDouble(o);
  if (*x == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}
// An integer, or what has one's value (numpy's).
bool whole(PyObject* o, long long* x) {
  if (!PyIndex_Check(o)) return false;
  *x = PyLong_AsLongLong(o);
  if (*x == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}
bool small(PyObject* o, int* x) {
  long long v;
  if (!whole(o, &v) || v < INT32_MIN || v > INT32_MAX) return false;
  *x = (int)v;
  return true;
}

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 5) return PyErr_Format(PyExc_TypeError, "bind takes five addresses");
  void* p[5];
  for (int i = 0; i < 5; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i]) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "null address");
  }
  p_adjust = reinterpret_cast<decltype(p_adjust)>(p[0]);
  p_attention = reinterpret_cast<decltype(p_attention)>(p[1]);
  p_workspace = reinterpret_cast<decltype(p_workspace)>(p[2]);
  p_weights = reinterpret_cast<decltype(p_weights)>(p[3]);
  p_evict = reinterpret_cast<decltype(p_evict)>(p[4]);
  return none();
}

// logits, history, hist_len, prompt_len, draft_tokens, num_draft, repetition, presence, frequency,
// bias_tokens, bias_values, allowed, out, stream
PyObject* adjust(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 14) return none();
  const Arg z(a[0]), hist(a[1], true), hlen(a[2], true), plen(a[3], true), draft(a[4], true),
      nd(a[5], true), rep(a[6], true), pres(a[7], true), freq(a[8], true), bt(a[9], true),
      bv(a[10], true), allowed(a[11], true), out(a[12]);
  long long stream;
  if (!z || !out || !whole(a[13], &stream) || z.t->dim() != 3 || !z.t->is_cuda()) return none();
  const at::ScalarType type = z.t->scalar_type();
  const at::Device dev = z.t->device();
  const int64_t B = z.t->size(0), P = z.t->size(1), V = z.t->size(2);
  if ((type != at::kFloat && type != at::kBFloat16) || (V > 1 && z.t->stride(2) != 1)) return none();
  if (out.t->scalar_type() != type || out.t->device() != dev || out.t->sizes() != z.t->sizes() ||
      (V > 1 && out.t->stride(2) != 1))
    return none();
  const int64_t L = hist && hist.t->dim() == 2 ? hist.t->size(1) : 0;
  const int64_t nb = bt && bt.t->dim() == 2 ? bt.t->size(1) : 0;
  if (B > INT32_MAX || V > INT32_MAX || L > INT32_MAX || nb > INT32_MAX) return none();
  if (!hist.fits(at::kInt, dev, {B, L}) || !hlen.fits(at::kInt, dev, {B}) ||
      !plen.fits(at::kInt, dev, {B}) || !draft.fits(at::kInt, dev, {B, P - 1}) ||
      !nd.fits(at::kInt, dev, {B}) || !rep.fits(at::kFloat, dev, {B}) ||
      !pres.fits(at::kFloat, dev, {B}) || !freq.fits(at::kFloat, dev, {B}) ||
      !bt.fits(at::kInt, dev, {B, nb}) || !bv.fits(at::kFloat, dev, {B, nb}) ||
      !allowed.fits(at::kInt, dev, {B, P, (V + 31) / 32}))
    return none();
  const bool biased = nb > 0;
  const sv_status s = p_adjust(
      z.ptr<void>(), z.t->stride(0), z.t->stride(1), type == at::kFloat ? SV_F32 : SV_BF16,
      hist.ptr<int32_t>(), hlen.ptr<int32_t>(), plen.ptr<int32_t>(), (int)L, draft.ptr<int32_t>(),
      nd.ptr<int32_t>(), rep.ptr<float>(), pres.ptr<float>(), freq.ptr<float>(),
      biased ? bt.ptr<int32_t>() : nullptr, biased ? bv.ptr<float>() : nullptr, (int)nb,
      allowed.ptr<uint32_t>(), (int)B, (int)P, (int)V, out.ptr<void>(), out.t->stride(0),
      out.t->stride(1), reinterpret_cast<sv_stream_t>(stream));
  return PyLong_FromLong(s);
}

// A pool [pages, page_size, Hkv, D] like `k` (its type, device and last three sizes).
bool pool_of(const Arg& a, const at::Tensor& k, sv_kv_pool* p) {
  if (!a || a.t->dim() != 4 || k.dim() != 4) return false;
  const at::Tensor& t = *a.t;
  if (t.scalar_type() != k.scalar_type() || t.device() != k.device() || t.size(1) != k.size(1) ||
      t.size(2) != k.size(2) || t.size(3) != k.size(3) || (t.size(3) > 1 && t.stride(3) != 1))
    return false;
  *p = sv_kv_pool{t.data_ptr(), t.stride(0), t.stride(1), t.stride(2)};
  return true;
}

bool kv_dtype(const at::Tensor& t, sv_kv_dtype* d) {
  if (!t.is_cuda()) return false;
  if (t.scalar_type() == at::kBFloat16)
    *d = SV_KV_BF16;
  else if (t.scalar_type() == at::kHalf)
    *d = SV_KV_F16;
  else
    return false;
  return true;
}

// What the calls with queries share: q, k_cache, page_table, seq_len, num_draft, slopes, scale
// (None for D ** -0.5), softcap, window.
struct Queries {
  Arg q, k, table, lens, nd, slopes;
  sv_kv_shape shape;
  sv_score_rule rule;
  sv_kv_pool pool;
  bool ok = false;
  explicit Queries(PyObject* const* a)
      : q(a[0]), k(a[1]), table(a[2]), lens(a[3]), nd(a[4], true), slopes(a[5], true) {
    if (!q || !k || !table || !lens || q.t->dim() != 4 || k.t->dim() != 4 || table.t->dim() != 2)
      return;
    if (!kv_dtype(*q.t, &shape.dtype) || q.t->stride(3) != 1) return;
    const at::Device dev = q.t->device();
    const int64_t B = q.t->size(0), Hq = q.t->size(2), D = q.t->size(3), cols = table.t->size(1);
    if (k.t->scalar_type() != q.t->scalar_type() || k.t->device() != dev || k.t->size(3) != D)
      return;
    if (!table.fits(at::kInt, dev, {B, cols}) || !lens.fits(at::kInt, dev, {B}) ||
        !nd.fits(at::kInt, dev, {B}) || !slopes.fits(at::kFloat, dev, {Hq}))
      return;
    for (int64_t x : {B, Hq, k.t->size(0), cols})
      if (x > INT32_MAX) return;
    shape.B = (int)B;
    shape.P = (int)q.t->size(1);
    shape.Hq = (int)Hq;
    shape.Hkv = (int)k.t->size(2);
    shape.D = (int)D;
    shape.page_size = (int)k.t->size(1);
    shape.num_pages = (int)k.t->size(0);
    shape.max_pages = (int)cols;
    double scale = 1.0 / std::sqrt((double)D), softcap;
    if ((a[6] != Py_None && !number(a[6], &scale)) || !number(a[7], &softcap) ||
        !small(a[8], &rule.window))
      return;
    rule.scale = (float)scale;
    rule.softcap = (float)softcap;
    rule.slopes = slopes.ptr<float>();
    ok = pool_of(k, *k.t, &pool);
  }
};
constexpr int kQueryArgs = 9;

// <queries>, v_cache, out, out_lse, workspace, stream. With workspace None: the bytes it needs.
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != kQueryArgs + 5) return none();
  const Queries Q(a);
  const Arg v(a[9]), out(a[10]), lse(a[11], true), ws(a[12], true);
  long long stream;
  sv_kv_pool vp;
  if (!Q.ok || !out || !ws.ok || !whole(a[13], &stream) || !pool_of(v, *Q.k.t, &vp) ||
      v.t->size(0) != Q.k.t->size(0))
    return none();
  const at::Device dev = Q.q.t->device();
  const int64_t B = Q.shape.B, P = Q.shape.P, Hq = Q.shape.Hq, D = Q.shape.D;
  if (!out.fits(Q.q.t->scalar_type(), dev, {B, P, Hq, D}) || !lse.fits(at::kFloat, dev, {B, P, Hq}))
    return none();
  if (ws && (ws.t->device() != dev || !ws.t->is_contiguous())) return none();
  const size_t need = p_workspace(&Q.shape);
  if (!ws || ws.t->nbytes() < need) return PyLong_FromLongLong(-(long long)need - 1);
  const sv_status s = p_attention(
      &Q.shape, &Q.rule, Q.q.ptr<void>(), Q.q.t->stride(0), Q.q.t->stride(1), Q.q.t->stride(2),
      &Q.pool, &vp, Q.table.ptr<int32_t>(), Q.lens.ptr<int32_t>(), Q.nd.ptr<int32_t>(),
      out.ptr<void>(), lse.ptr<float>(), ws.ptr<void>(), ws.t->nbytes(),
      reinterpret_cast<sv_stream_t>(stream));
  return PyLong_FromLong(s);
}

// <queries>, lse, accept_len, prior, out, stream
PyObject* weights(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != kQueryArgs + 5) return none();
  const Queries Q(a);
  const Arg lse(a[9]), acc(a[10], true), prior(a[11], true), out(a[12]);
  long long stream;
  if (!Q.ok || !lse || !out || out.t->dim() != 3 || !whole(a[13], &stream)) return none();
  const at::Device dev = Q.q.t->device();
  const int64_t B = Q.shape.B, P = Q.shape.P, Hq = Q.shape.Hq, Hkv = Q.shape.Hkv;
  const int64_t N = out.t->size(2);
  if (lse.t->scalar_type() != at::kFloat || lse.t->device() != dev || lse.t->dim() != 3 ||
      lse.t->size(0) != B || lse.t->size(1) != P || lse.t->size(2) != Hq ||
      !acc.fits(at::kInt, dev, {B}) || !prior.fits(at::kFloat, dev, {B, Hkv, N}) ||
      !out.fits(at::kFloat, dev, {B, Hkv, N}))
    return none();
  const sv_status s = p_weights(
      &Q.shape, &Q.rule, Q.q.ptr<void>(), Q.q.t->stride(0), Q.q.t->stride(1), Q.q.t->stride(2),
      &Q.pool, Q.table.ptr<int32_t>(), Q.lens.ptr<int32_t>(), Q.nd.ptr<int32_t>(),
      lse.ptr<float>(), lse.t->stride(0), lse.t->stride(1), lse.t->stride(2), acc.ptr<int32_t>(),
      prior.ptr<float>(), out.ptr<float>(), N, reinterpret_cast<sv_stream_t>(stream));
  return PyLong_FromLong(s);
}

// k_cache, v_cache, page_table, seq_len, weights, budget, recent, new_k, new_v, new_page_table,
// out_len, out_index, out_weights (None: made here), stream. Returns (status, the three outputs).
PyObject* evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 14) return none();
  const Arg k(a[0]), v(a[1]), table(a[2]), lens(a[3]), w(a[4]), nk(a[7]), nv(a[8]), ntable(a[9]),
      len(a[10], true), index(a[11], true), kept(a[12], true);
  int budget, recent;
  long long stream;
  if (!k || !v || !table || !lens || !w || !nk || !nv || !ntable || !len.ok || !index.ok ||
      !kept.ok || !small(a[5], &budget) || !small(a[6], &recent) || !whole(a[13], &stream) ||
      budget < 0)
    return none();
  sv_kv_shape shape;
  sv_kv_pool pools[4];
  if (!kv_dtype(*k.t, &shape.dtype) || !pool_of(k, *k.t, &pools[0]) ||
      !pool_of(v, *k.t, &pools[1]) || !pool_of(nk, *k.t, &pools[2]) ||
      !pool_of(nv, *k.t, &pools[3]) || v.t->size(0) != k.t->size(0) ||
      nv.t->size(0) != nk.t->size(0) || table.t->dim() != 2 || ntable.t->dim() != 2 ||
      w.t->dim() != 3)
    return none();
  const at::Device dev = k.t->device();
  const int64_t B = table.t->size(0), cols = table.t->size(1), ncols = ntable.t->size(1);
  const int64_t Hkv = k.t->size(2), N = w.t->size(2);
  for (int64_t x : {B, cols, ncols, k.t->size(0), nk.t->size(0)})
    if (x > INT32_MAX) return none();
  if (!table.fits(at::kInt, dev, {B, cols}) || !lens.fits(at::kInt, dev, {B}) ||
      !w.fits(at::kFloat, dev, {B, Hkv, N}) || !ntable.fits(at::kInt, dev, {B, ncols}) ||
      !len.fits(at::kInt, dev, {B}) || !index.fits(at::kInt, dev, {B, Hkv, budget}) ||
      !kept.fits(at::kFloat, dev, {B, Hkv, budget}))
    return none();
  // (before outputs of that size are made)
  if (budget < 1 || budget > ncols * k.t->size(1))
    return Py_BuildValue("(iOOO)", (int)SV_ERR_INVALID_ARG, Py_None, Py_None, Py_None);
  const auto made = [&](const Arg& given, at::IntArrayRef sizes, at::ScalarType type) {
    return given ? *given.t : at::empty(sizes, at::TensorOptions().dtype(type).device(dev));
  };
  const at::Tensor o_len = made(len, {B}, at::kInt);
  const at::Tensor o_index = made(index, {B, Hkv, budget}, at::kInt);
  const at::Tensor o_kept = made(kept, {B, Hkv, budget}, at::kFloat);
  shape.B = (int)B;
  shape.P = 1;
  shape.Hq = shape.Hkv = (int)Hkv;
  shape.D = (int)k.t->size(3);
  shape.page_size = (int)k.t->size(1);
  shape.num_pages = (int)k.t->size(0);
  shape.max_pages = (int)cols;
  const sv_status s = p_evict(
      &shape, &pools[0], &pools[1], table.ptr<int32_t>(), lens.ptr<int32_t>(), w.ptr<float>(), N,
      budget, recent, &pools[2], &pools[3], (int)nk.t->size(0), ntable.ptr<int32_t>(),
      (int)ncols, static_cast<int32_t*>(o_len.data_ptr()),
      static_cast<int32_t*>(o_index.data_ptr()), static_cast<float*>(o_kept.data_ptr()),
      reinterpret_cast<sv_stream_t>(stream));
  return Py_BuildValue("(iNNN)", (int)s, THPVariable_Wrap(o_len), THPVariable_Wrap(o_index),
                       THPVariable_Wrap(o_kept));
}

// No exception may pass into the interpreter: a tensor without storage (of a transform, a sparse one)
// throws where its address or strides are read, an allocation where memory is short. The Python side
// then meets the same and raises it.
template <PyObject* (*kCall)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return kCall(self, a, n);
  } catch (...) {
    return none();
  }
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {"adjust", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<adjust>)), METH_FASTCALL, nullptr},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<attention>)), METH_FASTCALL, nullptr},
    {"weights", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<weights>)), METH_FASTCALL, nullptr},
    {"evict", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(guarded<evict>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&module); }
