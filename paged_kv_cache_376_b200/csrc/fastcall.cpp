// The ordinary calls of the serving operators without Python's per-tensor
// checks: about ten tensors a call, each with five attributes, cost 6-8 us
// there, more than the smallest of these calls take on the GPU.
//
// Every function here makes the same checks and the same C call as its Python
// counterpart in _lib.py, on the current device and stream.  It returns True
// when the call was made, and False, having done nothing, whenever anything is
// not exactly as it should be (or the C call returned an error): the Python
// counterpart then says what is wrong, or handles the rare form.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "tv.h"

namespace {

// The tensors of one call: all on one CUDA device.
struct Call {
  int device = -1;
  bool ok = true;

  const at::Tensor* any(PyObject* o, at::ScalarType type) {
    if (!THPVariable_Check(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.scalar_type() != type) {
      ok = false;
      return nullptr;
    }
    const int d = t.get_device();
    if (device < 0) device = d;
    if (d != device) ok = false;
    return &t;
  }
  const at::Tensor* contiguous(PyObject* o, at::ScalarType type) {
    const at::Tensor* t = any(o, type);
    if (t && !t->is_contiguous()) ok = false;
    return t;
  }
  const at::Tensor* bf16(PyObject* o) {
    return contiguous(o, at::kBFloat16);
  }
  const at::Tensor* ints(PyObject* o) { return contiguous(o, at::kInt); }
  // pointer of an optional tensor (one without elements has none, which must
  // not pass for None)
  void* maybe(PyObject* o, at::ScalarType type) {
    if (o == Py_None) return nullptr;
    const at::Tensor* t = contiguous(o, type);
    if (!t || t->numel() == 0) {
      ok = false;
      return nullptr;
    }
    return t->data_ptr();
  }
  void need(bool condition) { ok = ok && condition; }
  // the launch goes to the current device's current stream
  bool ready() { return ok && c10::cuda::current_device() == device; }
  void* stream() {
    return c10::cuda::getCurrentCUDAStream(device).stream();
  }
};

bool to_int(PyObject* o, long long* v) {
  *v = PyLong_AsLongLong(o);
  if (*v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}

PyObject* done(bool made) {
  if (made) Py_RETURN_TRUE;
  Py_RETURN_FALSE;
}

// A tensor that has no strides, or no memory, throws when asked for them; that
// ends here, not in the interpreter.
using Function = PyObject* (*)(PyObject* const*, Py_ssize_t);
template <Function kFunction>
PyObject* guarded(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    return kFunction(a, n);
  } catch (...) {
    return done(false);
  }
}
template <Function kFunction>
PyMethodDef method(const char* name) {
  return {name, (PyCFunction)(void (*)())guarded<kFunction>, METH_FASTCALL,
          nullptr};
}

bool fits_int(int64_t v) { return v >= 0 && v <= INT32_MAX; }

// chunk(causal, out, q, query_start_loc, k_pool, v_pool, block_tables, lens,
//       scale, max_query_len, workspace, err)
PyObject* chunk(PyObject* const* a, Py_ssize_t n) {
  if (n != 12) return done(false);
  Call c;
  const int causal = PyObject_IsTrue(a[0]);
  const at::Tensor* out = c.bf16(a[1]);
  const at::Tensor* q = c.bf16(a[2]);
  const at::Tensor* qsl = c.ints(a[3]);
  const at::Tensor* k = c.bf16(a[4]);
  const at::Tensor* v = c.bf16(a[5]);
  const at::Tensor* bt = c.ints(a[6]);
  const at::Tensor* lens = c.ints(a[7]);
  const double scale = PyFloat_Check(a[8]) ? PyFloat_AS_DOUBLE(a[8]) : -1.0;
  long long max_len = 0;
  c.need(PyFloat_Check(a[8]) && to_int(a[9], &max_len) && fits_int(max_len));
  void* ws = c.maybe(a[10], at::kByte);
  void* err = c.maybe(a[11], at::kInt);
  if (!c.ready()) return done(false);
  c.need(q->dim() == 3 && out->sizes() == q->sizes() && k->dim() == 4 &&
         v->sizes() == k->sizes() && lens->dim() == 1 && qsl->dim() == 1 &&
         bt->dim() == 2);
  if (!c.ok) return done(false);
  const int64_t b = lens->size(0);
  c.need(q->size(2) == k->size(3) && qsl->size(0) == b + 1 &&
         bt->size(0) == b && fits_int(b) && fits_int(bt->size(1)));
  if (!c.ok) return done(false);
  const size_t bytes =
      ws ? (size_t)THPVariable_Unpack(a[10]).numel() : (size_t)0;
  const auto call = causal ? tv_paged_chunk : tv_paged_cross_attention;
  return done(
      call(out->data_ptr(), q->data_ptr(), q->size(0),
           (const int32_t*)qsl->data_ptr(), k->data_ptr(), v->data_ptr(),
           (const int32_t*)bt->data_ptr(), (int)bt->size(1),
           (const int32_t*)lens->data_ptr(), (int)b, (int)max_len,
           (int)q->size(1), (int)k->size(2), (int)k->size(3),
           (int)k->size(1), k->size(0), (float)scale, ws, bytes,
           (uint32_t*)err, c.stream()) == TV_OK);
}

// mrope(q_out, q, k_new, v_new, slot_mapping, positions, pair_axis, k_pool,
//       v_pool, cos_sin, err), q and q_out not None
PyObject* mrope(PyObject* const* a, Py_ssize_t n) {
  if (n != 11) return done(false);
  Call c;
  const at::Tensor* out = c.bf16(a[0]);
  const at::Tensor* q = c.any(a[1], at::kBFloat16);
  const at::Tensor* k = c.any(a[2], at::kBFloat16);
  const at::Tensor* v = c.any(a[3], at::kBFloat16);
  const at::Tensor* slots = c.ints(a[4]);
  const at::Tensor* pos = c.ints(a[5]);
  const at::Tensor* axis = c.ints(a[6]);
  const at::Tensor* kp = c.bf16(a[7]);
  const at::Tensor* vp = c.bf16(a[8]);
  const at::Tensor* tab = c.contiguous(a[9], at::kFloat);
  void* err = c.maybe(a[10], at::kInt);
  if (!c.ready()) return done(false);
  c.need(kp->dim() == 4 && vp->sizes() == kp->sizes() && q->dim() == 3 &&
         k->dim() == 3 && v->dim() == 3 && out->sizes() == q->sizes() &&
         v->sizes() == k->sizes() && pos->dim() == 2 && tab->dim() == 3);
  if (!c.ok) return done(false);
  const int64_t t = k->size(0), hkv = kp->size(2), d = kp->size(3);
  c.need(t > 0 && k->size(1) == hkv && k->size(2) == d && q->size(0) == t &&
         q->size(2) == d && slots->dim() == 1 && slots->size(0) == t &&
         pos->size(1) == t && axis->dim() == 1 && axis->size(0) == d / 2 &&
         tab->size(1) == 2 && tab->size(2) == d / 2 &&
         fits_int(tab->size(0)));
  // token rows may be strided, the heads of one are contiguous
  for (const at::Tensor* x : {q, k, v})
    c.need(x->stride(2) == 1 && (x->size(1) == 1 || x->stride(1) == d));
  if (!c.ok) return done(false);
  auto row = [t](const at::Tensor* x) {   // one token has no stride to speak of
    return t > 1 ? x->stride(0) : x->size(1) * x->size(2);
  };
  return done(
      tv_kv_append_mrope(
          out->data_ptr(), q->data_ptr(), row(q), k->data_ptr(), row(k),
          v->data_ptr(), row(v),
          (const int32_t*)slots->data_ptr(), (const int32_t*)pos->data_ptr(),
          (int)pos->size(0), (const int32_t*)axis->data_ptr(), t,
          kp->data_ptr(), vp->data_ptr(), kp->size(0), (int)q->size(1),
          (int)hkv, (int)d, (int)kp->size(1), (const float*)tab->data_ptr(),
          (int)tab->size(0), (uint32_t*)err, c.stream()) == TV_OK);
}

int64_t pool_pages(const at::Tensor* state) {
  const int64_t n = state->numel() - 4 - TV_POOL_MAX_SEQS;
  return n > 0 && n % 4 == 0 ? n / 4 : -1;
}

// truncate(state, block_tables, context_lens, new_lens, err)
PyObject* truncate(PyObject* const* a, Py_ssize_t n) {
  if (n != 5) return done(false);
  Call c;
  const at::Tensor* state = c.ints(a[0]);
  const at::Tensor* bt = c.ints(a[1]);
  const at::Tensor* ctx = c.ints(a[2]);
  const at::Tensor* len = c.ints(a[3]);
  void* err = c.maybe(a[4], at::kInt);
  if (!c.ready()) return done(false);
  c.need(bt->dim() == 2 && ctx->dim() == 1 && len->sizes() == ctx->sizes() &&
         bt->size(0) == ctx->size(0) && fits_int(bt->size(0)) &&
         fits_int(bt->size(1)) && pool_pages(state) > 0);
  if (!c.ok) return done(false);
  return done(tv_pool_truncate(
                  (int32_t*)state->data_ptr(), pool_pages(state),
                  (int32_t*)bt->data_ptr(), (int)bt->size(1),
                  (int32_t*)ctx->data_ptr(), (const int32_t*)len->data_ptr(),
                  (int)bt->size(0), (uint32_t*)err, c.stream()) == TV_OK);
}

// compact(state, block_tables, context_lens, moves, num_moves, k_pool, v_pool,
//         err), pools not None
PyObject* compact(PyObject* const* a, Py_ssize_t n) {
  if (n != 8) return done(false);
  Call c;
  const at::Tensor* state = c.ints(a[0]);
  const at::Tensor* bt = c.ints(a[1]);
  const at::Tensor* ctx = c.ints(a[2]);
  const at::Tensor* moves = c.ints(a[3]);
  const at::Tensor* count = c.ints(a[4]);
  const at::Tensor* k = c.bf16(a[5]);
  const at::Tensor* v = c.bf16(a[6]);
  void* err = c.maybe(a[7], at::kInt);
  if (!c.ready()) return done(false);
  c.need(bt->dim() == 2 && ctx->dim() == 1 && bt->size(0) == ctx->size(0) &&
         fits_int(bt->size(0)) && fits_int(bt->size(1)) && moves->dim() == 2 &&
         moves->size(0) == 2 && count->numel() >= 1 && k->dim() == 4 &&
         v->sizes() == k->sizes() && pool_pages(state) > 0 &&
         k->size(0) == pool_pages(state));
  if (!c.ok) return done(false);
  const int64_t cap = moves->size(1);
  int32_t* list = (int32_t*)moves->data_ptr();
  return done(tv_pool_compact(
                  (int32_t*)state->data_ptr(), pool_pages(state),
                  (int32_t*)bt->data_ptr(), (int)bt->size(1),
                  (const int32_t*)ctx->data_ptr(), (int)bt->size(0), list,
                  list + cap, cap, (int32_t*)count->data_ptr(), k->data_ptr(),
                  v->data_ptr(), (int)k->size(2), (int)k->size(3),
                  (int)k->size(1), (uint32_t*)err, c.stream()) == TV_OK);
}

// page_copy(k_pool, v_pool, src_pages, dst_pages, num_pairs, err)
PyObject* page_copy(PyObject* const* a, Py_ssize_t n) {
  if (n != 6) return done(false);
  Call c;
  const at::Tensor* k = c.bf16(a[0]);
  const at::Tensor* v = c.bf16(a[1]);
  const at::Tensor* src = c.ints(a[2]);
  const at::Tensor* dst = c.ints(a[3]);
  void* pairs = c.maybe(a[4], at::kInt);
  void* err = c.maybe(a[5], at::kInt);
  if (!c.ready()) return done(false);
  c.need(k->dim() == 4 && v->sizes() == k->sizes() && src->dim() == 1 &&
         dst->sizes() == src->sizes());
  if (!c.ok) return done(false);
  return done(tv_page_copy(k->data_ptr(), v->data_ptr(), k->size(0),
                           (const int32_t*)src->data_ptr(),
                           (const int32_t*)dst->data_ptr(), src->size(0),
                           (const int32_t*)pairs, (int)k->size(2),
                           (int)k->size(3), (int)k->size(1), (uint32_t*)err,
                           c.stream()) == TV_OK);
}

PyMethodDef kMethods[] = {
    method<chunk>("chunk"),         method<mrope>("mrope"),
    method<truncate>("truncate"),   method<compact>("compact"),
    method<page_copy>("page_copy"), {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fastcall",
                       "The serving operators' ordinary calls.", -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&kModule); }
