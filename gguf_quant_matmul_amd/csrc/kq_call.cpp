// Calls of the 4-bit cache entry points straight from Python tensors.
//
// kq.py checks its arguments and marshals them through ctypes, about 5 us for
// a store and 8 us for an attention call, which is as long as the kernels of
// a decode step run.  The functions here do the same for the plain good case
// (tensors of the current device, the codec q4_0) in about 1 us: they check
// what kq.py checks and call the C ABI.  Anything else returns None, and the
// caller takes the path in kq.py, which words the error or makes the call.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/kq.h"

namespace {

bool tensor(PyObject* o, long device, const at::Tensor** t) {
  if (!THPVariable_Check(o)) return false;
  *t = &THPVariable_Unpack(o);
  return (*t)->is_cuda() && (*t)->get_device() == device;
}

// contiguous 32-bit integers; n entries unless n < 0
bool ints(PyObject* o, long device, int64_t n, const at::Tensor** t) {
  if (!tensor(o, device, t)) return false;
  const auto type = (*t)->scalar_type();
  return (type == at::kInt || type == at::kUInt32) && (*t)->is_contiguous() && (n < 0 || (*t)->numel() == n);
}
int32_t* ptr(const at::Tensor* t) { return (int32_t*)t->data_ptr(); }

int dtype(const at::Tensor* t) {
  switch (t->scalar_type()) {
    case at::kFloat: return KQ_F32;
    case at::kHalf: return KQ_F16;
    case at::kBFloat16: return KQ_BF16;
    default: return -1;
  }
}

// x [tokens, heads, d] with dense rows; elements between rows
bool rows(const at::Tensor* x, int64_t* stride) {
  if (x->dim() != 3 || x->numel() == 0) return false;
  if (x->stride(2) != 1 || (x->size(1) > 1 && x->stride(1) != x->size(2))) return false;
  *stride = x->size(0) > 1 ? x->stride(0) : x->size(1) * x->size(2);
  return true;
}

// two caches uint8 [pages, kv_heads, page_bytes]
bool caches(PyObject* ko, PyObject* vo, long device, int64_t page, int64_t d, const at::Tensor** k,
            const at::Tensor** v) {
  if (!tensor(ko, device, k) || !tensor(vo, device, v)) return false;
  if ((*k)->scalar_type() != at::kByte || (*v)->scalar_type() != at::kByte || (*k)->dim() != 3 ||
      (*k)->sizes() != (*v)->sizes() || !(*k)->is_contiguous() || !(*v)->is_contiguous())
    return false;
  int64_t bytes;
  return kq_kv_page_bytes(KQ_Q4_0, page, d, &bytes) == KQ_OK && (*k)->size(2) == bytes;
}

bool number(PyObject* o, int64_t* v) {
  *v = PyLong_AsLongLong(o);
  if (*v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}

PyObject* status(int st) { return PyLong_FromLong(st); }

// A C++ exception (an undefined tensor, say) must not pass through Python's
// frames: it takes the caller to the path that reports it.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (...) {
    Py_RETURN_NONE;
  }
}

// (k, v, slots, k_cache, v_cache, page, stream, device)
PyObject* kv_store(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *k, *v, *slots, *kc, *vc;
    int64_t page, stream, device, ks, vs;
    if (n != 8 || !number(a[5], &page) || !number(a[6], &stream) || !number(a[7], &device)) Py_RETURN_NONE;
    if (!tensor(a[0], device, &k) || !tensor(a[1], device, &v) || !rows(k, &ks) || !rows(v, &vs)) Py_RETURN_NONE;
    if (k->sizes() != v->sizes() || k->scalar_type() != v->scalar_type() || dtype(k) < 0) Py_RETURN_NONE;
    const int64_t tokens = k->size(0), heads = k->size(1), d = k->size(2);
    if (!caches(a[3], a[4], device, page, d, &kc, &vc) || kc->size(1) != heads) Py_RETURN_NONE;
    if (!ints(a[2], device, tokens, &slots)) Py_RETURN_NONE;
    return status(kq_kv_store(KQ_Q4_0, k->data_ptr(), v->data_ptr(), dtype(k), tokens, heads, d, ks, vs, ptr(slots),
                              kc->data_ptr(), vc->data_ptr(), kc->size(0), page, (void*)stream));
  });
}

// (k_cache, v_cache, slots, page, k, v, stream, device)
PyObject* kv_load(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *k, *v, *slots, *kc, *vc;
    int64_t page, stream, device;
    if (n != 8 || !number(a[3], &page) || !number(a[6], &stream) || !number(a[7], &device)) Py_RETURN_NONE;
    if (!tensor(a[4], device, &k) || !tensor(a[5], device, &v) || k->dim() != 3) Py_RETURN_NONE;
    if (k->sizes() != v->sizes() || k->scalar_type() != v->scalar_type() || dtype(k) < 0 || !k->is_contiguous() ||
        !v->is_contiguous())
      Py_RETURN_NONE;
    const int64_t tokens = k->size(0), heads = k->size(1), d = k->size(2);
    if (!caches(a[0], a[1], device, page, d, &kc, &vc) || kc->size(1) != heads) Py_RETURN_NONE;
    if (!ints(a[2], device, tokens, &slots)) Py_RETURN_NONE;
    return status(kq_kv_load(KQ_Q4_0, kc->data_ptr(), vc->data_ptr(), kc->size(0), page, heads, d, ptr(slots), tokens,
                             k->data_ptr(), v->data_ptr(), dtype(k), (void*)stream));
  });
}

// (ctx_lens, new_lens, free_pages, free_head, page, table, slots, cu_new, seq_lens, free_head_out, status or None,
//  stream, device)
PyObject* block_tables(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *ctx, *nw, *fp, *fh, *table, *slots, *cu, *lens, *ho, *st = nullptr;
    int64_t page, stream, device;
    if (n != 13 || !number(a[4], &page) || !number(a[11], &stream) || !number(a[12], &device)) Py_RETURN_NONE;
    if (!ints(a[0], device, -1, &ctx)) Py_RETURN_NONE;
    const int64_t m = ctx->numel();
    if (!ints(a[1], device, m, &nw) || !ints(a[2], device, -1, &fp) || !ints(a[3], device, 1, &fh) ||
        !ints(a[5], device, -1, &table) || !ints(a[6], device, -1, &slots) || !ints(a[7], device, m + 1, &cu) ||
        !ints(a[8], device, m, &lens) || !ints(a[9], device, 1, &ho))
      Py_RETURN_NONE;
    if (a[10] != Py_None && !ints(a[10], device, 1, &st)) Py_RETURN_NONE;
    if (table->dim() != 2 || table->size(0) != m) Py_RETURN_NONE;
    return status(kq_block_tables(ptr(ctx), ptr(nw), m, page, ptr(fp), fp->numel(), ptr(fh), ptr(table),
                                  table->size(1), ptr(slots), slots->numel(), ptr(cu), ptr(lens), ptr(ho),
                                  st ? (uint32_t*)ptr(st) : nullptr, (void*)stream));
  });
}

// (q, cu_new, seq_lens, table, k_cache, v_cache, page, out, scale, window, max_new, max_kv, workspace or None, stream,
//  device); no workspace only where none is needed
PyObject* kv_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *q, *cu, *lens, *table, *kc, *vc, *out, *ws = nullptr;
    int64_t page, window, max_new, max_kv, stream, device, qs;
    if (n != 15 || !number(a[6], &page) || !number(a[9], &window) || !number(a[10], &max_new) ||
        !number(a[11], &max_kv) || !number(a[13], &stream) || !number(a[14], &device))
      Py_RETURN_NONE;
    const double scale = PyFloat_AsDouble(a[8]);
    if (scale == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      Py_RETURN_NONE;
    }
    if (!tensor(a[0], device, &q) || !tensor(a[7], device, &out) || !rows(q, &qs) || q->sizes() != out->sizes() ||
        !out->is_contiguous() || dtype(q) < 0 || dtype(out) < 0)
      Py_RETURN_NONE;
    if (!ints(a[2], device, -1, &lens) || !ints(a[3], device, -1, &table)) Py_RETURN_NONE;
    const int64_t m = lens->numel(), tokens = q->size(0), heads = q->size(1), d = q->size(2);
    if (!ints(a[1], device, m + 1, &cu) || table->dim() != 2 || table->size(0) != m) Py_RETURN_NONE;
    if (!caches(a[4], a[5], device, page, d, &kc, &vc)) Py_RETURN_NONE;
    if (a[12] != Py_None && (!tensor(a[12], device, &ws) || !ws->is_contiguous())) Py_RETURN_NONE;
    const int st = kq_kv_attention(KQ_Q4_0, q->data_ptr(), dtype(q), tokens, heads, kc->size(1), d, qs, ptr(cu),
                                   ptr(lens), m, ptr(table), table->size(1), kc->data_ptr(), vc->data_ptr(),
                                   kc->size(0), page, (float)scale, window, max_new, max_kv, out->data_ptr(),
                                   dtype(out), ws ? ws->data_ptr() : nullptr,
                                   ws ? (int64_t)ws->nbytes() : 0, (void*)stream);
    if (st == KQ_ERR_CAPACITY && !ws) Py_RETURN_NONE;  // the caller allocates one
    return status(st);
  });
}

PyMethodDef methods[] = {{"kv_store", (PyCFunction)(void*)kv_store, METH_FASTCALL, nullptr},
                         {"kv_load", (PyCFunction)(void*)kv_load, METH_FASTCALL, nullptr},
                         {"block_tables", (PyCFunction)(void*)block_tables, METH_FASTCALL, nullptr},
                         {"kv_attention", (PyCFunction)(void*)kv_attention, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kqcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kqcall(void) {
  PyObject* m = PyModule_Create(&module);
  // the torch whose tensors this code reads
  if (m && PyModule_AddStringConstant(m, "TORCH", KQ_TORCH) < 0) Py_CLEAR(m);
  return m;
}
