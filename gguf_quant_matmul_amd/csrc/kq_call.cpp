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
bool byte_caches(PyObject* ko, PyObject* vo, long device, const at::Tensor** k, const at::Tensor** v) {
  return tensor(ko, device, k) && tensor(vo, device, v) && (*k)->scalar_type() == at::kByte &&
         (*v)->scalar_type() == at::kByte && (*k)->dim() == 3 && (*k)->sizes() == (*v)->sizes() && (*k)->is_contiguous() &&
         (*v)->is_contiguous();
}
bool caches(PyObject* ko, PyObject* vo, long device, int64_t page, int64_t d, const at::Tensor** k,
            const at::Tensor** v) {
  if (!byte_caches(ko, vo, device, k, v)) return false;
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

bool real(PyObject* o, double* v) {
  *v = PyFloat_AsDouble(o);
  if (*v == -1.0 && PyErr_Occurred()) {
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

// An attention call: q, cu_new, seq_lens, table, [prefix,] k_cache, v_cache, page, out, scale, [window, [sinks,]]
// max_new, max_kv, workspace or None, stream, device; no workspace only where none is needed.
enum Kind { PLAIN, SINKS, PREFIX };
template <Kind K>
PyObject* attention(PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *q, *cu, *lens, *table, *prefix = nullptr, *kc, *vc, *out, *ws = nullptr;
    int64_t page, window = 0, sinks = 0, max_new, max_kv, stream, device, qs;
    // places behind the table, behind the scale, behind the windows
    constexpr int at = K == PREFIX ? 5 : 4, win = at + 5, end = win + (K == PLAIN ? 1 : K == SINKS ? 2 : 0);
    if (n != end + 5 || !number(a[at + 2], &page) || (K != PREFIX && !number(a[win], &window)) ||
        (K == SINKS && !number(a[win + 1], &sinks)) || !number(a[end], &max_new) || !number(a[end + 1], &max_kv) ||
        !number(a[end + 3], &stream) || !number(a[end + 4], &device))
      Py_RETURN_NONE;
    double scale;
    if (!real(a[at + 4], &scale)) Py_RETURN_NONE;
    if (!tensor(a[0], device, &q) || !tensor(a[at + 3], device, &out) || !rows(q, &qs) || q->sizes() != out->sizes() ||
        !out->is_contiguous() || dtype(q) < 0 || dtype(out) < 0)
      Py_RETURN_NONE;
    if (!ints(a[2], device, -1, &lens) || !ints(a[3], device, -1, &table)) Py_RETURN_NONE;
    if (K == PREFIX && !ints(a[4], device, -1, &prefix)) Py_RETURN_NONE;
    const int64_t m = lens->numel(), tokens = q->size(0), heads = q->size(1), d = q->size(2);
    if (!ints(a[1], device, m + 1, &cu) || table->dim() != 2 || table->size(0) != m) Py_RETURN_NONE;
    if (!caches(a[at], a[at + 1], device, page, d, &kc, &vc)) Py_RETURN_NONE;
    PyObject* wo = a[end + 2];
    if (wo != Py_None && (!tensor(wo, device, &ws) || !ws->is_contiguous())) Py_RETURN_NONE;
    void* wp = ws ? ws->data_ptr() : nullptr;
    const int64_t wn = ws ? (int64_t)ws->nbytes() : 0;
    int st;
    if constexpr (K == PLAIN)
      st = kq_kv_attention(KQ_Q4_0, q->data_ptr(), dtype(q), tokens, heads, kc->size(1), d, qs, ptr(cu), ptr(lens), m,
                           ptr(table), table->size(1), kc->data_ptr(), vc->data_ptr(), kc->size(0), page, (float)scale,
                           window, max_new, max_kv, out->data_ptr(), dtype(out), wp, wn, (void*)stream);
    else if constexpr (K == SINKS)
      st = kq_kv_attention_sinks(KQ_Q4_0, q->data_ptr(), dtype(q), tokens, heads, kc->size(1), d, qs, ptr(cu), ptr(lens), m,
                                 ptr(table), table->size(1), kc->data_ptr(), vc->data_ptr(), kc->size(0), page,
                                 (float)scale, window, sinks, max_new, max_kv, out->data_ptr(), dtype(out), wp, wn,
                                 (void*)stream);
    else
      st = kq_kv_attention_prefix(KQ_Q4_0, q->data_ptr(), dtype(q), tokens, heads, kc->size(1), d, qs, ptr(cu), ptr(lens), m,
                                  ptr(table), table->size(1), ptr(prefix), prefix->numel(), kc->data_ptr(), vc->data_ptr(),
                                  kc->size(0), page, (float)scale, max_new, max_kv, out->data_ptr(), dtype(out), wp, wn,
                                  (void*)stream);
    if (st == KQ_ERR_CAPACITY && !ws) Py_RETURN_NONE;  // the caller allocates one
    return status(st);
  });
}
PyObject* kv_attention(PyObject*, PyObject* const* a, Py_ssize_t n) { return attention<PLAIN>(a, n); }
PyObject* kv_attention_sinks(PyObject*, PyObject* const* a, Py_ssize_t n) { return attention<SINKS>(a, n); }
PyObject* kv_attention_prefix(PyObject*, PyObject* const* a, Py_ssize_t n) { return attention<PREFIX>(a, n); }

// one count or head, or None
bool maybe_one(PyObject* o, long device, const at::Tensor** t) {
  *t = nullptr;
  return o == Py_None || ints(o, device, 1, t);
}

// (parents, children, lens, page, table, refs, free_pages, free_head, copy_src, copy_dst, free_head_out, status or None,
//  stream, device)
PyObject* kv_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *parents, *children, *lens, *table, *refs, *fp, *fh, *src, *dst, *ho, *st;
    int64_t page, stream, device;
    if (n != 14 || !number(a[3], &page) || !number(a[12], &stream) || !number(a[13], &device)) Py_RETURN_NONE;
    if (!ints(a[0], device, -1, &parents)) Py_RETURN_NONE;
    const int64_t m = parents->numel();
    if (!ints(a[1], device, m, &children) || !ints(a[2], device, m, &lens) || !ints(a[4], device, -1, &table) ||
        table->dim() != 2 || !ints(a[5], device, -1, &refs) || !ints(a[6], device, -1, &fp) || !ints(a[7], device, 1, &fh) ||
        !ints(a[8], device, m, &src) || !ints(a[9], device, m, &dst) || !ints(a[10], device, 1, &ho) ||
        !maybe_one(a[11], device, &st))
      Py_RETURN_NONE;
    return status(kq_kv_fork(ptr(parents), ptr(children), ptr(lens), m, page, ptr(table), table->size(0), table->size(1),
                             ptr(refs), refs->numel(), ptr(fp), fp->numel(), ptr(fh), ptr(src), ptr(dst), ptr(ho),
                             st ? (uint32_t*)ptr(st) : nullptr, (void*)stream));
  });
}

// (first, last, table, refs, free_pages, free_head, free_head_out, status or None, stream, device)
PyObject* kv_free(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *first, *last, *table, *refs, *fp, *fh, *ho, *st;
    int64_t stream, device;
    if (n != 10 || !number(a[8], &stream) || !number(a[9], &device)) Py_RETURN_NONE;
    if (!ints(a[0], device, -1, &first)) Py_RETURN_NONE;
    const int64_t m = first->numel();
    if (!ints(a[1], device, m, &last) || !ints(a[2], device, -1, &table) || table->dim() != 2 || table->size(0) != m ||
        !ints(a[3], device, -1, &refs) || !ints(a[4], device, -1, &fp) || !ints(a[5], device, 1, &fh) ||
        !ints(a[6], device, 1, &ho) || !maybe_one(a[7], device, &st))
      Py_RETURN_NONE;
    return status(kq_kv_free(ptr(first), ptr(last), m, ptr(table), table->size(1), ptr(refs), refs->numel(), ptr(fp),
                             fp->numel(), ptr(fh), ptr(ho), st ? (uint32_t*)ptr(st) : nullptr, (void*)stream));
  });
}

// (free_pages, free_head, table, refs, table_out, refs_out, free_out, remap, copy_src, copy_dst, free_head_out,
//  status or None, stream, device)
PyObject* kv_compact(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *fp, *fh, *table, *refs, *to, *ro, *fo, *remap, *src, *dst, *ho, *st;
    int64_t stream, device;
    if (n != 14 || !number(a[12], &stream) || !number(a[13], &device)) Py_RETURN_NONE;
    if (!ints(a[0], device, -1, &fp) || !ints(a[1], device, 1, &fh) || !ints(a[2], device, -1, &table) ||
        !ints(a[3], device, -1, &refs) || !ints(a[8], device, -1, &src))
      Py_RETURN_NONE;
    const int64_t pages = refs->numel(), entries = table->numel(), n_free = fp->numel(), n_copy = src->numel();
    if (!ints(a[4], device, entries, &to) || !ints(a[5], device, pages, &ro) || !ints(a[6], device, n_free, &fo) ||
        !ints(a[7], device, pages, &remap) || !ints(a[9], device, n_copy, &dst) || !ints(a[10], device, 1, &ho) ||
        !maybe_one(a[11], device, &st))
      Py_RETURN_NONE;
    return status(kq_kv_compact(ptr(fp), n_free, ptr(fh), ptr(table), entries, ptr(refs), pages, ptr(to), ptr(ro), ptr(fo),
                                ptr(remap), ptr(src), ptr(dst), n_copy, ptr(ho), st ? (uint32_t*)ptr(st) : nullptr,
                                (void*)stream));
  });
}

// (src, dst, k_cache, v_cache, stream, device)
PyObject* kv_copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *src, *dst, *k, *v;
    int64_t stream, device;
    if (n != 6 || !number(a[4], &stream) || !number(a[5], &device)) Py_RETURN_NONE;
    if (!ints(a[0], device, -1, &src) || !ints(a[1], device, src->numel(), &dst) || !byte_caches(a[2], a[3], device, &k, &v))
      Py_RETURN_NONE;
    return status(kq_kv_copy_pages(ptr(src), ptr(dst), src->numel(), k->data_ptr(), v->data_ptr(), k->size(0),
                                   k->size(1) * k->size(2), (void*)stream));
  });
}

// (q or None, k or None, cu_new, seq_lens, inv_freq, q_out or None, k_out or None, layout, mscale, stream, device); no
// output: in place
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *x[2] = {nullptr, nullptr}, *out[2], *cu, *lens, *freq, *one = nullptr;
    int64_t layout, stream, device, stride[2] = {0, 0}, ostride[2] = {0, 0};
    double mscale;
    if (n != 11 || !number(a[7], &layout) || !real(a[8], &mscale) || !number(a[9], &stream) || !number(a[10], &device))
      Py_RETURN_NONE;
    if (!ints(a[3], device, -1, &lens) || !ints(a[2], device, lens->numel() + 1, &cu) || !tensor(a[4], device, &freq) ||
        freq->scalar_type() != at::kFloat || !freq->is_contiguous())
      Py_RETURN_NONE;
    for (int i = 0; i < 2; ++i) {
      if (a[i] == Py_None) {
        if (a[5 + i] != Py_None) Py_RETURN_NONE;
        continue;
      }
      if (!tensor(a[i], device, &x[i]) || !rows(x[i], &stride[i]) || dtype(x[i]) < 0) Py_RETURN_NONE;
      out[i] = x[i];
      if (a[5 + i] != Py_None && !tensor(a[5 + i], device, &out[i])) Py_RETURN_NONE;
      if (out[i]->sizes() != x[i]->sizes() || out[i]->scalar_type() != x[i]->scalar_type() || !rows(out[i], &ostride[i]))
        Py_RETURN_NONE;
      if (one && (one->size(0) != x[i]->size(0) || one->size(2) != x[i]->size(2) || one->scalar_type() != x[i]->scalar_type()))
        Py_RETURN_NONE;
      one = x[i];
    }
    if (!one) Py_RETURN_NONE;
    const auto at = [&](const at::Tensor* const* t, int i) { return x[i] ? t[i]->data_ptr() : nullptr; };
    return status(kq_rope(at(x, 0), x[0] ? x[0]->size(1) : 0, stride[0], at(x, 1), x[1] ? x[1]->size(1) : 0, stride[1],
                          dtype(one), one->size(0), one->size(2), 2 * freq->numel(), (int)layout, ptr(cu), ptr(lens),
                          lens->numel(), (const float*)freq->data_ptr(), (float)mscale, at(out, 0), ostride[0], at(out, 1),
                          ostride[1], (void*)stream));
  });
}

PyMethodDef methods[] = {{"kv_store", (PyCFunction)(void*)kv_store, METH_FASTCALL, nullptr},
                         {"kv_load", (PyCFunction)(void*)kv_load, METH_FASTCALL, nullptr},
                         {"block_tables", (PyCFunction)(void*)block_tables, METH_FASTCALL, nullptr},
                         {"kv_attention", (PyCFunction)(void*)kv_attention, METH_FASTCALL, nullptr},
                         {"kv_attention_sinks", (PyCFunction)(void*)kv_attention_sinks, METH_FASTCALL, nullptr},
                         {"kv_attention_prefix", (PyCFunction)(void*)kv_attention_prefix, METH_FASTCALL, nullptr},
                         {"kv_fork", (PyCFunction)(void*)kv_fork, METH_FASTCALL, nullptr},
                         {"kv_free", (PyCFunction)(void*)kv_free, METH_FASTCALL, nullptr},
                         {"kv_compact", (PyCFunction)(void*)kv_compact, METH_FASTCALL, nullptr},
                         {"kv_copy_pages", (PyCFunction)(void*)kv_copy_pages, METH_FASTCALL, nullptr},
                         {"rope", (PyCFunction)(void*)rope, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kqcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kqcall(void) {
  PyObject* m = PyModule_Create(&module);
  // the torch whose tensors this code reads
  if (m && PyModule_AddStringConstant(m, "TORCH", KQ_TORCH) < 0) Py_CLEAR(m);
  return m;
}
