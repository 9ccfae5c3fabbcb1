// The Python binding's marshalling of the serving step's calls, in C++.
//
// A step's calls are a few microseconds of GPU work each; reading a dozen
// tensors' attributes, cutting outputs and converting thirty arguments from
// Python costs two to three times the launch itself (a Grace host: 25 us for a
// layout, 22 us for a norm and rotation).  These functions do that part for the
// ordinary case -- tensors as documented, outputs allocated here, the current
// device and stream -- and call the same C entry points.  Anything else returns
// None, nothing launched: the binding's Python code then takes the call, or says
// what is wrong with it.  A status other than 0 comes back as a number.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "dsa.h"

namespace {

decltype(&dsa_batch_layout) batch_layout_fn = nullptr;
decltype(&dsa_qk_norm_rope) qk_norm_rope_fn = nullptr;
decltype(&dsa_chunk_mla_fwd) chunk_mla_fn = nullptr;
decltype(&dsa_combine) combine_fn = nullptr;
decltype(&dsa_chunk_pick_num_splits) pick_fn = nullptr;
decltype(&dsa_verify_draft_req) verify_draft_fn = nullptr;

// Reads a call's arguments; `good` is false once one is not as documented.
struct Args {
  PyObject* const* a;
  int i = 0;
  int dev = -1;
  bool good = true;

  PyObject* next() { return a[i++]; }
  // a tensor, or null for None
  const at::Tensor* any() {
    PyObject* o = next();
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) {
      good = false;
      return nullptr;
    }
    return &THPVariable_Unpack(o);
  }
  bool placed(const at::Tensor& t, int64_t dim) {
    if (!t.is_cuda() || t.dim() != dim) return good = false;
    const int d = (int)t.get_device();
    if (dev < 0) {
      dev = d;
      if (d != (int)c10::cuda::current_device()) good = false;
    }
    return good = good && d == dev;
  }
  // contiguous, of this type and rank, on the first tensor's device (the current one)
  const at::Tensor* tensor(at::ScalarType type, int64_t dim, bool optional = false) {
    const at::Tensor* t = any();
    if (!t) {
      good = good && optional;
      return nullptr;
    }
    if (t->scalar_type() != type || !placed(*t, dim) || !t->is_contiguous()) good = false;
    return t;
  }
  int64_t integer() {
    const long long v = PyLong_AsLongLong(next());
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      good = false;
    }
    return v;
  }
  int32_t int32() {
    const int64_t v = integer();
    if (v != (int32_t)v) good = false;
    return (int32_t)v;
  }
  float number() {
    const double v = PyFloat_AsDouble(next());
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      good = false;
    }
    return (float)v;
  }
  int32_t* status() {
    const at::Tensor* t = any();
    if (!t) return nullptr;
    if (t->scalar_type() != at::kInt || !placed(*t, t->dim()) || !t->is_contiguous() || t->numel() < 1) good = false;
    return good ? t->data_ptr<int32_t>() : nullptr;
  }
  void* stream() const { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream(); }
};

// Other threads run while an entry point launches (a full launch queue makes it wait).
struct Unlocked {
  PyThreadState* s = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(s); }
};
template <class F, class... A>
dsa_status call(F fn, A... args) {
  Unlocked u;
  return fn(args...);
}

template <class T>
T* ptr(const at::Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}
int64_t stride(const at::Tensor* t, int64_t dim) { return t && t->size(dim) > 1 ? t->stride(dim) : 0; }
bool fits32(int64_t n) { return n <= INT32_MAX; }

// A contiguous tensor over part of a fresh buffer's storage (`at` in elements of
// `type`): outputs that share an allocation, which lives as long as one of them.
at::Tensor cut(const at::Tensor& buf, int64_t at, at::IntArrayRef sizes, at::ScalarType type) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(buf.storage()), buf.key_set(),
                                                         c10::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_storage_offset(at);
  t.unsafeGetTensorImpl()->set_sizes_contiguous(sizes);
  return t;
}
at::Tensor bytes(int64_t n, const at::Tensor& like) { return at::empty({n}, like.options().dtype(at::kByte)); }

PyObject* tuple_of(std::initializer_list<const at::Tensor*> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor* t : ts) {
    PyObject* o = t ? THPVariable_Wrap(*t) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

// (ctx_len, new_len, pages_held, block_table, free_pages, free_used, page_size, num_pages, capacity, dev_status)
PyObject* batch_layout(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  HANDLE_TH_ERRORS
  if (argc != 10) Py_RETURN_NONE;
  Args a{argv};
  const at::Tensor* ctx = a.tensor(at::kInt, 1);
  const at::Tensor* nw = a.tensor(at::kInt, 1);
  const at::Tensor* held = a.tensor(at::kInt, 1);
  const at::Tensor* table = a.tensor(at::kInt, 2);
  const at::Tensor* free = a.tensor(at::kInt, 1);
  const at::Tensor* used = a.tensor(at::kInt, 1);
  const int32_t page = a.int32();
  const int64_t pages = a.integer();
  const int32_t cap = a.int32();
  int32_t* st = a.status();
  if (!a.good || cap < 0) Py_RETURN_NONE;
  const int64_t R = ctx->size(0);
  if (nw->size(0) != R || held->size(0) != R || table->size(0) != R || used->size(0) != 1 || !fits32(R) ||
      !fits32(table->size(1)) || !fits32(free->size(0)))
    Py_RETURN_NONE;
  // The token arrays first, a multiple of 16 bytes apart.  The requests' state, which the
  // next step keeps, does not keep token arrays of more than 64 KB with it: it then has an
  // allocation of its own (0.8 us of host time, 7.7 -> 8.5, which only short calls show).
  const int64_t c4 = ((int64_t)cap + 3) / 4 * 4, words = 3 * R + 2;
  const bool apart = 12 * c4 > 64 * 1024;
  const at::Tensor buf = at::empty({3 * c4 + (apart ? 0 : words)}, ctx->options());
  const at::Tensor state = apart ? at::empty({words}, ctx->options()) : buf;
  auto part = [](const at::Tensor& b, int64_t at, int64_t n) { return cut(b, at, {n}, at::kInt); };
  const int64_t s0 = apart ? 0 : 3 * c4;
  const at::Tensor req = part(buf, 0, cap), pos = part(buf, c4, cap), slot = part(buf, 2 * c4, cap),
                   cu = part(state, s0, R + 1), co = part(state, s0 + R + 1, R), ho = part(state, s0 + 2 * R + 1, R),
                   uo = part(state, s0 + 3 * R + 1, 1);
  const dsa_status s = call(batch_layout_fn, ptr<int32_t>(ctx), ptr<int32_t>(nw), ptr<int32_t>(held), (int32_t)R,
                                       ptr<int32_t>(table), (int32_t)table->size(1), ptr<int32_t>(free),
                                       (int32_t)free->size(0), ptr<int32_t>(used), page, pages, cap, ptr<int32_t>(&cu),
                                       ptr<int32_t>(&req), ptr<int32_t>(&pos), ptr<int32_t>(&slot), ptr<int32_t>(&co),
                                       ptr<int32_t>(&ho), ptr<int32_t>(&uo), st, a.stream());
  if (s != DSA_OK) return PyLong_FromLong(s);
  return tuple_of({&cu, &req, &pos, &slot, &co, &ho, &uo});
  END_HANDLE_TH_ERRORS
}

// (q, k, pos, cos_sin, d_rope, q_weight, k_weight, eps, interleaved, slot, kv, kv_scale, dev_status)
PyObject* qk_norm_rope(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  HANDLE_TH_ERRORS
  if (argc != 13) Py_RETURN_NONE;
  Args a{argv};
  auto rows = [&a]() -> const at::Tensor* {
    const at::Tensor* t = a.any();
    if (t && ((t->scalar_type() != at::kBFloat16 && t->scalar_type() != at::kHalf) || !a.placed(*t, 3) ||
              (t->size(2) > 1 && t->stride(2) != 1)))
      a.good = false;
    return t;
  };
  const at::Tensor* q = rows();
  const at::Tensor* k = rows();
  const at::Tensor* pos = a.tensor(at::kInt, 1, true);
  const at::Tensor* cs = a.tensor(at::kFloat, 2, true);
  const int32_t rope = a.int32();
  const at::Tensor* qw = a.tensor(at::kFloat, 1, true);
  const at::Tensor* kw = a.tensor(at::kFloat, 1, true);
  const float eps = a.number();
  const int inter = PyObject_IsTrue(a.next());
  const at::Tensor* slot = a.tensor(at::kInt, 1, true);
  const at::Tensor* kv = a.tensor(at::kByte, 2, true);
  const at::Tensor* sc = a.tensor(at::kFloat, 1, true);
  int32_t* st = a.status();
  const at::Tensor* x = q ? q : k;
  if (!a.good || !x || inter < 0) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  const int64_t n = x->size(0), d = x->size(2);
  const bool cache = slot || kv || sc;
  if ((q && k && (k->size(0) != n || k->size(2) != d || k->scalar_type() != q->scalar_type())) ||
      (rope != 0 && (!pos || !cs || cs->size(1) != rope)) || (pos && pos->size(0) != n) || !fits32(n) || !fits32(d) ||
      (q && !fits32(q->size(1))) || (k && !fits32(k->size(1))) || (cs && !fits32(cs->size(0))))
    Py_RETURN_NONE;
  if (cache && (!k || !slot || !kv || !sc || slot->size(0) != n || kv->size(1) != d || sc->size(0) != kv->size(0)))
    Py_RETURN_NONE;
  at::Tensor qo, ko;
  if (q) qo = at::empty(q->sizes(), x->options());
  if (k && !cache) ko = at::empty(k->sizes(), x->options());
  const dsa_status s = call(
      qk_norm_rope_fn, ptr<void>(q), stride(q, 0), stride(q, 1), q ? (int32_t)q->size(1) : 0, ptr<float>(qw),
      qw ? (int32_t)qw->size(0) : 0, q ? qo.data_ptr() : nullptr, ptr<void>(k), stride(k, 0),
      stride(k, 1), k ? (int32_t)k->size(1) : 0, ptr<float>(kw), kw ? (int32_t)kw->size(0) : 0,
      k && !cache ? ko.data_ptr() : nullptr, (int32_t)n, (int32_t)d, rope,
      x->scalar_type() == at::kHalf ? DSA_FP16 : DSA_BF16, ptr<int32_t>(pos), ptr<float>(cs),
      cs ? (int32_t)cs->size(0) : 0, eps, inter, ptr<int32_t>(slot), ptr<uint8_t>(kv), ptr<float>(sc),
      cache ? kv->size(0) : 0, st, a.stream());
  if (s != DSA_OK) return PyLong_FromLong(s);
  return tuple_of({q ? &qo : nullptr, k && !cache ? &ko : nullptr});
  END_HANDLE_TH_ERRORS
}

// (q, kv, kv_scale, block_table, q_req, q_pos, d_latent, d_rope, page_size, softmax_scale, max_ctx, num_splits
// (0: by the rule), dev_status)
PyObject* chunk_mla(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  HANDLE_TH_ERRORS
  if (argc != 13) Py_RETURN_NONE;
  Args a{argv};
  const at::Tensor* q = a.tensor(at::kBFloat16, 3);
  const at::Tensor* kv = a.tensor(at::kByte, 2);
  const at::Tensor* sc = a.tensor(at::kFloat, 1);
  const at::Tensor* bt = a.tensor(at::kInt, 2);
  const at::Tensor* req = a.tensor(at::kInt, 1);
  const at::Tensor* pos = a.tensor(at::kInt, 1);
  const int32_t dl = a.int32(), dr = a.int32(), page = a.int32();
  const float scale = a.number();
  const int64_t ctx = a.integer();
  int32_t S = a.int32();
  int32_t* st = a.status();
  if (!a.good || page <= 0) Py_RETURN_NONE;
  const int64_t n = q->size(0), H = q->size(1), slots = kv->size(0);
  if (q->size(2) != (int64_t)dl + dr || kv->size(1) != q->size(2) || slots % page != 0 || req->size(0) != n ||
      pos->size(0) != n || sc->size(0) != slots || n == 0 || !fits32(n) || !fits32(H) || !fits32(bt->size(0)) ||
      !fits32(bt->size(1)) || dl <= 0)
    Py_RETURN_NONE;
  if (S == 0)
    S = pick_fn((int32_t)n, (int32_t)H, dl, dr, (int32_t)std::min<int64_t>(std::max<int64_t>(ctx, 1), INT32_MAX), 0);
  if (S < 1 || S > 64) Py_RETURN_NONE;
  // out, then lse; the partials of a split call in a buffer of their own
  const int64_t ob = (2 * n * H * dl + 15) / 16 * 16;
  const at::Tensor buf = bytes(ob + 4 * n * H, *q);
  const at::Tensor out = cut(buf, 0, {n, H, dl}, at::kBFloat16), lse = cut(buf, ob / 4, {n, H}, at::kFloat);
  at::Tensor parts;
  float *op = nullptr, *lp = nullptr;
  if (S > 8) {  // (fewer are merged by the call)
    const int64_t pn = ((int64_t)S * n * H * dl + 3) / 4 * 4;
    parts = at::empty({pn + (int64_t)S * n * H}, sc->options());
    op = ptr<float>(&parts);
    lp = op + pn;
  }
  void* stream = a.stream();
  dsa_status s = call(chunk_mla_fn, q->data_ptr(), ptr<uint8_t>(kv), ptr<float>(sc), slots / page, ptr<int32_t>(bt),
                              (int32_t)bt->size(0), (int32_t)bt->size(1), ptr<int32_t>(req), ptr<int32_t>(pos),
                              (int32_t)n, (int32_t)H, dl, dr, page, scale, S, op ? nullptr : out.data_ptr(),
                              op ? nullptr : ptr<float>(&lse), op, lp, st, stream);
  if (s == DSA_OK && op)
    s = call(combine_fn, op, lp, S, (int32_t)n, (int32_t)H, dl, out.data_ptr(), ptr<float>(&lse), stream);
  if (s != DSA_OK) return PyLong_FromLong(s);
  return tuple_of({&out, &lse});
  END_HANDLE_TH_ERRORS
}

// (target_probs, draft_tokens, cu_rows, u_accept, u_sample, draft_probs, ctx_len, q_req, max_out, dev_status)
PyObject* verify_draft(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  HANDLE_TH_ERRORS
  if (argc != 10) Py_RETURN_NONE;
  Args a{argv};
  auto probs = [&a]() -> const at::Tensor* {
    const at::Tensor* t = a.any();
    if (t && (t->scalar_type() != at::kFloat || !a.placed(*t, 2) || (t->size(1) > 1 && t->stride(1) != 1) ||
              (t->size(0) > 1 && t->stride(0) < t->size(1))))
      a.good = false;
    return t;
  };
  const at::Tensor* p = probs();
  const at::Tensor* tok = a.tensor(at::kInt, 1);
  const at::Tensor* cu = a.tensor(at::kInt, 1);
  const at::Tensor* ua = a.tensor(at::kFloat, 1);
  const at::Tensor* us = a.tensor(at::kFloat, 1);
  const at::Tensor* q = probs();
  const at::Tensor* ctx = a.tensor(at::kInt, 1, true);
  const at::Tensor* own = a.tensor(at::kInt, 1, true);
  const int32_t max_out = a.int32();
  int32_t* st = a.status();
  if (!a.good || !p || max_out < 1) Py_RETURN_NONE;
  const int64_t rows = p->size(0), V = p->size(1), R = us->size(0);
  if (cu->size(0) != R + 1 || tok->size(0) != rows || ua->size(0) != rows || (q && q->sizes() != p->sizes()) ||
      (ctx && ctx->size(0) != R) || (own && own->size(0) < rows) || !fits32(rows) || !fits32(V) || !fits32(R))
    Py_RETURN_NONE;
  const at::Tensor buf = at::empty({R * max_out + (ctx ? 2 : 1) * R}, cu->options());
  const at::Tensor tokens = cut(buf, 0, {R, max_out}, at::kInt), num = cut(buf, R * max_out, {R}, at::kInt);
  at::Tensor co;
  if (ctx) co = cut(buf, R * max_out + R, {R}, at::kInt);
  const dsa_status s = call(verify_draft_fn, ptr<float>(p), rows > 1 ? p->stride(0) : V, (int32_t)rows, (int32_t)V,
                                       ptr<float>(q), q && rows > 1 ? q->stride(0) : V, ptr<int32_t>(tok),
                                       ptr<float>(ua), ptr<float>(us), ptr<int32_t>(cu), ptr<int32_t>(own), (int32_t)R, max_out,
                                       ptr<int32_t>(ctx), ptr<int32_t>(&tokens), ptr<int32_t>(&num),
                                       ctx ? ptr<int32_t>(&co) : nullptr, st, a.stream());
  if (s != DSA_OK) return PyLong_FromLong(s);
  return tuple_of({&tokens, &num, ctx ? &co : nullptr});
  END_HANDLE_TH_ERRORS
}

// bind(batch_layout, qk_norm_rope, chunk_mla_fwd, combine, chunk_pick_num_splits, verify_draft_req): the entry points' addresses
PyObject* bind(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  if (argc != 6) {
    PyErr_SetString(PyExc_TypeError, "bind takes 6 addresses");
    return nullptr;
  }
  void* p[6];
  for (int i = 0; i < 6; ++i) {
    p[i] = PyLong_AsVoidPtr(argv[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  batch_layout_fn = reinterpret_cast<decltype(batch_layout_fn)>(p[0]);
  qk_norm_rope_fn = reinterpret_cast<decltype(qk_norm_rope_fn)>(p[1]);
  chunk_mla_fn = reinterpret_cast<decltype(chunk_mla_fn)>(p[2]);
  combine_fn = reinterpret_cast<decltype(combine_fn)>(p[3]);
  pick_fn = reinterpret_cast<decltype(pick_fn)>(p[4]);
  verify_draft_fn = reinterpret_cast<decltype(verify_draft_fn)>(p[5]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<batch_layout>("batch_layout"), method<qk_norm_rope>("qk_norm_rope"),
                         method<chunk_mla>("chunk_mla"),       method<verify_draft>("verify_draft"),
                         method<bind>("bind"),                 {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() {
  PyObject* m = PyModule_Create(&module_def);
  // the signatures that the addresses given to bind() are called with
  if (m && PyModule_AddIntConstant(m, "header_version", DSA_VERSION) != 0) Py_CLEAR(m);
  return m;
}
