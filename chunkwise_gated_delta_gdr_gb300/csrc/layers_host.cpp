// layers_host.cpp -- the calls of layers.py for the ordinary case, in one step from torch
// tensors to the C ABI.
//
// A decoder makes a few such calls per layer for a few microseconds of GPU work each, and
// reading a tensor's attributes one by one from Python costs more than that. Each function
// here takes the arguments of its namesake in layers.py (without `stream`: torch's current
// one), checks everything the namesake checks, allocates the results that were not passed
// and makes the call. Where anything is out of the ordinary before that call (a wrong argument,
// an allocation that fails) it returns None, and layers.py goes its own way, with its messages.
// Once the call is made it is not made again: a status other than GDR_OK is returned, an int.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>

#include "gdr.h"

namespace {

using at::Tensor;

// A call's running verdict: every check is ANDed in, nothing is launched unless all held.
struct Call {
  bool ok = true;
  int device = -1;
  void need(bool c) { ok = ok && c; }

  // The tensor behind o; null for None (if allowed) and, with ok cleared, for anything else.
  const Tensor* get(PyObject* o, bool optional = false) {
    if (o == Py_None) {
      need(optional);
      return nullptr;
    }
    if (!THPVariable_Check(o)) {
      need(false);
      return nullptr;
    }
    const Tensor* t = &THPVariable_Unpack(o);
    if (!t->is_cuda()) {
      need(false);
      return nullptr;
    }
    const int d = t->get_device();
    if (device < 0) device = d;
    need(d == device);
    return t;
  }
  static int code(const Tensor* t) {
    const auto s = t->scalar_type();
    return s == at::kBFloat16 ? GDR_BF16 : s == at::kFloat ? GDR_F32 : -1;
  }
  int float_code(const Tensor* t) {
    const int c = t ? code(t) : -1;
    need(c >= 0);
    return c;
  }
  bool shaped(const Tensor* t, at::IntArrayRef shape) { return t && t->sizes() == shape; }
  // A view: this shape, the last dimension dense.
  void view(const Tensor* t, at::IntArrayRef shape) {
    need(shaped(t, shape) && (t->stride(-1) == 1 || shape.back() == 1));
  }
  // A dense tensor (or none) of this shape and type; its address.
  void* dense(const Tensor* t, at::IntArrayRef shape, at::ScalarType type = at::kFloat) {
    if (!t) return nullptr;
    need(shaped(t, shape) && t->scalar_type() == type && t->is_contiguous());
    return t->data_ptr();
  }
  bool ready() {
    if (!ok || device < 0) return false;
    c10::DeviceIndex now = -1;
    return c10::cuda::GetDevice(&now) == cudaSuccess && now == device;
  }
  gdr_stream_t stream() const {
    return reinterpret_cast<gdr_stream_t>(c10::cuda::getCurrentCUDAStream(device).stream());
  }
  Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    return at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, device), std::nullopt);
  }
};

int truth(PyObject* o, Call& c) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    c.need(false);
  }
  return v > 0;
}
double number(PyObject* o, Call& c) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    c.need(false);
  }
  return v;
}
// A size that fits the C ABI's int.
int fit(int64_t v, Call& c) {
  c.need(v >= 0 && v <= INT32_MAX);
  return (int)v;
}
// A C integer from a Python one (no floats).
int integer(PyObject* o, Call& c) {
  if (!PyLong_Check(o)) {
    c.need(false);
    return 0;
  }
  int over = 0;
  const long long v = PyLong_AsLongLongAndOverflow(o, &over);
  c.need(!over && v >= INT32_MIN && v <= INT32_MAX);
  return (int)v;
}

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }
// The object that was passed, or the new tensor, or None.
PyObject* result(PyObject* passed, const Tensor& made) {
  if (passed != Py_None) return Py_NewRef(passed);
  return made.defined() ? wrap(made) : Py_NewRef(Py_None);
}
template <typename... P>
PyObject* tuple_of(P*... items) {
  PyObject* t = PyTuple_New(sizeof...(items));
  int i = 0;
  bool good = t != nullptr;
  for (PyObject* p : {items...}) {
    if (!p) good = false;
    if (t && p) PyTuple_SET_ITEM(t, i, p);
    ++i;
  }
  if (!good) Py_CLEAR(t);
  return t;
}

PyObject* none() {                               // layers.py takes over
  if (PyErr_Occurred()) PyErr_Clear();
  Py_RETURN_NONE;
}
// What a call answers: its results, made before the call was, or its status.
PyObject* answer(PyObject* results, gdr_status status) {
  if (status == GDR_OK) return results;
  Py_XDECREF(results);
  return PyLong_FromLong(status);
}

// C++ exceptions (of an allocation) become None: layers.py then meets the same one itself.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (...) {
    return none();
  }
}

// (x, g, initial_state, gated_input, output_final_state, out, final_state, checkpoints)
PyObject* linear_scan_fwd(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  if (n != 8) Py_RETURN_NONE;
  return guarded([&]() -> PyObject* {
    Call c;
    const Tensor *x = c.get(arg[0]), *g = c.get(arg[1]), *s0 = c.get(arg[2], true);
    const Tensor *out = c.get(arg[5], true), *fin = c.get(arg[6], true);
    const Tensor* ck = c.get(arg[7], true);
    if (!c.ok || x->dim() != 3) Py_RETURN_NONE;
    const int64_t B = x->size(0), T = x->size(1), D = x->size(2);
    c.view(x, {B, T, D});
    c.view(g, {B, T, D});
    const bool want = truth(arg[4], c);
    gdr_scan_dims d = {};
    d.gated_input = truth(arg[3], c);
    d.B = fit(B, c); d.T = fit(T, c); d.D = fit(D, c);
    d.x_dtype = c.float_code(x);
    d.g_dtype = c.float_code(g);
    d.h_dtype = out ? c.float_code(out) : d.x_dtype;
    const void* ps0 = c.dense(s0, {B, D});
    void* pck = c.dense(ck, {B, (T + GDR_SCAN_CHECKPOINT - 1) / GDR_SCAN_CHECKPOINT, D});
    if (out) c.dense(out, {B, T, D}, out->scalar_type());
    c.dense(fin, {B, D});
    if (!c.ready()) Py_RETURN_NONE;
    d.x_stride_b = x->stride(0); d.x_stride_t = x->stride(1);
    d.g_stride_b = g->stride(0); d.g_stride_t = g->stride(1);
    Tensor made_out, made_fin;
    if (!out) out = &(made_out = c.empty({B, T, D}, x->scalar_type()));
    if (!fin && want) fin = &(made_fin = c.empty({B, D}, at::kFloat));
    PyObject* results = tuple_of(result(arg[5], made_out), result(arg[6], made_fin));
    if (!results) return none();
    return answer(results,
                  gdr_linear_scan_fwd(x->data_ptr(), g->data_ptr(),
                                      static_cast<const float*>(ps0), out->data_ptr(),
                                      fin ? fin->data_ptr<float>() : nullptr,
                                      static_cast<float*>(pck), &d, c.stream()));
  });
}

// (dh, x, g, checkpoints, d_final_state, gated_input, output_initial_state_grad, dx, dg,
//  d_initial_state)
PyObject* linear_scan_bwd(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  if (n != 10) Py_RETURN_NONE;
  return guarded([&]() -> PyObject* {
    Call c;
    const Tensor *dh = c.get(arg[0]), *x = c.get(arg[1]), *g = c.get(arg[2]), *ck = c.get(arg[3]);
    const Tensor *df = c.get(arg[4], true), *dx = c.get(arg[7], true), *dg = c.get(arg[8], true);
    const Tensor* d0 = c.get(arg[9], true);
    if (!c.ok || x->dim() != 3) Py_RETURN_NONE;
    const int64_t B = x->size(0), T = x->size(1), D = x->size(2);
    for (const Tensor* t : {dh, x, g}) c.view(t, {B, T, D});
    gdr_scan_dims d = {};
    d.gated_input = truth(arg[5], c);
    const bool want = truth(arg[6], c);
    d.B = fit(B, c); d.T = fit(T, c); d.D = fit(D, c);
    d.x_dtype = c.float_code(x);
    d.g_dtype = c.float_code(g);
    d.h_dtype = c.float_code(dh);
    const void* pck = c.dense(ck, {B, (T + GDR_SCAN_CHECKPOINT - 1) / GDR_SCAN_CHECKPOINT, D});
    const void* pdf = c.dense(df, {B, D});
    c.dense(dx, {B, T, D}, x->scalar_type());
    c.dense(dg, {B, T, D}, g->scalar_type());
    c.dense(d0, {B, D});
    if (!c.ready()) Py_RETURN_NONE;
    d.x_stride_b = x->stride(0); d.x_stride_t = x->stride(1);
    d.g_stride_b = g->stride(0); d.g_stride_t = g->stride(1);
    d.dh_stride_b = dh->stride(0); d.dh_stride_t = dh->stride(1);
    Tensor made_dx, made_dg, made_d0;
    if (!dx) dx = &(made_dx = c.empty({B, T, D}, x->scalar_type()));
    if (!dg) dg = &(made_dg = c.empty({B, T, D}, g->scalar_type()));
    if (!d0 && want) d0 = &(made_d0 = c.empty({B, D}, at::kFloat));
    PyObject* results =
        tuple_of(result(arg[7], made_dx), result(arg[8], made_dg), result(arg[9], made_d0));
    if (!results) return none();
    return answer(results,
                  gdr_linear_scan_bwd(dh->data_ptr(), x->data_ptr(), g->data_ptr(),
                                      static_cast<const float*>(pck),
                                      static_cast<const float*>(pdf), dx->data_ptr(),
                                      dg->data_ptr(), d0 ? d0->data_ptr<float>() : nullptr, &d,
                                      c.stream()));
  });
}

// What the three norm-and-rotation calls share, from q, k, (v), weights, cos, sin, positions.
struct Qk {
  gdr_qk_dims d = {};
  const Tensor *q, *k;
  const float *wq = nullptr, *wk = nullptr, *cos = nullptr, *sin = nullptr;
  const void* pos = nullptr;
  int64_t B = 0, T = 0, HQ = 0, HK = 0, D = 0;

  // arg: q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved
  bool read(Call& c, PyObject* const* arg, const Tensor* v) {
    q = c.get(arg[0]);
    k = c.get(arg[1]);
    const Tensor *tq = c.get(arg[2], true), *tk = c.get(arg[3], true);
    const Tensor *tc = c.get(arg[4], true), *ts = c.get(arg[5], true), *tp = c.get(arg[6], true);
    if (!c.ok || q->dim() != 4 || k->dim() != 4) return false;
    B = q->size(0); T = q->size(1); HQ = q->size(2); D = q->size(3); HK = k->size(2);
    c.view(q, {B, T, HQ, D});
    c.view(k, {B, T, HK, D});
    c.need(q->scalar_type() == k->scalar_type() && !tc == !ts && (!tc || tp));
    wq = static_cast<float*>(c.dense(tq, {D}));
    wk = static_cast<float*>(c.dense(tk, {D}));
    d.position_bits = 32;
    if (tc) {
      if (tc->dim() != 2) return false;
      cos = static_cast<float*>(c.dense(tc, tc->sizes()));
      sin = static_cast<float*>(c.dense(ts, tc->sizes()));
      d.table_rows = fit(tc->size(0), c);
      d.R = fit(2 * tc->size(1), c);
    }
    if (tp) {
      const bool wide = tp->scalar_type() == at::kLong;
      pos = c.dense(tp, {B, T}, wide ? at::kLong : at::kInt);
      d.position_bits = wide ? 64 : 32;
    }
    d.B = fit(B, c); d.T = fit(T, c); d.HQ = fit(HQ, c); d.HK = fit(HK, c); d.D = fit(D, c);
    d.in_dtype = c.float_code(q);
    d.eps = (float)number(arg[7], c);
    d.interleaved = truth(arg[8], c);
    d.q_stride_b = q->stride(0); d.q_stride_t = q->stride(1); d.q_stride_h = q->stride(2);
    d.k_stride_b = k->stride(0); d.k_stride_t = k->stride(1); d.k_stride_h = k->stride(2);
    if (v) {
      c.view(v, {B, T, HK, D});
      c.need(v->scalar_type() == q->scalar_type());
      if (!c.ok) return false;
      d.v_stride_b = v->stride(0); d.v_stride_t = v->stride(1); d.v_stride_h = v->stride(2);
    }
    return c.ok;
  }
};

// (q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved, q_out, k_out)
PyObject* qk_norm_rope(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  if (n != 11) Py_RETURN_NONE;
  return guarded([&]() -> PyObject* {
    Call c;
    Qk a;
    const Tensor *qo = c.get(arg[9], true), *ko = c.get(arg[10], true);
    if (!a.read(c, arg, nullptr)) Py_RETURN_NONE;
    const auto type = qo ? qo->scalar_type() : a.q->scalar_type();
    a.d.out_dtype = qo ? c.float_code(qo) : a.d.in_dtype;
    c.dense(qo, {a.B, a.T, a.HQ, a.D}, type);
    c.dense(ko, {a.B, a.T, a.HK, a.D}, type);
    if (!c.ready()) Py_RETURN_NONE;
    Tensor made_q, made_k;
    if (!qo) qo = &(made_q = c.empty({a.B, a.T, a.HQ, a.D}, type));
    if (!ko) ko = &(made_k = c.empty({a.B, a.T, a.HK, a.D}, type));
    PyObject* results = tuple_of(result(arg[9], made_q), result(arg[10], made_k));
    if (!results) return none();
    return answer(results,
                  gdr_qk_norm_rope(a.q->data_ptr(), a.k->data_ptr(), a.wq, a.wk, a.cos, a.sin,
                                   a.pos, qo->data_ptr(), ko->data_ptr(), &a.d, c.stream()));
  });
}

// (q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved, dq_out, dk_out, dq, dk,
//  output_weight_grads, workspace)
PyObject* qk_norm_rope_bwd(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  if (n != 15) Py_RETURN_NONE;
  return guarded([&]() -> PyObject* {
    Call c;
    Qk a;
    const Tensor *dqo = c.get(arg[9]), *dko = c.get(arg[10]);
    const Tensor *dq = c.get(arg[11], true), *dk = c.get(arg[12], true);
    const Tensor* ws = c.get(arg[14], true);
    if (!a.read(c, arg, nullptr)) Py_RETURN_NONE;
    const bool weights = truth(arg[13], c);
    a.d.out_dtype = c.float_code(dqo);
    const auto type = a.q->scalar_type();
    c.dense(dqo, {a.B, a.T, a.HQ, a.D}, dqo->scalar_type());
    c.dense(dko, {a.B, a.T, a.HK, a.D}, dqo->scalar_type());
    c.dense(dq, {a.B, a.T, a.HQ, a.D}, type);
    c.dense(dk, {a.B, a.T, a.HK, a.D}, type);
    if (ws) c.need(ws->scalar_type() == at::kByte && ws->is_contiguous());
    if (!c.ready()) Py_RETURN_NONE;
    Tensor made_dq, made_dk, made_wq, made_wk, made_ws;
    if (!dq) dq = &(made_dq = c.empty({a.B, a.T, a.HQ, a.D}, type));
    if (!dk) dk = &(made_dk = c.empty({a.B, a.T, a.HK, a.D}, type));
    if (weights) {
      made_wq = c.empty({a.D}, at::kFloat);
      made_wk = c.empty({a.D}, at::kFloat);
      if (!ws) {
        const size_t size = gdr_qk_norm_rope_bwd_workspace_size(&a.d);
        if (!size) Py_RETURN_NONE;
        ws = &(made_ws = c.empty({(int64_t)size}, at::kByte));
      }
    }
    PyObject* results = tuple_of(result(arg[11], made_dq), result(arg[12], made_dk),
                                 result(Py_None, made_wq), result(Py_None, made_wk));
    if (!results) return none();
    return answer(results,
                  gdr_qk_norm_rope_bwd(dqo->data_ptr(), dko->data_ptr(), a.q->data_ptr(),
                                       a.k->data_ptr(), a.wq, a.wk, a.cos, a.sin, a.pos,
                                       dq->data_ptr(), dk->data_ptr(),
                                       weights ? made_wq.data_ptr<float>() : nullptr,
                                       weights ? made_wk.data_ptr<float>() : nullptr, &a.d,
                                       ws ? ws->data_ptr() : nullptr, ws ? ws->numel() : 0,
                                       c.stream()));
  });
}

// k_cache, v_cache [pages, page_size, HK, D], page_table [B, max_pages].
bool read_cache(Call& c, gdr_paged_cache& p, const Tensor* kc, const Tensor* vc, const Tensor* pt,
                int64_t B) {
  if (!c.ok || kc->dim() != 4 || pt->dim() != 2) return false;
  c.view(kc, kc->sizes());
  c.view(vc, kc->sizes());
  c.need(vc->scalar_type() == kc->scalar_type() && vc->strides() == kc->strides());
  c.dense(pt, {B, pt->size(1)}, at::kInt);
  p.num_pages = fit(kc->size(0), c);
  p.page_size = fit(kc->size(1), c);
  p.HK = fit(kc->size(2), c);
  p.D = fit(kc->size(3), c);
  p.dtype = c.float_code(kc);
  p.max_pages = fit(pt->size(1), c);
  p.page_stride = kc->stride(0);
  p.token_stride = kc->stride(1);
  p.head_stride = kc->stride(2);
  return c.ok;
}

// (q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved, v, k_cache, v_cache,
//  page_table, q_out)
PyObject* qk_norm_rope_append(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  if (n != 14) Py_RETURN_NONE;
  return guarded([&]() -> PyObject* {
    Call c;
    Qk a;
    const Tensor *v = c.get(arg[9]), *kc = c.get(arg[10]), *vc = c.get(arg[11]);
    const Tensor *pt = c.get(arg[12]), *qo = c.get(arg[13], true);
    gdr_paged_cache p = {};
    if (!c.ok || !a.read(c, arg, v) || !a.pos || !read_cache(c, p, kc, vc, pt, a.B))
      Py_RETURN_NONE;
    const auto type = qo ? qo->scalar_type() : a.q->scalar_type();
    a.d.out_dtype = qo ? c.float_code(qo) : a.d.in_dtype;
    c.dense(qo, {a.B, a.T, a.HQ, a.D}, type);
    if (!c.ready()) Py_RETURN_NONE;
    Tensor made;
    if (!qo) qo = &(made = c.empty({a.B, a.T, a.HQ, a.D}, type));
    PyObject* results = result(arg[13], made);
    if (!results) return none();
    return answer(results,
                  gdr_qk_norm_rope_append(a.q->data_ptr(), a.k->data_ptr(), v->data_ptr(), a.wq,
                                          a.wk, a.cos, a.sin, a.pos, qo->data_ptr(),
                                          kc->data_ptr(), vc->data_ptr(), pt->data_ptr<int32_t>(),
                                          &a.d, &p, c.stream()));
  });
}

// (q, k_cache, v_cache, page_table, lens, scale or None, window, out, lse, workspace)
PyObject* paged_decode_attn(PyObject*, PyObject* const* arg, Py_ssize_t n) {
  if (n != 10) Py_RETURN_NONE;
  return guarded([&]() -> PyObject* {
    Call c;
    const Tensor *q = c.get(arg[0]), *kc = c.get(arg[1]), *vc = c.get(arg[2]), *pt = c.get(arg[3]);
    const Tensor *lens = c.get(arg[4]), *out = c.get(arg[7], true), *lse = c.get(arg[8], true);
    const Tensor* ws = c.get(arg[9], true);
    if (!c.ok || q->dim() != 3) Py_RETURN_NONE;
    const int64_t B = q->size(0), HQ = q->size(1), D = q->size(2);
    gdr_paged_cache p = {};
    if (!read_cache(c, p, kc, vc, pt, B)) Py_RETURN_NONE;
    c.view(q, {B, HQ, (int64_t)p.D});
    c.dense(lens, {B}, at::kInt);
    gdr_attn_dims d = {};
    d.B = fit(B, c); d.HQ = fit(HQ, c);
    d.q_dtype = c.float_code(q);
    d.out_dtype = out ? c.float_code(out) : d.q_dtype;
    d.window = integer(arg[6], c);
    d.scale = arg[5] == Py_None ? (float)(1.0 / std::sqrt((double)D)) : (float)number(arg[5], c);
    const auto type = out ? out->scalar_type() : q->scalar_type();
    c.dense(out, {B, HQ, D}, type);
    c.dense(lse, {B, HQ});
    if (ws) c.need(ws->scalar_type() == at::kByte && ws->is_contiguous());
    if (!c.ready()) Py_RETURN_NONE;
    d.q_stride_b = q->stride(0); d.q_stride_h = q->stride(1);
    Tensor made_out, made_lse, made_ws;
    if (!out) out = &(made_out = c.empty({B, HQ, D}, type));
    if (!lse) lse = &(made_lse = c.empty({B, HQ}, at::kFloat));
    if (!ws) {
      const size_t size = gdr_paged_decode_attn_workspace_size(&d, &p);
      if (!size) Py_RETURN_NONE;
      ws = &(made_ws = c.empty({(int64_t)size}, at::kByte));
    }
    PyObject* results = tuple_of(result(arg[7], made_out), result(arg[8], made_lse));
    if (!results) return none();
    return answer(results,
                  gdr_paged_decode_attn(q->data_ptr(), kc->data_ptr(), vc->data_ptr(),
                                        pt->data_ptr<int32_t>(), lens->data_ptr<int32_t>(),
                                        out->data_ptr(), lse->data_ptr<float>(), &d, &p,
                                        ws->data_ptr(), ws->numel(), c.stream()));
  });
}

#define FAST(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST(linear_scan_fwd),     FAST(linear_scan_bwd),
                         FAST(qk_norm_rope),        FAST(qk_norm_rope_bwd),
                         FAST(qk_norm_rope_append), FAST(paged_decode_attn),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layers_host", nullptr, -1, methods,
                      nullptr,               nullptr,        nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layers_host() { return PyModule_Create(&module); }
