// fast_call.cpp — the layer operators' argument checks and packing in compiled
// code.  A decode step makes these calls dozens of times, and what Python spends on
// looking at a dozen tensors (4 to 7 us) is longer than the kernels of a small
// batch.  Each function takes the arguments of the binding's function of the same
// operator, applies the same checks, fills the C struct and calls the C entry;
// whatever it does not find in order it leaves to the Python form (returns -1),
// which names what is wrong.

#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cfloat>
#include <cmath>
#include <initializer_list>

#include "moe.h"

namespace {

using NormFn = moe_status_t (*)(const moe_norm_t*, void*);
using RopeFn = moe_status_t (*)(const moe_kv_cache_t*, const moe_rope_t*, void*, size_t, void*);
using AttnFn = moe_status_t (*)(const moe_kv_cache_t*, const moe_attention_t*, void*, size_t, void*);
using QuantFn = moe_status_t (*)(const moe_quant_t*, void*);
using LinearFn = moe_status_t (*)(const moe_linear_t*, void*, size_t, void*);
using SampleFn = moe_status_t (*)(const moe_sampling_t*, void*);
QuantFn quant_entry = nullptr;
LinearFn linear_entry = nullptr;
SampleFn sample_entry = nullptr;
NormFn norm_entry = nullptr;
RopeFn rope_entry = nullptr;
AttnFn attn_entry = nullptr;

PyObject* leave_it() {
  PyErr_Clear();
  return PyLong_FromLong(-1);
}

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// A tensor of these sizes, type and device with contiguous rows.
bool rows(const at::Tensor* t, std::initializer_list<int64_t> sizes, at::ScalarType dtype, int dev) {
  if (!t || !t->is_cuda() || t->get_device() != dev || t->scalar_type() != dtype || t->layout() != at::kStrided ||
      t->dim() != static_cast<int64_t>(sizes.size()))
    return false;
  int i = 0;
  for (int64_t s : sizes)
    if (t->size(i++) != s) return false;
  return t->stride(-1) == 1 || t->size(-1) <= 1;
}
bool flat(const at::Tensor* t, std::initializer_list<int64_t> sizes, at::ScalarType dtype, int dev) {
  return rows(t, sizes, dtype, dev) && t->is_contiguous();
}

// A workspace: elements one after the other (an expanded tensor counts more than it has).
bool workspace(const at::Tensor& t, int dev) {
  return t.is_cuda() && t.get_device() == dev && t.layout() == at::kStrided && t.is_contiguous();
}

int float_code(at::ScalarType t) {
  return t == at::kHalf ? MOE_F16 : t == at::kBFloat16 ? MOE_BF16 : 0;
}

// The stream to launch on: the device's current one, a stream object or a number.
bool stream_of(PyObject* o, int dev, void** st) {
  if (dev != c10::cuda::current_device()) return false;
  if (o == Py_None) {
    *st = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    return true;
  }
  PyObject* n = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
  if (!n) return false;
  *st = PyLong_AsVoidPtr(n);
  Py_DECREF(n);
  return !PyErr_Occurred();
}

const moe_kv_cache_t* cache_of(PyObject* o) {
  return PyBytes_Check(o) && PyBytes_GET_SIZE(o) == static_cast<Py_ssize_t>(sizeof(moe_kv_cache_t))
             ? reinterpret_cast<const moe_kv_cache_t*>(PyBytes_AS_STRING(o))
             : nullptr;
}

constexpr int64_t kIntMax = 0x7fffffff;

// Whether a number is one in fp32 too.
bool fits(double v) { return !std::isfinite(v) || std::fabs(v) <= FLT_MAX; }

// norm(x, weight, out, residual, residual_out, scales, group, eps, stream)
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const at::Tensor *x, *w, *out, *r = nullptr, *ro = nullptr, *sc = nullptr;
  if (n != 9 || !norm_entry || !(x = tensor(a[0])) || !(w = tensor(a[1])) || !(out = tensor(a[2]))) return leave_it();
  const long group = PyLong_AsLong(a[6]);
  const double eps = PyFloat_AsDouble(a[7]);
  if (PyErr_Occurred() || !fits(eps) || !x->is_cuda() || x->dim() != 2 || group < 0 || group > 65536) return leave_it();
  const int dev = x->get_device();
  const int64_t T = x->size(0), H = x->size(1);
  const at::ScalarType dt = x->scalar_type();
  const int code = float_code(dt);
  const bool e4m3 = out->scalar_type() == at::kFloat8_e4m3fn;
  if (!code || T > kIntMax || H > kIntMax || !rows(x, {T, H}, dt, dev) || !rows(w, {H}, dt, dev) ||
      !rows(out, {T, H}, e4m3 ? at::kFloat8_e4m3fn : dt, dev))
    return leave_it();
  if (a[3] != Py_None && !rows(r = tensor(a[3]), {T, H}, dt, dev)) return leave_it();
  if (a[4] != Py_None && (!r || !rows(ro = tensor(a[4]), {T, H}, dt, dev))) return leave_it();
  if ((a[5] != Py_None) != e4m3) return leave_it();
  if (e4m3 && !flat(sc = tensor(a[5]), {T, group ? (H + group - 1) / group : 1}, at::kFloat, dev)) return leave_it();
  moe_norm_t m;
  m.x = x->data_ptr();
  m.residual = r ? r->data_ptr() : nullptr;
  m.weight = w->data_ptr();
  m.out = out->data_ptr();
  m.residual_out = ro ? ro->data_ptr() : nullptr;
  m.scales = sc ? static_cast<float*>(sc->data_ptr()) : nullptr;
  const bool one = T == 1;  // a single row's stride says nothing
  m.x_stride = one ? H : x->stride(0);
  m.residual_stride = !r ? 0 : one ? H : r->stride(0);
  m.out_stride = one ? H : out->stride(0);
  m.residual_out_stride = !ro ? 0 : one ? H : ro->stride(0);
  m.T = static_cast<int32_t>(T);
  m.H = static_cast<int32_t>(H);
  m.dtype = code;
  m.out_dtype = e4m3 ? MOE_E4M3 : code;
  m.group = static_cast<int32_t>(group);
  m.eps = static_cast<float>(eps);
  void* st;
  if (!stream_of(a[8], dev, &st)) return leave_it();
  return PyLong_FromLong(norm_entry(&m, st));
}

// rope(cache, cache device, q, k, v, positions, slots, inv_freq, q_out, ws, q_norm_w, k_norm_w, eps, interleaved, stream)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 15 || !rope_entry) return leave_it();
  const moe_kv_cache_t* c = cache_of(a[0]);
  const at::Tensor* t[8];  // q k v positions slots inv_freq q_out ws
  for (int i = 0; i < 8; ++i)
    if (!(t[i] = tensor(a[2 + i]))) return leave_it();
  const at::Tensor &q = *t[0], &ws = *t[7], *qn = nullptr, *kn = nullptr;
  const long cache_dev = PyLong_AsLong(a[1]);
  const double eps = PyFloat_AsDouble(a[12]);
  const int inter = PyObject_IsTrue(a[13]);
  if (PyErr_Occurred() || !fits(eps) || !c || !q.is_cuda() || q.dim() != 3) return leave_it();
  const int dev = q.get_device();
  const int64_t T = q.size(0), hq = q.size(1), D = c->head_dim, hkv = c->n_kv_heads, nf = t[5]->numel();
  const at::ScalarType dt = q.scalar_type();
  const int code = float_code(dt);
  if (!code || cache_dev != dev || !workspace(ws, dev) || T > kIntMax || hq > kIntMax ||
      nf > kIntMax / 2 || !rows(&q, {T, hq, D}, dt, dev) || !rows(t[1], {T, hkv, D}, dt, dev) ||
      !rows(t[2], {T, hkv, D}, dt, dev) || !flat(t[3], {T}, at::kLong, dev) || !flat(t[4], {T}, at::kLong, dev) ||
      !flat(t[5], {nf}, at::kFloat, dev) || !rows(t[6], {T, hq, D}, dt, dev))
    return leave_it();
  if (a[10] != Py_None || a[11] != Py_None)
    if (!flat(qn = tensor(a[10]), {D}, dt, dev) || !flat(kn = tensor(a[11]), {D}, dt, dev)) return leave_it();
  moe_rope_t m;
  m.q = q.data_ptr();
  m.k = t[1]->data_ptr();
  m.v = t[2]->data_ptr();
  m.q_out = t[6]->data_ptr();
  m.positions = static_cast<const int64_t*>(t[3]->data_ptr());
  m.slots = static_cast<const int64_t*>(t[4]->data_ptr());
  m.inv_freq = static_cast<const float*>(t[5]->data_ptr());
  m.q_norm_w = qn ? qn->data_ptr() : nullptr;
  m.k_norm_w = kn ? kn->data_ptr() : nullptr;
  m.q_token_stride = q.stride(0);
  m.q_head_stride = q.stride(1);
  m.k_token_stride = t[1]->stride(0);
  m.k_head_stride = t[1]->stride(1);
  m.v_token_stride = t[2]->stride(0);
  m.v_head_stride = t[2]->stride(1);
  m.out_token_stride = t[6]->stride(0);
  m.out_head_stride = t[6]->stride(1);
  m.T = static_cast<int32_t>(T);
  m.n_q_heads = static_cast<int32_t>(hq);
  m.rot_dim = static_cast<int32_t>(2 * nf);
  m.dtype = code;
  m.interleaved = inter ? 1 : 0;
  m.eps = static_cast<float>(eps);
  void* st;
  if (!stream_of(a[14], dev, &st)) return leave_it();
  return PyLong_FromLong(rope_entry(c, &m, ws.data_ptr(), ws.nbytes(), st));
}

// attention(cache, cache device, q, block_table, seq_lens, out, ws, scale, window, lse, stream)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 11 || !attn_entry) return leave_it();
  const moe_kv_cache_t* c = cache_of(a[0]);
  const at::Tensor *q = tensor(a[2]), *table = tensor(a[3]), *lens = tensor(a[4]), *out = tensor(a[5]),
                   *ws = tensor(a[6]), *lse = nullptr;
  if (!c || !q || !table || !lens || !out || !ws || !q->is_cuda() || q->dim() != 3 || table->dim() != 2)
    return leave_it();
  const long cache_dev = PyLong_AsLong(a[1]), window = PyLong_AsLong(a[8]);
  const int dev = q->get_device();
  const int64_t B = q->size(0), hq = q->size(1), D = c->head_dim, pages = table->size(1);
  const at::ScalarType dt = q->scalar_type();
  const int code = float_code(dt);
  if (PyErr_Occurred() || !code || cache_dev != dev || !workspace(*ws, dev) || B > kIntMax ||
      hq > kIntMax || pages > kIntMax || window < 0 || window > kIntMax || !rows(q, {B, hq, D}, dt, dev) ||
      !rows(out, {B, hq, D}, dt, dev) || !rows(table, {B, pages}, at::kInt, dev) || !flat(lens, {B}, at::kInt, dev))
    return leave_it();
  if (a[9] != Py_None && !flat(lse = tensor(a[9]), {B, hq}, at::kFloat, dev)) return leave_it();
  moe_attention_t m;
  m.q = q->data_ptr();
  m.out = out->data_ptr();
  m.lse = lse ? static_cast<float*>(lse->data_ptr()) : nullptr;
  m.block_table = static_cast<const int32_t*>(table->data_ptr());
  m.seq_lens = static_cast<const int32_t*>(lens->data_ptr());
  m.q_seq_stride = q->stride(0);
  m.q_head_stride = q->stride(1);
  m.out_seq_stride = out->stride(0);
  m.out_head_stride = out->stride(1);
  m.table_stride = table->stride(0);
  m.B = static_cast<int32_t>(B);
  m.n_q_heads = static_cast<int32_t>(hq);
  m.max_pages = static_cast<int32_t>(pages);
  m.window = static_cast<int32_t>(window);
  m.dtype = code;
  const double scale = a[7] == Py_None ? 1.0 / std::sqrt(static_cast<double>(D)) : PyFloat_AsDouble(a[7]);
  if (PyErr_Occurred() || !fits(scale)) return leave_it();
  m.scale = static_cast<float>(scale);
  void* st;
  if (!stream_of(a[10], dev, &st)) return leave_it();
  return PyLong_FromLong(attn_entry(c, &m, ws->data_ptr(), ws->nbytes(), st));
}

// quant(x, out, scales, rows, stream)
PyObject* quant(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const at::Tensor *x, *out, *sc;
  if (n != 5 || !quant_entry || !(x = tensor(a[0])) || !(out = tensor(a[1])) || !(sc = tensor(a[2]))) return leave_it();
  const long rows_of = PyLong_AsLong(a[3]);
  if (PyErr_Occurred() || !x->is_cuda() || x->dim() != 2 || (rows_of != 1 && rows_of != 128)) return leave_it();
  const int dev = x->get_device();
  const int64_t T = x->size(0), H = x->size(1);
  const at::ScalarType dt = x->scalar_type();
  const int code = float_code(dt);
  if (!code || T > kIntMax || H > kIntMax || !rows(x, {T, H}, dt, dev) || !rows(out, {T, H}, at::kFloat8_e4m3fn, dev) ||
      !flat(sc, {(T + rows_of - 1) / rows_of, (H + 127) / 128}, at::kFloat, dev))
    return leave_it();
  moe_quant_t m;
  m.x = x->data_ptr();
  m.out = out->data_ptr();
  m.scales = static_cast<float*>(sc->data_ptr());
  m.x_stride = x->stride(0);
  m.out_stride = out->stride(0);
  m.T = static_cast<int32_t>(T);
  m.H = static_cast<int32_t>(H);
  m.rows = static_cast<int32_t>(rows_of);
  m.dtype = code;
  void* st;
  if (!stream_of(a[4], dev, &st)) return leave_it();
  return PyLong_FromLong(quant_entry(&m, st));
}

// linear(x, x_scales, w, w_scales, out, ws, stream)
PyObject* linear(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const at::Tensor* t[6];
  if (n != 7 || !linear_entry) return leave_it();
  for (int i = 0; i < 6; ++i)
    if (!(t[i] = tensor(a[i]))) return leave_it();
  const at::Tensor &x = *t[0], &w = *t[2], &out = *t[4], &ws = *t[5];
  if (!x.is_cuda() || x.dim() != 2 || w.dim() != 2) return leave_it();
  const int dev = x.get_device();
  const int64_t M = x.size(0), K = x.size(1), N = w.size(0), kb = (K + 127) / 128;
  const at::ScalarType dt = out.scalar_type();
  const int code = dt == at::kFloat ? MOE_F32 : float_code(dt);
  if (!code || M > kIntMax || N > kIntMax || K > kIntMax || !rows(&x, {M, K}, at::kFloat8_e4m3fn, dev) ||
      !flat(t[1], {M, kb}, at::kFloat, dev) || !rows(&w, {N, K}, at::kFloat8_e4m3fn, dev) ||
      !flat(t[3], {(N + 127) / 128, kb}, at::kFloat, dev) || !rows(&out, {M, N}, dt, dev) || !workspace(ws, dev))
    return leave_it();
  moe_linear_t m;
  m.x = x.data_ptr();
  m.x_scales = static_cast<const float*>(t[1]->data_ptr());
  m.w = w.data_ptr();
  m.w_scales = static_cast<const float*>(t[3]->data_ptr());
  m.out = out.data_ptr();
  m.x_stride = x.stride(0);
  m.w_stride = w.stride(0);
  m.out_stride = out.stride(0);
  m.M = static_cast<int32_t>(M);
  m.N = static_cast<int32_t>(N);
  m.K = static_cast<int32_t>(K);
  m.out_dtype = code;
  void* st;
  if (!stream_of(a[6], dev, &st)) return leave_it();
  return PyLong_FromLong(linear_entry(&m, ws.data_ptr(), ws.nbytes(), st));
}

// sample(logits, uniforms, tokens, temperature, top_k, top_p, min_p, logprobs, stream)
PyObject* sample(PyObject*, PyObject* const* a, Py_ssize_t n) {
  const at::Tensor *l, *u, *tok;
  if (n != 9 || !sample_entry || !(l = tensor(a[0])) || !(u = tensor(a[1])) || !(tok = tensor(a[2])) || !l->is_cuda() ||
      l->dim() != 2)
    return leave_it();
  const int dev = l->get_device();
  const int64_t B = l->size(0), V = l->size(1);
  const at::ScalarType dt = l->scalar_type();
  const int code = dt == at::kFloat ? MOE_F32 : float_code(dt);
  if (!code || !V || B > kIntMax || V > kIntMax || !rows(l, {B, V}, dt, dev) || !flat(u, {B}, at::kFloat, dev) ||
      !flat(tok, {B}, at::kLong, dev))
    return leave_it();
  void* p[5];  // temperature top_k top_p min_p logprobs
  for (int i = 0; i < 5; ++i) {
    p[i] = nullptr;
    if (a[3 + i] == Py_None) continue;
    const at::Tensor* t = tensor(a[3 + i]);
    if (!flat(t, {B}, i == 1 ? at::kInt : at::kFloat, dev)) return leave_it();
    p[i] = t->data_ptr();
  }
  moe_sampling_t m;
  m.logits = l->data_ptr();
  m.uniforms = static_cast<const float*>(u->data_ptr());
  m.temperature = static_cast<const float*>(p[0]);
  m.top_k = static_cast<const int32_t*>(p[1]);
  m.top_p = static_cast<const float*>(p[2]);
  m.min_p = static_cast<const float*>(p[3]);
  m.tokens = static_cast<int64_t*>(tok->data_ptr());
  m.logprobs = static_cast<float*>(p[4]);
  m.logits_stride = l->stride(0);
  m.B = static_cast<int32_t>(B);
  m.V = static_cast<int32_t>(V);
  m.dtype = code;
  void* st;
  if (!stream_of(a[8], dev, &st)) return leave_it();
  return PyLong_FromLong(sample_entry(&m, st));
}

// bind_projections(moe_quantize_e4m3, moe_linear_e4m3, moe_sample, sizes of moe_quant_t, moe_linear_t,
// moe_sampling_t): as bind().
PyObject* bind_projections(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "three addresses and three sizes expected");
    return nullptr;
  }
  void* entries[3];
  for (int i = 0; i < 3; ++i) entries[i] = PyLong_AsVoidPtr(a[i]);
  const size_t sizes[3] = {sizeof(moe_quant_t), sizeof(moe_linear_t), sizeof(moe_sampling_t)};
  bool same = true;
  for (int i = 0; i < 3; ++i) same &= PyLong_AsSize_t(a[3 + i]) == sizes[i];
  if (PyErr_Occurred()) return nullptr;
  if (!same) Py_RETURN_FALSE;
  quant_entry = reinterpret_cast<QuantFn>(entries[0]);
  linear_entry = reinterpret_cast<LinearFn>(entries[1]);
  sample_entry = reinterpret_cast<SampleFn>(entries[2]);
  Py_RETURN_TRUE;
}

// bind(moe_add_rmsnorm, moe_rope_append, moe_paged_attention: the loaded library's entries,
// sizes of moe_norm_t, moe_kv_cache_t, moe_rope_t, moe_attention_t): False, and nothing
// bound, where the structs compiled here are others.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "three addresses and four sizes expected");
    return nullptr;
  }
  void* entries[3];
  for (int i = 0; i < 3; ++i) entries[i] = PyLong_AsVoidPtr(a[i]);
  const size_t sizes[4] = {sizeof(moe_norm_t), sizeof(moe_kv_cache_t), sizeof(moe_rope_t), sizeof(moe_attention_t)};
  bool same = true;
  for (int i = 0; i < 4; ++i) same &= PyLong_AsSize_t(a[3 + i]) == sizes[i];
  if (PyErr_Occurred()) return nullptr;
  if (!same) Py_RETURN_FALSE;
  norm_entry = reinterpret_cast<NormFn>(entries[0]);
  rope_entry = reinterpret_cast<RopeFn>(entries[1]);
  attn_entry = reinterpret_cast<AttnFn>(entries[2]);
  Py_RETURN_TRUE;
}

// C++ exceptions (of torch's accessors) end here.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  try {
    return F(self, a, n);
  } catch (...) {
    return leave_it();
  }
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<norm>("norm"), method<rope>("rope"), method<attention>("attention"),
                         method<bind>("bind"), method<quant>("quant"), method<linear>("linear"),
                         method<sample>("sample"), method<bind_projections>("bind_projections"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast_call", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast_call() {
  PyObject* mod = PyModule_Create(&module);
  // The tensor class is compiled in: the binding uses this module with that PyTorch only.
  if (mod && PyModule_AddStringConstant(mod, "built_for", MOE_TORCH_VERSION) < 0) Py_CLEAR(mod);
  return mod;
}
