// python_calls.cpp -- the calls of attention.h and sampling.h on PyTorch
// tensors, as a Python extension module (_build/wse_calls.so).
//
// A call at a decode step's sizes takes the GPU 3 to 15 microseconds; looking
// ten tensors over and filling the argument block in Python took the host 10 to
// 15 of its own, here it takes 1 to 2.  The functions check types, shapes,
// strides and devices, allocate the outputs and make the C call.  They return
// the outputs, or an int: -1 where an argument does not fit (the Python side
// then says which), else the call's status.
//
// PyTorch is used for the tensors' metadata and memory only.
#include <ATen/ATen.h>
#include <Python.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "attention.h"
#include "sampling.h"

namespace {

using at::Tensor;

constexpr int kDoesNotFit = -1;

PyObject* number(long v) { return PyLong_FromLong(v); }

// The arguments of a call in their order.
struct Args {
  PyObject* const* a;
  Py_ssize_t n, i = 0;
  bool bad = false;

  PyObject* next() { return i < n ? a[i++] : (bad = true, Py_None); }
  long long integer() {
    const long long v = PyLong_AsLongLong(next());
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      bad = true;
    }
    return v;
  }
  double real() {
    const double v = PyFloat_AsDouble(next());
    if (v == -1. && PyErr_Occurred()) {
      PyErr_Clear();
      bad = true;
    }
    return v;
  }
  bool truth() { return PyObject_IsTrue(next()) == 1; }
  // a tensor; with `optional` None gives an undefined one
  Tensor tensor(bool optional = false) {
    PyObject* o = next();
    if (THPVariable_Check(o)) return THPVariable_Unpack(o);
    if (!(optional && o == Py_None)) bad = true;
    return Tensor();
  }
};

int dtype_of(const Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return MOE_DTYPE_BF16;
    case at::kHalf: return MOE_DTYPE_FP16;
    default: return kDoesNotFit;
  }
}
bool on(const Tensor& t, int64_t gpu) { return t.is_cuda() && t.get_device() == gpu; }
bool plain(const Tensor& t, at::ScalarType type, int64_t n, int64_t gpu) {
  return t.dim() == 1 && t.size(0) == n && t.scalar_type() == type && on(t, gpu) && t.is_contiguous();
}
// [tokens, heads, dim], each head's values contiguous
bool heads(const Tensor& t, at::ScalarType type, int64_t tokens, int64_t n, int64_t dim, int64_t gpu) {
  return t.dim() == 3 && t.scalar_type() == type && on(t, gpu) && t.size(0) == tokens && t.size(1) == n &&
         t.size(2) == dim && t.stride(2) == 1;
}
// [pages, page_size, heads, dim], each row contiguous
bool cache(const Tensor& t, at::ScalarType type, int64_t n, int64_t dim, int64_t gpu) {
  return t.dim() == 4 && t.scalar_type() == type && on(t, gpu) && t.size(2) == n && t.size(3) == dim &&
         t.stride(3) == 1 && t.stride(2) == dim;
}
// scales of a quantised cache: [pages, heads, page_size], each head's contiguous
bool scales(const Tensor& t, const Tensor& cache, int64_t gpu) {
  return t.dim() == 3 && t.scalar_type() == at::kByte && on(t, gpu) && t.size(0) == cache.size(0) &&
         t.size(1) == cache.size(2) && t.size(2) == cache.size(1) && (t.size(2) < 2 || t.stride(2) == 1);
}
template <typename T>
T* ptr(const Tensor& t) {
  return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}
bool fits_int(int64_t v) { return v >= 0 && v <= 0x7fffffff; }

moe_cache_scales_t scales_of(const Tensor& k, const Tensor& v) {
  if (!k.defined()) return moe_cache_scales_t{};
  // the stride of a single page or head is any number
  auto stride = [](const Tensor& t, int64_t d) { return t.size(d) > 1 ? t.stride(d) : 0; };
  return moe_cache_scales_t{k.data_ptr(), v.data_ptr(), stride(k, 0), stride(k, 1), stride(v, 0), stride(v, 1)};
}

PyObject* qk_norm_rope(Args x) {
  const int64_t gpu = x.integer(), stream = x.integer(), dim = x.integer(), rotary = x.integer();
  const bool interleaved = x.truth();
  const double eps = x.real();
  const Tensor turns = x.tensor(), q = x.tensor(), k = x.tensor(), v = x.tensor();
  const Tensor qw = x.tensor(true), kw = x.tensor(true), positions = x.tensor(), slots = x.tensor();
  const Tensor k_cache = x.tensor(), v_cache = x.tensor();
  Tensor out = x.tensor(true);
  const Tensor k_scale = x.tensor(true), v_scale = x.tensor(true);
  if (x.bad || q.dim() != 3 || k.dim() != 3) return number(kDoesNotFit);
  const bool quantised = k_scale.defined();
  const auto type = q.scalar_type(), cached = quantised ? at::kFloat8_e4m3fn : type;
  const int64_t T = q.size(0), Hq = q.size(1), Hk = k.size(1);
  if (dtype_of(q) < 0 || !heads(q, type, T, Hq, dim, gpu) || !heads(k, type, T, Hk, dim, gpu) ||
      !heads(v, type, T, Hk, dim, gpu) || !cache(k_cache, cached, Hk, dim, gpu) ||
      !cache(v_cache, cached, Hk, dim, gpu) || !k_cache.sizes().equals(v_cache.sizes()) ||
      quantised != v_scale.defined() ||
      (quantised && (!scales(k_scale, k_cache, gpu) || !scales(v_scale, v_cache, gpu))) || !plain(positions, at::kInt, T, gpu) ||
      !plain(slots, at::kLong, T, gpu) || (qw.defined() && !plain(qw, type, dim, gpu)) ||
      (kw.defined() && !plain(kw, type, dim, gpu)) || (out.defined() && !heads(out, type, T, Hq, dim, gpu)) ||
      !fits_int(T) || !fits_int(Hq) || !fits_int(Hk) || !fits_int(k_cache.size(0)) || !fits_int(k_cache.size(1)))
    return number(kDoesNotFit);
  if (!out.defined()) out = at::empty({T, Hq, dim}, q.options());
  const moe_qk_norm_rope_args_t a{dtype_of(q), (int)T, (int)Hq, (int)Hk, (int)dim, (int)rotary, interleaved,
                                  (float)eps, q.data_ptr(), k.data_ptr(), v.data_ptr(), q.stride(0), q.stride(1),
                                  k.stride(0), k.stride(1), v.stride(0), v.stride(1), ptr<void>(qw), ptr<void>(kw),
                                  ptr<uint64_t>(turns), ptr<int32_t>(positions), ptr<int64_t>(slots), out.data_ptr(),
                                  out.stride(0), out.stride(1), k_cache.data_ptr(), v_cache.data_ptr(),
                                  k_cache.stride(0), k_cache.stride(1), v_cache.stride(0), v_cache.stride(1),
                                  (int)k_cache.size(0), (int)k_cache.size(1)};
  const auto on_stream = reinterpret_cast<moe_stream_t>(stream);
  const moe_cache_scales_t s = scales_of(k_scale, v_scale);
  const int status = quantised ? moe_qk_norm_rope_e4m3(&a, &s, on_stream) : moe_qk_norm_rope(&a, on_stream);
  return status == MOE_OK ? THPVariable_Wrap(std::move(out)) : number(status);
}

PyObject* attention(Args x) {
  const int64_t gpu = x.integer(), stream = x.integer(), handle = x.integer(), Hq = x.integer(), Hk = x.integer();
  const int64_t dim = x.integer();
  const Tensor q = x.tensor(), k_cache = x.tensor(), v_cache = x.tensor(), table = x.tensor(), starts = x.tensor();
  const Tensor kv_lens = x.tensor();
  const int64_t max_q = x.integer();
  const double scale = x.real();
  const Tensor tree = x.tensor(true);
  Tensor out = x.tensor(true), lse;
  const bool want_lse = x.truth();
  const Tensor k_scale = x.tensor(true), v_scale = x.tensor(true);
  const int64_t prefix = x.integer();
  if (x.bad || q.dim() != 3 || table.dim() != 2) return number(kDoesNotFit);
  const bool quantised = k_scale.defined();
  const auto type = q.scalar_type(), cached = quantised ? at::kFloat8_e4m3fn : type;
  const int64_t T = q.size(0), B = table.size(0);
  // a row's distance and its pages are two things: rows may be shared, or part of a wider table
  const int64_t row_step = B > 1 && table.size(1) > 0 ? table.stride(0) : 0;
  if (dtype_of(q) < 0 || !heads(q, type, T, Hq, dim, gpu) || !cache(k_cache, cached, Hk, dim, gpu) ||
      !cache(v_cache, cached, Hk, dim, gpu) || !k_cache.sizes().equals(v_cache.sizes()) ||
      quantised != v_scale.defined() || !fits_int(prefix) ||
      (quantised && (!scales(k_scale, k_cache, gpu) || !scales(v_scale, v_cache, gpu))) ||
      table.scalar_type() != at::kInt || !on(table, gpu) || table.stride(1) != 1 ||
      !plain(starts, at::kInt, B + 1, gpu) ||
      !plain(kv_lens, at::kInt, B, gpu) || (tree.defined() && !plain(tree, at::kLong, T, gpu)) ||
      (out.defined() && !heads(out, type, T, Hq, dim, gpu)) || !fits_int(T) || !fits_int(B) || !fits_int(max_q) ||
      !fits_int(k_cache.size(0)) || !fits_int(k_cache.size(1)) || !fits_int(row_step) || !fits_int(table.size(1)))
    return number(kDoesNotFit);
  if (!out.defined()) out = at::empty({T, Hq, dim}, q.options());
  if (want_lse) lse = at::empty({T, Hq}, q.options().dtype(at::kFloat));
  const moe_attn_args_t a{dtype_of(q), (int)B, (int)T, (int)max_q, (float)scale, q.data_ptr(), q.stride(0), q.stride(1),
                          k_cache.data_ptr(), v_cache.data_ptr(), k_cache.stride(0), k_cache.stride(1),
                          v_cache.stride(0), v_cache.stride(1), (int)k_cache.size(0), (int)k_cache.size(1),
                          ptr<int32_t>(table), (int)row_step, ptr<int32_t>(starts), ptr<int32_t>(kv_lens),
                          ptr<int64_t>(tree), out.data_ptr(), out.stride(0), out.stride(1), ptr<float>(lse),
                          (int)table.size(1)};
  auto* const h = reinterpret_cast<moe_attn_t*>(handle);
  const auto on_stream = reinterpret_cast<moe_stream_t>(stream);
  int status;
  if (quantised || prefix > 0) {
    const moe_cache_scales_t s = scales_of(k_scale, v_scale);
    moe_attn_opts_t o{quantised ? &s : nullptr, (int)prefix, nullptr, 0};
    o.workspace_bytes = moe_attn_workspace(h, &a, &o);
    Tensor workspace;  // goes back to the allocator at once, which keeps the stream's order
    if (o.workspace_bytes > 0) {
      workspace = at::empty({(int64_t)o.workspace_bytes}, q.options().dtype(at::kByte));
      o.workspace = workspace.data_ptr();
    }
    status = moe_attn_forward_ex(h, &a, &o, on_stream);
  } else {
    status = moe_attn_forward(h, &a, on_stream);
  }
  if (status != MOE_OK) return number(status);
  PyObject* o = THPVariable_Wrap(std::move(out));
  if (!want_lse || !o) return o;
  PyObject* l = THPVariable_Wrap(std::move(lse));
  return l ? Py_BuildValue("(NN)", o, l) : (Py_DECREF(o), nullptr);
}

// src and dst: int32 pages or int64 slots
PyObject* copy(Args x) {
  const int64_t stream = x.integer();
  const bool rows = x.truth();
  const Tensor k = x.tensor(), v = x.tensor(), src = x.tensor(), dst = x.tensor();
  if (x.bad || k.dim() != 5 || !k.is_cuda() || src.dim() != 1) return number(kDoesNotFit);
  const int64_t gpu = k.get_device(), n = src.size(0), row = k.size(3) * k.size(4), e = k.element_size();
  const auto type = rows ? at::kLong : at::kInt;
  if (!k.sizes().equals(v.sizes()) || k.scalar_type() != v.scalar_type() || !on(v, gpu) || !plain(src, type, n, gpu) ||
      !plain(dst, type, n, gpu) || !fits_int(n) || !fits_int(k.size(0)) || !fits_int(k.size(1)) || !fits_int(k.size(2)))
    return number(kDoesNotFit);
  for (const Tensor* t : {&k, &v})
    if (t->stride(2) != row || t->stride(3) != k.size(4) || t->stride(4) != 1) return number(kDoesNotFit);
  const auto s = reinterpret_cast<moe_stream_t>(stream);
  const int status =
      rows ? moe_copy_rows(k.data_ptr(), v.data_ptr(), (int)k.size(0), k.stride(0) * e, v.stride(0) * e,
                           k.stride(1) * e, v.stride(1) * e, (int)k.size(1), (int)k.size(2), row * e, ptr<int64_t>(src),
                           ptr<int64_t>(dst), (int)n, s)
           : moe_copy_pages(k.data_ptr(), v.data_ptr(), (int)k.size(0), k.stride(0) * e, v.stride(0) * e,
                            k.stride(1) * e, v.stride(1) * e, (int)k.size(1), k.size(2) * row * e, ptr<int32_t>(src),
                            ptr<int32_t>(dst), (int)n, s);
  return number(status);
}

PyObject* read_cache(Args x) {
  const int64_t stream = x.integer();
  const bool bf16 = x.truth();
  const Tensor k = x.tensor(), v = x.tensor(), ks = x.tensor(), vs = x.tensor(), slots = x.tensor();
  Tensor k_out = x.tensor(true), v_out = x.tensor(true);
  if (x.bad || k.dim() != 4 || !k.is_cuda() || slots.dim() != 1) return number(kDoesNotFit);
  const int64_t gpu = k.get_device(), n = slots.size(0), H = k.size(2), D = k.size(3);
  const auto type = bf16 ? at::kBFloat16 : at::kHalf;
  if (!cache(k, at::kFloat8_e4m3fn, H, D, gpu) || !cache(v, at::kFloat8_e4m3fn, H, D, gpu) ||
      !k.sizes().equals(v.sizes()) || !scales(ks, k, gpu) || !scales(vs, v, gpu) || !plain(slots, at::kLong, n, gpu) ||
      (k_out.defined() && !heads(k_out, type, n, H, D, gpu)) ||
      (v_out.defined() && !heads(v_out, type, n, H, D, gpu)) || !fits_int(n) || !fits_int(H) || !fits_int(D) ||
      !fits_int(k.size(0)) || !fits_int(k.size(1)))
    return number(kDoesNotFit);
  if (!k_out.defined()) k_out = at::empty({n, H, D}, k.options().dtype(type));
  if (!v_out.defined()) v_out = at::empty({n, H, D}, k.options().dtype(type));
  const moe_read_e4m3_args_t a{bf16 ? MOE_DTYPE_BF16 : MOE_DTYPE_FP16, (int)n, (int)H, (int)D, k.data_ptr(), v.data_ptr(),
                               k.stride(0), k.stride(1), v.stride(0), v.stride(1), scales_of(ks, vs), (int)k.size(0),
                               (int)k.size(1), ptr<int64_t>(slots), k_out.data_ptr(), v_out.data_ptr(), k_out.stride(0),
                               k_out.stride(1), v_out.stride(0), v_out.stride(1)};
  const int status = moe_read_e4m3(&a, reinterpret_cast<moe_stream_t>(stream));
  if (status != MOE_OK) return number(status);
  PyObject* o = THPVariable_Wrap(std::move(k_out));
  PyObject* l = o ? THPVariable_Wrap(std::move(v_out)) : nullptr;
  return l ? Py_BuildValue("(NN)", o, l) : (Py_XDECREF(o), nullptr);
}

// the scales of moved rows: pools [layers, pages, heads, page_size]
PyObject* copy_scales(Args x) {
  const int64_t stream = x.integer();
  const Tensor k = x.tensor(), v = x.tensor(), src = x.tensor(), dst = x.tensor();
  if (x.bad || k.dim() != 4 || !k.is_cuda() || src.dim() != 1) return number(kDoesNotFit);
  const int64_t gpu = k.get_device(), n = src.size(0);
  if (!k.sizes().equals(v.sizes()) || k.scalar_type() != at::kByte || v.scalar_type() != at::kByte || !on(v, gpu) ||
      !plain(src, at::kLong, n, gpu) || !plain(dst, at::kLong, n, gpu) || !fits_int(n) || !fits_int(k.size(0)) ||
      !fits_int(k.size(1)) || !fits_int(k.size(2)) || !fits_int(k.size(3)))
    return number(kDoesNotFit);
  for (const Tensor* t : {&k, &v})
    if (t->size(3) > 1 && t->stride(3) != 1) return number(kDoesNotFit);
  return number(moe_copy_scales(k.data_ptr(), v.data_ptr(), (int)k.size(0), k.stride(0), v.stride(0), k.stride(1),
                                v.stride(1), k.stride(2), v.stride(2), (int)k.size(1), (int)k.size(3), (int)k.size(2),
                                ptr<int64_t>(src), ptr<int64_t>(dst), (int)n, reinterpret_cast<moe_stream_t>(stream)));
}

PyObject* sample(Args x) {
  const int64_t stream = x.integer();
  const Tensor logits = x.tensor(), u = x.tensor();
  const Tensor t = x.tensor(true), k = x.tensor(true), p = x.tensor(true), least = x.tensor(true);
  Tensor tokens = x.tensor(true), probs;
  const bool want_probs = x.truth();
  if (x.bad || logits.dim() != 2 || !logits.is_cuda()) return number(kDoesNotFit);
  const int64_t gpu = logits.get_device(), M = logits.size(0), V = logits.size(1);
  if (logits.scalar_type() != at::kFloat || (V > 1 && logits.stride(1) != 1) || !plain(u, at::kFloat, M, gpu) ||
      (t.defined() && !plain(t, at::kFloat, M, gpu)) || (k.defined() && !plain(k, at::kInt, M, gpu)) ||
      (p.defined() && !plain(p, at::kFloat, M, gpu)) || (least.defined() && !plain(least, at::kFloat, M, gpu)) ||
      (tokens.defined() && !plain(tokens, at::kInt, M, gpu)) || !fits_int(M) || !fits_int(V))
    return number(kDoesNotFit);
  if (!tokens.defined()) tokens = at::empty({M}, logits.options().dtype(at::kInt));
  if (want_probs) probs = at::empty({M}, logits.options());
  const int status = moe_sample(ptr<float>(logits), logits.stride(0), (int)M, (int)V, ptr<float>(u), ptr<float>(t),
                                ptr<int32_t>(k), ptr<float>(p), ptr<float>(least), ptr<int32_t>(tokens),
                                ptr<float>(probs), reinterpret_cast<moe_stream_t>(stream));
  if (status != MOE_OK) return number(status);
  PyObject* o = THPVariable_Wrap(std::move(tokens));
  if (!want_probs || !o) return o;
  PyObject* l = THPVariable_Wrap(std::move(probs));
  return l ? Py_BuildValue("(NN)", o, l) : (Py_DECREF(o), nullptr);
}

PyObject* adjust_logits(Args x) {
  const int64_t stream = x.integer();
  const Tensor logits = x.tensor(), history = x.tensor(true), spans = x.tensor(true), repetition = x.tensor(true);
  const Tensor presence = x.tensor(true), frequency = x.tensor(true), ids = x.tensor(true), values = x.tensor(true);
  const Tensor starts = x.tensor(true), allowed = x.tensor(true);
  Tensor out = x.tensor(true);
  if (x.bad || logits.dim() != 2 || !logits.is_cuda()) return number(kDoesNotFit);
  const int64_t gpu = logits.get_device(), M = logits.size(0), V = logits.size(1), words = (V + 31) / 32;
  auto row = [&](const Tensor& t) { return !t.defined() || plain(t, at::kFloat, M, gpu); };
  // [M, columns], rows any distance apart
  auto rows_of = [&](const Tensor& t, at::ScalarType type, int64_t columns) {
    return t.dim() == 2 && t.scalar_type() == type && on(t, gpu) && t.size(0) == M && t.size(1) == columns &&
           (columns < 2 || t.stride(1) == 1);
  };
  if (!rows_of(logits, at::kFloat, V) || (out.defined() && !rows_of(out, at::kFloat, V)) || !row(repetition) ||
      !row(presence) || !row(frequency) || history.defined() != spans.defined() ||
      (history.defined() && (!plain(history, at::kInt, history.numel(), gpu) || !rows_of(spans, at::kInt, 3) ||
                             !spans.is_contiguous() || !fits_int(history.numel()))) ||
      ids.defined() != values.defined() || ids.defined() != starts.defined() ||
      (ids.defined() && (!plain(ids, at::kInt, ids.numel(), gpu) || !plain(values, at::kFloat, ids.numel(), gpu) ||
                         !plain(starts, at::kInt, M + 1, gpu) || !fits_int(ids.numel()))) ||
      (allowed.defined() && !rows_of(allowed, at::kInt, words)) || !fits_int(M) || !fits_int(V))
    return number(kDoesNotFit);
  if (!out.defined()) out = at::empty({M, V}, logits.options());
  const moe_adjust_logits_args_t a{ptr<float>(logits), logits.stride(0), ptr<float>(out), out.stride(0), (int)M, (int)V,
                                   // an empty history or list has no address
                                   history.defined() && history.numel() > 0 ? ptr<int32_t>(history) : nullptr,
                                   history.defined() ? (int)history.numel() : 0, ptr<int32_t>(spans),
                                   ptr<float>(repetition), ptr<float>(presence), ptr<float>(frequency),
                                   ids.defined() && ids.numel() > 0 ? ptr<int32_t>(ids) : nullptr, ptr<float>(values),
                                   ids.defined() ? (int)ids.numel() : 0, ptr<int32_t>(starts),
                                   ptr<uint32_t>(allowed), allowed.defined() ? allowed.stride(0) : 0};
  const int status = moe_adjust_logits(&a, reinterpret_cast<moe_stream_t>(stream));
  return status == MOE_OK ? THPVariable_Wrap(std::move(out)) : number(status);
}

// C++ exceptions (of an allocation, say) become the Python ones that PyTorch's
// own calls raise.
template <PyObject* (*kCall)(Args)>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return kCall(Args{args, n});
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*kCall)(Args)>
PyCFunction entry() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&call<kCall>));
}

PyMethodDef methods[] = {{"qk_norm_rope", entry<qk_norm_rope>(), METH_FASTCALL, nullptr},
                         {"attention", entry<attention>(), METH_FASTCALL, nullptr},
                         {"copy", entry<copy>(), METH_FASTCALL, nullptr},
                         {"read_cache", entry<read_cache>(), METH_FASTCALL, nullptr},
                         {"copy_scales", entry<copy_scales>(), METH_FASTCALL, nullptr},
                         {"sample", entry<sample>(), METH_FASTCALL, nullptr},
                         {"adjust_logits", entry<adjust_logits>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "wse_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit_wse_calls() { return PyModule_Create(&module); }
