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
template <typename T>
T* ptr(const Tensor& t) {
  return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}
bool fits_int(int64_t v) { return v >= 0 && v <= 0x7fffffff; }

PyObject* qk_norm_rope(Args x) {
  const int64_t gpu = x.integer(), stream = x.integer(), dim = x.integer(), rotary = x.integer();
  const bool interleaved = x.truth();
  const double eps = x.real();
  const Tensor turns = x.tensor(), q = x.tensor(), k = x.tensor(), v = x.tensor();
  const Tensor qw = x.tensor(true), kw = x.tensor(true), positions = x.tensor(), slots = x.tensor();
  const Tensor k_cache = x.tensor(), v_cache = x.tensor();
  Tensor out = x.tensor(true);
  if (x.bad || q.dim() != 3 || k.dim() != 3) return number(kDoesNotFit);
  const auto type = q.scalar_type();
  const int64_t T = q.size(0), Hq = q.size(1), Hk = k.size(1);
  if (dtype_of(q) < 0 || !heads(q, type, T, Hq, dim, gpu) || !heads(k, type, T, Hk, dim, gpu) ||
      !heads(v, type, T, Hk, dim, gpu) || !cache(k_cache, type, Hk, dim, gpu) || !cache(v_cache, type, Hk, dim, gpu) ||
      !k_cache.sizes().equals(v_cache.sizes()) || !plain(positions, at::kInt, T, gpu) ||
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
  const int status = moe_qk_norm_rope(&a, reinterpret_cast<moe_stream_t>(stream));
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
  if (x.bad || q.dim() != 3 || table.dim() != 2) return number(kDoesNotFit);
  const auto type = q.scalar_type();
  const int64_t T = q.size(0), B = table.size(0);
  // a row's distance and its pages are two things: rows may be shared, or part of a wider table
  const int64_t row_step = B > 1 && table.size(1) > 0 ? table.stride(0) : 0;
  if (dtype_of(q) < 0 || !heads(q, type, T, Hq, dim, gpu) || !cache(k_cache, type, Hk, dim, gpu) ||
      !cache(v_cache, type, Hk, dim, gpu) || !k_cache.sizes().equals(v_cache.sizes()) ||
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
  const int status =
      moe_attn_forward(reinterpret_cast<moe_attn_t*>(handle), &a, reinterpret_cast<moe_stream_t>(stream));
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
                         {"sample", entry<sample>(), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "wse_calls", nullptr, -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit_wse_calls() { return PyModule_Create(&module); }
