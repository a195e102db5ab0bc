// operators_binding.cpp -- marshalling of the operators around the GEMMs (operators.py): checks of
// the tensors, allocation of outputs and scratch, the call of the C ABI.  Compiled, because a call of a
// decode step takes as long as its host side: through ctypes the router took 20 us of host time, the
// layout and the dispatch 20, an adapter call 11.
//
// Every function takes its arguments by position and runs on the current device and stream.  It returns
// None, having done nothing, if the first tensor is on another device.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "fp8gemm.h"

namespace {

typedef at::Tensor Tensor;
PyObject* g_error = nullptr;  // FP8GemmError(code, what)

// The Python error that is to be raised is set.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& text) {
  PyErr_SetString(type, text.c_str());
  throw Raised();
}

void check(fg_status code, const char* what) {
  if (code == FG_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", static_cast<int>(code), what);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Raised();
}

const char* type_name(at::ScalarType t) {
  switch (t) {
    case at::kInt: return "int32";
    case at::kFloat: return "float32";
    case at::kBFloat16: return "bfloat16";
    case at::kByte: return "uint8";
    case at::kBool: return "bool";
    default: return "?";
  }
}

std::string shape_text(at::IntArrayRef s) {
  std::string text = "(";
  for (size_t i = 0; i < s.size(); ++i) text += (i ? ", " : "") + std::to_string(s[i]);
  return text + (s.size() == 1 ? ",)" : ")");
}

const Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(what) + " must be a tensor");
  return THPVariable_Unpack(o);
}

void need_type(const Tensor& t, at::ScalarType type, const char* what) {
  if (t.scalar_type() != type || !t.is_cuda() || !t.is_contiguous())
    raise(PyExc_TypeError, std::string(what) + " must be a contiguous CUDA " + type_name(type) + " tensor");
}

void need_shape(const Tensor& t, at::IntArrayRef shape, const char* what) {
  if (t.sizes() != shape)
    raise(PyExc_ValueError, std::string(what) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
}

// A tensor beside `first`: its type, device and shape.
const Tensor& beside(PyObject* o, at::ScalarType type, at::IntArrayRef shape, const Tensor& first, const char* what) {
  const Tensor& t = tensor(o, what);
  need_type(t, type, what);
  if (t.get_device() != first.get_device())
    raise(PyExc_ValueError, std::string(what) + " is on cuda:" + std::to_string(t.get_device()) +
                                ", the first operand on cuda:" + std::to_string(first.get_device()));
  need_shape(t, shape, what);
  return t;
}
const Tensor* beside_or_none(PyObject* o, at::ScalarType type, at::IntArrayRef shape, const Tensor& first,
                             const char* what) {
  return o == Py_None ? nullptr : &beside(o, type, shape, first, what);
}

template <typename T = void>
T* ptr(const Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
template <typename T = void>
T* ptr(const Tensor* t) {
  return t ? static_cast<T*>(t->data_ptr()) : nullptr;
}

// An output must not share memory with an input (or another output).
void apart(const Tensor& out, const char* what, const Tensor* other, const char* name) {
  if (!other || out.nbytes() == 0 || other->nbytes() == 0) return;
  const char *a = ptr<char>(out), *b = ptr<char>(*other);
  if (a < b + other->nbytes() && b < a + out.nbytes())
    raise(PyExc_ValueError, std::string(what) + " must not overlap " + name);
}

bool elsewhere(const Tensor& t) { return t.get_device() != c10::cuda::current_device(); }
void* stream_of(const Tensor& t) { return c10::cuda::getCurrentCUDAStream(t.get_device()).stream(); }

Tensor empty(at::IntArrayRef shape, const Tensor& like, at::ScalarType type) {
  return at::empty(shape, like.options().dtype(type));
}
Tensor scratch_of(size_t bytes, const Tensor& like) {
  return bytes ? empty({static_cast<int64_t>(bytes)}, like, at::kByte) : Tensor();
}
void* address(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

int to_int(int64_t v, const char* what) {
  if (v < 0 || v > 0x7fffffff) raise(PyExc_ValueError, std::string(what) + " is too large");
  return static_cast<int>(v);
}
int arg_int(PyObject* o, const char* what) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  if (v < -0x7fffffffll || v > 0x7fffffffll) raise(PyExc_ValueError, std::string(what) + " is too large");
  return static_cast<int>(v);
}

bool arg_bool(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised();
  return v != 0;
}

PyObject* wrap(const Tensor& t) { return THPVariable_Wrap(t); }
PyObject* given(PyObject* o) {
  Py_INCREF(o);
  return o;
}
// A tuple of new references (each may be null after a failed wrap).
template <typename... Objects>
PyObject* tuple_of(Objects*... objects) {
  PyObject* list[] = {objects...};
  bool ok = true;
  for (PyObject* o : list) ok = ok && o;
  PyObject* t = ok ? PyTuple_New(sizeof...(objects)) : nullptr;
  Py_ssize_t i = 0;
  for (PyObject* o : list) {
    if (t)
      PyTuple_SET_ITEM(t, i++, o);
    else
      Py_XDECREF(o);
  }
  return t;
}

struct Logits {
  const Tensor& t;
  int type, S, T, E;
  at::IntArrayRef lead;  // [] or [S]
};
Logits logits_of(PyObject* o) {
  const Tensor& t = tensor(o, "logits");
  int type;
  if (t.scalar_type() == at::kFloat)
    type = FG_F32;
  else if (t.scalar_type() == at::kBFloat16)
    type = FG_BF16;
  else if (t.scalar_type() == at::kHalf)
    type = FG_F16;
  else
    raise(PyExc_TypeError, "logits must be float32, bfloat16 or float16");
  if (!t.is_cuda() || !t.is_contiguous()) raise(PyExc_ValueError, "logits must be a contiguous CUDA tensor");
  const int64_t d = t.dim();
  if (d != 2 && d != 3) raise(PyExc_ValueError, "logits must be [T, E] or [S, T, E]");
  return {t, type, d == 3 ? to_int(t.size(0), "logits") : 1, to_int(t.size(d - 2), "logits"),
          to_int(t.size(d - 1), "logits"), t.sizes().slice(0, d - 2)};
}
c10::SmallVector<int64_t, 4> joined(at::IntArrayRef lead, std::initializer_list<int64_t> rest) {
  c10::SmallVector<int64_t, 4> v(lead.begin(), lead.end());
  v.append(rest.begin(), rest.end());
  return v;
}

// (logits, k, mask, renormalize)
PyObject* moe_route(PyObject* const* a) {
  const Logits l = logits_of(a[0]);
  const int k = arg_int(a[1], "top_k"), renorm = arg_bool(a[3]);
  if (k < 1 || k > l.E)
    raise(PyExc_ValueError, "top_k must be in 1.." + std::to_string(l.E) + ", got " + std::to_string(k));
  const Tensor* mask = beside_or_none(a[2], at::kBool, joined(l.lead, {l.T}), l.t, "mask");
  if (elsewhere(l.t)) Py_RETURN_NONE;
  const Tensor ids = empty(joined(l.lead, {l.T, k}), l.t, at::kInt);
  const Tensor weights = empty(joined(l.lead, {l.T, k}), l.t, at::kFloat);
  const Tensor counts = empty(joined(l.lead, {l.E}), l.t, at::kInt);
  const Tensor slope = empty(joined(l.lead, {l.E}), l.t, at::kFloat);
  const Tensor loss = empty(l.lead, l.t, at::kFloat);
  const size_t bytes = fg_moe_route_scratch_bytes(l.S, l.T, l.E);
  const Tensor scratch = scratch_of(bytes, l.t);
  check(fg_moe_route(ptr(l.t), l.type, ptr<unsigned char>(mask), ptr<int>(ids), ptr<float>(weights), ptr<int>(counts),
                     ptr<float>(loss), ptr<float>(slope), l.S, l.T, l.E, k, renorm, address(scratch), bytes,
                     stream_of(l.t)),
        "fg_moe_route");
  return tuple_of(wrap(ids), wrap(weights), wrap(counts), wrap(loss), wrap(slope));
}

// (logits, ids, slope, grad_weights, grad_loss, renormalize)
PyObject* moe_route_backward(PyObject* const* a) {
  const Logits l = logits_of(a[0]);
  const Tensor& given_ids = tensor(a[1], "ids");
  if (given_ids.dim() != l.t.dim()) raise(PyExc_ValueError, "ids must be [..., k] beside logits [..., E]");
  const int k = to_int(given_ids.size(-1), "ids");
  const auto choices = joined(l.lead, {l.T, k});
  const Tensor& ids = beside(a[1], at::kInt, choices, l.t, "ids");
  const Tensor& slope = beside(a[2], at::kFloat, joined(l.lead, {l.E}), l.t, "slope");
  const Tensor* grad_weights = beside_or_none(a[3], at::kFloat, choices, l.t, "grad_weights");
  const Tensor* grad_loss = beside_or_none(a[4], at::kFloat, l.lead, l.t, "grad_loss");
  const int renorm = arg_bool(a[5]);
  if (elsewhere(l.t)) Py_RETURN_NONE;
  const Tensor grad = empty(l.t.sizes(), l.t, l.t.scalar_type());
  check(fg_moe_route_backward(ptr(l.t), l.type, ptr<int>(ids), ptr<float>(slope), ptr<float>(grad_weights),
                              ptr<float>(grad_loss), ptr(grad), l.S, l.T, l.E, k, renorm, stream_of(l.t)),
        "fg_moe_route_backward");
  return wrap(grad);
}

// (ids, num_experts, mmax): mmax 0 for the contiguous layout
PyObject* moe_layout(PyObject* const* a) {
  const Tensor& ids = tensor(a[0], "ids");
  need_type(ids, at::kInt, "ids");
  const int E = arg_int(a[1], "num_experts"), mmax = arg_int(a[2], "mmax");
  if (E < 1 || E > FG_MOE_MAX_EXPERTS)
    raise(PyExc_ValueError, "num_experts must be in 1.." + std::to_string(FG_MOE_MAX_EXPERTS) + ", got " + std::to_string(E));
  if (elsewhere(ids)) Py_RETURN_NONE;
  const int64_t pairs = ids.numel();
  const Tensor rows = empty(ids.sizes(), ids, at::kInt);
  const int n = mmax > 0 ? E : to_int(fg_moe_layout_rows(pairs, E), "the layout");
  const Tensor group = empty({n}, ids, at::kInt);
  const size_t bytes = fg_moe_layout_scratch_bytes(pairs, E);
  const Tensor scratch = scratch_of(bytes, ids);
  if (mmax > 0)
    check(fg_moe_layout_masked(ptr<int>(ids), ptr<int>(rows), ptr<int>(group), pairs, E, mmax, address(scratch), bytes,
                               stream_of(ids)),
          "fg_moe_layout_masked");
  else
    check(fg_moe_layout_contiguous(ptr<int>(ids), ptr<int>(rows), ptr<int>(group), pairs, E, n, address(scratch), bytes,
                                   stream_of(ids)),
          "fg_moe_layout_contiguous");
  return tuple_of(wrap(rows), wrap(group));
}

// rows int32 [tokens, k] (tokens < 0: any number)
const Tensor& rows_of(PyObject* o, int64_t tokens, const Tensor& first) {
  const Tensor& rows = tensor(o, "rows");
  if (rows.dim() != 2 || (tokens >= 0 && rows.size(0) != tokens))
    raise(PyExc_ValueError, "rows must be [" + (tokens < 0 ? "T" : std::to_string(tokens)) + ", k], got " + shape_text(rows.sizes()));
  return beside(o, at::kInt, rows.sizes(), first, "rows");
}

// (x, rows, layout shape (M,) or (G, Mmax) or None, A, sfa, format code)
PyObject* moe_dispatch_fp8(PyObject* const* a) {
  const Tensor& x = tensor(a[0], "x");
  need_type(x, at::kBFloat16, "x");
  if (x.dim() != 2) raise(PyExc_ValueError, "x must be [T, K]");
  const int T = to_int(x.size(0), "x"), K = to_int(x.size(1), "x");
  const Tensor& rows = rows_of(a[1], T, x);
  const int fmt = arg_int(a[5], "fmt");
  const bool have = a[3] != Py_None;
  if (have != (a[4] != Py_None) || (!have && a[2] == Py_None)) raise(PyExc_ValueError, "give shape, or both A and sfa");
  c10::SmallVector<int64_t, 4> lead;
  if (a[2] != Py_None) {
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(a[2]); ++i) {
      const int n = arg_int(PyTuple_GET_ITEM(a[2], i), "shape");
      if (n < 0) raise(PyExc_ValueError, "shape must not be negative");
      lead.push_back(n);
    }
  }
  if (have) {
    const Tensor& A = tensor(a[3], "A");
    if (A.dim() < 1 || (a[2] != Py_None && A.sizes().slice(0, A.dim() - 1) != at::IntArrayRef(lead)))
      raise(PyExc_ValueError, "A does not have the given shape");
    lead.assign(A.sizes().begin(), A.sizes().end() - 1);
  }
  if (lead.size() != 1 && lead.size() != 2) raise(PyExc_ValueError, "the layout is M rows or (G, Mmax)");
  const int M = to_int(lead.back(), "the layout"), G = lead.size() == 2 ? to_int(lead[0], "the layout") : 1;
  if (M > FG_MOE_MAX_ROWS) raise(PyExc_ValueError, "the layout is too large");
  const auto scales = joined(at::IntArrayRef(lead).slice(0, lead.size() - 1), {(static_cast<int64_t>(K) + 127) / 128, fg_sfa_ld(M)});
  const auto codes = joined(lead, {K});
  Tensor A, sfa;
  if (have) {
    // codes as bytes or as values of the format, as the GEMMs take them
    const at::ScalarType float8 = fmt == FG_E4M3 ? at::kFloat8_e4m3fn : at::kFloat8_e5m2;
    A = beside(a[3], tensor(a[3], "A").scalar_type() == float8 ? float8 : at::kByte, codes, x, "A");
    sfa = beside(a[4], at::kFloat, scales, x, "sfa");
    apart(A, "A", &x, "x");
    apart(A, "A", &rows, "rows");
    apart(A, "A", &sfa, "sfa");
    apart(sfa, "sfa", &x, "x");
    apart(sfa, "sfa", &rows, "rows");
  }
  if (elsewhere(x)) Py_RETURN_NONE;
  if (!have) {
    A = empty(codes, x, at::kByte);
    sfa = at::zeros(scales, x.options().dtype(at::kFloat));
  }
  check(fg_moe_dispatch_fp8(ptr(x), ptr<int>(rows), ptr(A), ptr<float>(sfa), T, to_int(rows.size(1), "rows"), G, M, K,
                            fmt, stream_of(x)),
        "fg_moe_dispatch_fp8");
  return have ? tuple_of(given(a[3]), given(a[4])) : tuple_of(wrap(A), wrap(sfa));
}

// C bf16 [M, N] or [G, Mmax, N]
struct ExpertRows {
  const Tensor& t;
  int M, N;
};
ExpertRows expert_rows(PyObject* o) {
  const Tensor& t = tensor(o, "C");
  need_type(t, at::kBFloat16, "C");
  if (t.dim() != 2 && t.dim() != 3) raise(PyExc_ValueError, "C must be [M, N] or [G, Mmax, N]");
  return {t, to_int(t.dim() == 2 ? t.size(0) : t.size(0) * t.size(1), "C"), to_int(t.size(-1), "C")};
}

// (C, rows, weights, out)
PyObject* moe_combine(PyObject* const* a) {
  const ExpertRows C = expert_rows(a[0]);
  const Tensor& rows = rows_of(a[1], -1, C.t);
  const Tensor* weights = beside_or_none(a[2], at::kFloat, rows.sizes(), C.t, "weights");
  const int T = to_int(rows.size(0), "rows");
  const bool have = a[3] != Py_None;
  Tensor out;
  if (have) {
    out = beside(a[3], at::kBFloat16, {T, C.N}, C.t, "out");
    apart(out, "out", &C.t, "C");
    apart(out, "out", &rows, "rows");
    apart(out, "out", weights, "weights");
  }
  if (elsewhere(C.t)) Py_RETURN_NONE;
  if (!have) out = empty({T, C.N}, C.t, at::kBFloat16);
  check(fg_moe_combine(ptr(C.t), ptr<int>(rows), ptr<float>(weights), ptr(out), T, to_int(rows.size(1), "rows"), C.M, C.N,
                       stream_of(C.t)),
        "fg_moe_combine");
  return have ? given(a[3]) : wrap(out);
}

// (grad_out, C, rows, weights, grad_C)
PyObject* moe_combine_backward(PyObject* const* a) {
  const ExpertRows C = expert_rows(a[1]);
  const Tensor& rows = rows_of(a[2], -1, C.t);
  const int T = to_int(rows.size(0), "rows");
  const Tensor& grad_out = beside(a[0], at::kBFloat16, {T, C.N}, C.t, "grad_out");
  const Tensor& weights = beside(a[3], at::kFloat, rows.sizes(), C.t, "weights");
  const bool have = a[4] != Py_None;
  Tensor grad_C;
  if (have) {
    grad_C = beside(a[4], at::kBFloat16, C.t.sizes(), C.t, "grad_C");
    apart(grad_C, "grad_C", &C.t, "C");
    apart(grad_C, "grad_C", &grad_out, "grad_out");
    apart(grad_C, "grad_C", &rows, "rows");
    apart(grad_C, "grad_C", &weights, "weights");
  }
  if (elsewhere(C.t)) Py_RETURN_NONE;
  if (!have) grad_C = empty(C.t.sizes(), C.t, at::kBFloat16);
  const Tensor grad_weights = empty(rows.sizes(), C.t, at::kFloat);
  check(fg_moe_combine_backward(ptr(grad_out), ptr(C.t), ptr<int>(rows), ptr<float>(weights), ptr(grad_C),
                                ptr<float>(grad_weights), T, to_int(rows.size(1), "rows"), C.M, C.N, stream_of(C.t)),
        "fg_moe_combine_backward");
  return tuple_of(have ? given(a[4]) : wrap(grad_C), wrap(grad_weights));
}

// (C, x, lora_a, lora_b, adapters, scaling, out)
PyObject* lora_add(PyObject* const* a) {
  const Tensor& C = tensor(a[0], "C");
  need_type(C, at::kBFloat16, "C");
  const Tensor& any_a = tensor(a[2], "lora_a");
  if (C.dim() != 2 || any_a.dim() != 3) raise(PyExc_ValueError, "C must be [M, N], x [M, K], lora_a [L, R, K]");
  const int M = to_int(C.size(0), "C"), N = to_int(C.size(1), "C");
  const int L = to_int(any_a.size(0), "lora_a"), R = to_int(any_a.size(1), "lora_a"), K = to_int(any_a.size(2), "lora_a");
  const Tensor& x = beside(a[1], at::kBFloat16, {M, K}, C, "x");
  const Tensor& lora_a = beside(a[2], at::kBFloat16, {L, R, K}, C, "lora_a");
  const Tensor& lora_b = beside(a[3], at::kBFloat16, {L, N, R}, C, "lora_b");
  const Tensor& adapters = beside(a[4], at::kInt, {M}, C, "adapters");
  const Tensor* scaling = beside_or_none(a[5], at::kFloat, {L}, C, "scaling");
  const bool have = a[6] != Py_None;
  Tensor out;
  if (have) {
    out = beside(a[6], at::kBFloat16, {M, N}, C, "out");
    if (ptr(out) != ptr(C)) apart(out, "out", &C, "C");  // in place is fine
    apart(out, "out", &x, "x");
    apart(out, "out", &lora_a, "lora_a");
    apart(out, "out", &lora_b, "lora_b");
    apart(out, "out", &adapters, "adapters");
    apart(out, "out", scaling, "scaling");
  }
  if (elsewhere(C)) Py_RETURN_NONE;
  if (!have) out = empty({M, N}, C, at::kBFloat16);
  const size_t bytes = fg_lora_scratch_bytes(M, R, L);
  const Tensor scratch = scratch_of(bytes, C);
  check(fg_lora_add(ptr(C), ptr(x), ptr(lora_a), ptr(lora_b), ptr<int>(adapters), ptr<float>(scaling), ptr(out), M, N, K, R,
                    L, address(scratch), bytes, stream_of(C)),
        "fg_lora_add");
  return have ? given(a[6]) : wrap(out);
}

// The entry of a function of N arguments.
template <PyObject* (*F)(PyObject* const*), Py_ssize_t N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_XDECREF(g_error);
  g_error = given(type);
  Py_RETURN_NONE;
}

#define ENTRY(f, n) \
  { #f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<f, n>)), METH_FASTCALL, nullptr }

PyMethodDef methods[] = {ENTRY(moe_route, 4),
                         ENTRY(moe_route_backward, 6),
                         ENTRY(moe_layout, 3),
                         ENTRY(moe_dispatch_fp8, 6),
                         ENTRY(moe_combine, 4),
                         ENTRY(moe_combine_backward, 5),
                         ENTRY(lora_add, 7),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_operators", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__operators() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", FG_TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
