// Native side of binding.quant_fp8, gemm_fp8, balance_loss and balance_loss_backward: argument checks,
// output allocation and the C-ABI call, on the tensors' device and its current stream.  The kernels of one
// decode token or a small batch run for a few microseconds; marshalling their twenty-odd arguments in
// Python took longer than that.  Wrong arguments raise ValueError or TypeError; a refusal by the library
// is returned as its code, which the Python side raises.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <string>

#include "../../include/moe_b200.h"

namespace {

struct Refused {
  PyObject* type;
  std::string what;
};
template <class... A>
[[noreturn]] void value_error(const A&... a) {
  std::ostringstream s;
  (s << ... << a);
  throw Refused{PyExc_ValueError, s.str()};
}
template <class... A>
[[noreturn]] void type_error(const A&... a) {
  std::ostringstream s;
  (s << ... << a);
  throw Refused{PyExc_TypeError, s.str()};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) type_error(name, " must be a tensor, got ", Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}
at::ScalarType dtype(PyObject* o, const char* name) {
  if (!THPDtype_Check(o)) type_error(name, " must be a torch.dtype, got ", Py_TYPE(o)->tp_name);
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}
bool truth(PyObject* o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw Refused{nullptr, ""};
  return r != 0;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{nullptr, ""};
  return v;
}
int to_int(int64_t v, const char* name) {
  if (v > INT32_MAX) value_error(name, " of ", v, " rows or columns is beyond 2^31 - 1");
  return (int)v;
}
bool is_none(PyObject* o) { return o == Py_None; }

void on_cuda(const at::Tensor& t) {
  if (!t.is_cuda()) value_error("tensors must be on a CUDA device, got ", t.device());
}
void beside(const at::Tensor& t, const char* name, c10::Device d) {
  if (t.device() != d) value_error(name, " on ", t.device(), ", expected ", d);
}
void shaped(const at::Tensor& t, const char* name, at::IntArrayRef shape) {
  if (t.sizes() != shape) value_error(name, " must be ", shape, ", got shape ", t.sizes());
}
// Row pitch (elements) of a matrix whose rows are contiguous.
int64_t pitch(const at::Tensor& t, const char* name) {
  const int64_t rows = t.size(0), cols = t.size(1);
  if (cols > 1 && t.stride(1) != 1) value_error("the rows of ", name, " must be contiguous, got strides ", t.strides());
  return rows > 1 ? t.stride(0) : cols > 1 ? cols : 1;
}
void matrix(const at::Tensor& t, const char* name) {
  if (t.dim() != 2) value_error(name, " must be a matrix, got shape ", t.sizes());
}

int format_of(at::ScalarType t, const char* name) {
  switch (t) {
    case at::kFloat8_e4m3fn:
    case at::kByte: return MOE_FP8_E4M3;       // plain bytes are E4M3 codes
    case at::kFloat8_e5m2: return MOE_FP8_E5M2;
    default: type_error(name, " must be float8_e4m3fn, float8_e5m2 or uint8 (E4M3 codes), got ", t);
  }
}
int scale_type_of(at::ScalarType t) {
  if (t == at::kFloat) return MOE_SCALE_FP32;
  if (t == at::kByte) return MOE_SCALE_UE8M0;
  type_error("scales must be float32 or uint8 (UE8M0), got ", t);
}
int64_t blocks(int64_t n) { return (n + 127) / 128; }

struct Launch {                                // the tensors' device, and its current stream
  c10::cuda::CUDAGuard guard;
  void* stream;
  explicit Launch(c10::Device d) : guard(d), stream(c10::cuda::getCurrentCUDAStream(d.index()).stream()) {}
};
at::Tensor make(at::IntArrayRef shape, at::ScalarType t, c10::Device d) {
  return at::empty(shape, at::TensorOptions().dtype(t).device(d));
}
PyObject* wrap(const at::Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
PyObject* tuple(std::initializer_list<at::Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = wrap(t);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    if (n != N) type_error("takes ", N, " arguments, got ", n);
    return F(args);
  } catch (const Refused& e) {
    if (e.type) PyErr_SetString(e.type, e.what.c_str());
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(PyExc_MemoryError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// ------------------------------------------------------------------ quant_fp8
struct Side {                                  // codes and scales of one direction
  at::Tensor q, s;
  int64_t ld = 0;
};
Side side(PyObject* given_q, PyObject* given_s, int64_t n, int64_t m, int64_t s_rows, int64_t s_blocks, at::ScalarType t,
          at::ScalarType st, c10::Device d) {
  Side r;
  if (is_none(given_q)) {
    r.ld = (m + 15) / 16 * 16;
    r.q = make({n, r.ld}, t, d);
    if (r.ld != m) r.q = r.q.narrow(1, 0, m);
  } else {
    r.q = tensor(given_q, "out codes");
    shaped(r.q, "out codes", {n, m});
    beside(r.q, "out codes", d);
    if (r.q.scalar_type() != t) type_error("out codes must be ", t, ", got ", r.q.scalar_type());
    r.ld = pitch(r.q, "out codes");
  }
  if (is_none(given_s)) {                      // scales of consecutive rows next to each other
    r.s = at::empty_strided({s_rows, s_blocks}, {1, s_rows > 0 ? s_rows : 1}, at::TensorOptions().dtype(st).device(d));
  } else {
    r.s = tensor(given_s, "out scales");
    shaped(r.s, "out scales", {s_rows, s_blocks});
    beside(r.s, "out scales", d);
    if (r.s.scalar_type() != st) type_error("out scales must be ", st, ", got ", r.s.scalar_type());
  }
  return r;
}

// x, tile, rows, cols, dtype, scale_dtype, q, s, qt, st
PyObject* quant_fp8(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "x");
  matrix(x, "x");
  const bool tile = truth(a[1]), rows = truth(a[2]), cols = truth(a[3]);
  const at::ScalarType t = dtype(a[4], "dtype"), st = dtype(a[5], "scale_dtype");
  const int fmt = format_of(t, "dtype"), stype = scale_type_of(st);
  if (!rows && !cols) value_error("nothing to write: rows or cols");
  const int64_t M = x.size(0), K = x.size(1), mb = blocks(M), kb = blocks(K);
  int xt;
  switch (x.scalar_type()) {
    case at::kBFloat16: xt = MOE_TYPE_BF16; break;
    case at::kFloat: xt = MOE_TYPE_FP32; break;
    case at::kHalf: xt = MOE_TYPE_FP16; break;
    default: type_error("x must be bfloat16, float16 or float32, got ", x.scalar_type());
  }
  const int64_t ldx = pitch(x, "x");
  on_cuda(x);
  const c10::Device d = x.device();
  const int m = to_int(M, "x"), k = to_int(K, "x");
  Launch on(d);
  Side r, c;
  if (rows) r = side(a[6], a[7], M, K, tile ? mb : M, kb, t, st, d);
  if (cols) c = side(a[8], a[9], K, M, tile ? kb : K, mb, t, st, d);
  const int rc = moe_quant_fp8(
      m, k, x.data_ptr(), ldx, xt, tile ? MOE_BLOCK_TILE : MOE_BLOCK_ROW, fmt, stype, rows ? r.q.data_ptr() : nullptr, r.ld,
      rows ? r.s.data_ptr() : nullptr, rows ? r.s.stride(0) : 0, rows ? r.s.stride(1) : 0,
      cols ? c.q.data_ptr() : nullptr, c.ld, cols ? c.s.data_ptr() : nullptr, cols ? c.s.stride(0) : 0,
      cols ? c.s.stride(1) : 0, on.stream);
  if (rc != MOE_OK) return PyLong_FromLong(rc);
  return tuple({r.q, r.s, c.q, c.s});
}

// ------------------------------------------------------------------ gemm_fp8
int scale_rows(const at::Tensor& s, const char* name, int64_t rows, int64_t kb, at::ScalarType t, c10::Device d) {
  if (s.scalar_type() != t) type_error(name, " must be ", t, " like the other operand's, got ", s.scalar_type());
  beside(s, name, d);
  if (s.dim() == 2 && s.size(1) == kb) {
    if (s.size(0) == rows) return 1;
    if (s.size(0) == blocks(rows)) return 128;
  }
  value_error(name, " must be [", rows, ", ", kb, "] or [", blocks(rows), ", ", kb, "], got shape ", s.sizes());
}

// A, A_scales, B, B_scales, out, out_dtype, accumulate, workspace
PyObject* gemm_fp8(PyObject* const* a) {
  const at::Tensor &A = tensor(a[0], "A"), &As = tensor(a[1], "A_scales"), &B = tensor(a[2], "B"),
                   &Bs = tensor(a[3], "B_scales");
  matrix(A, "A");
  matrix(B, "B");
  const int64_t M = A.size(0), K = A.size(1), N = B.size(0), kb = blocks(K);
  if (B.size(1) != K) value_error("B must be [N, ", K, "], got shape ", B.sizes());
  const c10::Device d = A.device();
  beside(B, "B", d);
  const int fa = format_of(A.scalar_type(), "A"), fb = format_of(B.scalar_type(), "B");
  const int stype = scale_type_of(As.scalar_type());
  const int ar = scale_rows(As, "A_scales", M, kb, As.scalar_type(), d);
  const int br = scale_rows(Bs, "B_scales", N, kb, As.scalar_type(), d);
  const int64_t lda = pitch(A, "A"), ldb = pitch(B, "B");
  const bool add = truth(a[6]);
  at::Tensor out;
  at::ScalarType ot;
  int64_t ldo = N;
  if (is_none(a[4])) {
    if (add) value_error("accumulate needs the out to add to");
    ot = dtype(a[5], "out_dtype");
  } else {
    out = tensor(a[4], "out");
    shaped(out, "out", {M, N});
    beside(out, "out", d);
    ldo = pitch(out, "out");
    ot = out.scalar_type();
  }
  if (ot != at::kBFloat16 && ot != at::kFloat) type_error("out must be bfloat16 or float32, got ", ot);
  on_cuda(A);
  const int m = to_int(M, "A"), n = to_int(N, "B"), k = to_int(K, "A");
  Launch on(d);
  if (!out.defined()) out = make({M, N}, ot, d);
  at::Tensor ws;
  if (is_none(a[7])) {
    ws = make({(int64_t)moe_gemm_fp8_workspace_bytes()}, at::kByte, d);
  } else {
    ws = tensor(a[7], "workspace");
    beside(ws, "workspace", d);
    if (ws.scalar_type() != at::kByte || !ws.is_contiguous()) type_error("workspace must be contiguous uint8");
  }
  const int rc = moe_gemm_fp8(m, n, k, A.data_ptr(), lda, fa, As.data_ptr(), As.stride(0), As.stride(1), ar, B.data_ptr(),
                              ldb, fb, Bs.data_ptr(), Bs.stride(0), Bs.stride(1), br, stype, out.data_ptr(), ldo,
                              ot == at::kFloat ? MOE_TYPE_FP32 : MOE_TYPE_BF16, add, ws.data_ptr(), ws.numel(), on.stream);
  if (rc != MOE_OK) return PyLong_FromLong(rc);
  return tuple({out, ws});
}

// ------------------------------------------------------------------ balance loss
struct Routing {                               // what the loss and its gradient have in common
  int T, E, S = 1, type, score;
  int64_t ld;
  const void* logits;
  const int32_t* offsets = nullptr;
  const uint8_t* mask = nullptr;
  float coef;
  c10::Device d;
};
const int32_t* ints(const at::Tensor& t, const char* name, c10::Device d) {
  if (t.scalar_type() != at::kInt) type_error(name, " must be int32, got ", t.scalar_type());
  beside(t, name, d);
  if (!t.is_contiguous()) value_error(name, " must be contiguous");
  return static_cast<const int32_t*>(t.data_ptr());
}
Routing routing(PyObject* logits, PyObject* coef, PyObject* offsets, PyObject* mask, PyObject* sigmoid) {
  const at::Tensor& l = tensor(logits, "logits");
  matrix(l, "logits");
  const at::ScalarType t = l.scalar_type();
  if (t != at::kFloat && t != at::kBFloat16) type_error("logits must be float32 or bfloat16, got ", t);
  Routing r{to_int(l.size(0), "logits"),
            to_int(l.size(1), "logits"),
            1,
            t == at::kFloat ? MOE_TYPE_FP32 : MOE_TYPE_BF16,
            truth(sigmoid) ? MOE_SCORE_SIGMOID : MOE_SCORE_SOFTMAX,
            pitch(l, "logits"),
            l.data_ptr(),
            nullptr,
            nullptr,
            (float)number(coef),
            l.device()};
  if (!is_none(offsets)) {
    const at::Tensor& o = tensor(offsets, "offsets");
    if (o.dim() != 1 || o.numel() < 2) value_error("offsets must be [S + 1], got shape ", o.sizes());
    r.offsets = ints(o, "offsets", r.d);
    r.S = to_int(o.numel() - 1, "offsets");
  }
  if (!is_none(mask)) {
    const at::Tensor& m = tensor(mask, "mask");
    shaped(m, "mask", {r.T});
    beside(m, "mask", r.d);
    if (m.scalar_type() != at::kBool && m.scalar_type() != at::kByte) type_error("mask must be bool, got ", m.scalar_type());
    if (!m.is_contiguous()) value_error("mask must be contiguous");
    r.mask = static_cast<const uint8_t*>(m.data_ptr());
  }
  return r;
}

// logits, topk_ids, coef, offsets, mask, sigmoid, workspace
PyObject* balance_loss(PyObject* const* a) {
  const Routing r = routing(a[0], a[2], a[3], a[4], a[5]);
  const at::Tensor& ids = tensor(a[1], "topk_ids");
  if (ids.dim() != 2 || ids.size(0) != r.T) value_error("topk_ids must be [", r.T, ", k], got shape ", ids.sizes());
  const int k = to_int(ids.size(1), "topk_ids");
  const int32_t* idp = ints(ids, "topk_ids", r.d);
  const size_t need = moe_balance_workspace_bytes(r.T, r.E, r.S);
  if (need == 0) return PyLong_FromLong(MOE_ERR_UNSUPPORTED_SHAPE);
  on_cuda(THPVariable_Unpack(a[0]));
  Launch on(r.d);
  at::Tensor ws;
  if (is_none(a[6])) {
    ws = make({(int64_t)need}, at::kByte, r.d);
  } else {
    ws = tensor(a[6], "workspace");
    beside(ws, "workspace", r.d);
    if (ws.scalar_type() != at::kByte || !ws.is_contiguous()) type_error("workspace must be contiguous uint8");
  }
  at::Tensor loss = make({}, at::kFloat, r.d), counts = make({r.S, r.E}, at::kInt, r.d),
             probs = make({r.S, r.E}, at::kFloat, r.d), tokens = make({r.S}, at::kInt, r.d);
  const int rc = moe_balance_loss(r.T, r.E, k, r.S, r.logits, r.ld, r.type, idp, r.offsets, r.mask, r.score, r.coef,
                                  static_cast<float*>(loss.data_ptr()), static_cast<int32_t*>(counts.data_ptr()),
                                  static_cast<float*>(probs.data_ptr()), static_cast<int32_t*>(tokens.data_ptr()),
                                  ws.data_ptr(), ws.numel(), on.stream);
  if (rc != MOE_OK) return PyLong_FromLong(rc);
  return tuple({loss, counts, probs, tokens});
}

// grad_loss, logits, counts, tokens, k, coef, offsets, mask, sigmoid, out, accumulate
PyObject* balance_loss_backward(PyObject* const* a) {
  const Routing r = routing(a[1], a[5], a[6], a[7], a[8]);
  const at::Tensor &g = tensor(a[0], "grad_loss"), &counts = tensor(a[2], "counts"), &tokens = tensor(a[3], "tokens"),
                   &l = THPVariable_Unpack(a[1]);
  if (g.numel() != 1) value_error("grad_loss must be a scalar, got shape ", g.sizes());
  if (g.scalar_type() != at::kFloat) type_error("grad_loss must be float32, got ", g.scalar_type());
  beside(g, "grad_loss", r.d);
  shaped(counts, "counts", {r.S, r.E});
  shaped(tokens, "tokens", {r.S});
  const int32_t *cp = ints(counts, "counts", r.d), *tp = ints(tokens, "tokens", r.d);
  const long k = PyLong_AsLong(a[4]);
  if (k == -1 && PyErr_Occurred()) throw Refused{nullptr, ""};
  const bool add = truth(a[10]);
  at::Tensor out;
  int64_t ldg = r.E;
  if (is_none(a[9])) {
    if (add) value_error("accumulate needs the out to add to");
  } else {
    out = tensor(a[9], "out");
    shaped(out, "out", {r.T, r.E});
    beside(out, "out", r.d);
    if (out.scalar_type() != l.scalar_type()) type_error("out must be ", l.scalar_type(), ", got ", out.scalar_type());
    ldg = pitch(out, "out");
  }
  on_cuda(l);
  Launch on(r.d);
  if (!out.defined()) out = make({r.T, r.E}, l.scalar_type(), r.d);
  const int rc = moe_balance_loss_backward(r.T, r.E, k < 0 || k > 1024 ? -1 : (int)k, r.S, static_cast<const float*>(g.data_ptr()),
                                           r.logits, r.ld, r.type, cp, tp, r.offsets, r.mask, r.score, r.coef,
                                           out.data_ptr(), ldg, add, on.stream);
  if (rc != MOE_OK) return PyLong_FromLong(rc);
  return wrap(out);
}

#define MOE_METHOD(name, n) {#name, (PyCFunction)(void (*)(void))entry<name, n>, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {MOE_METHOD(quant_fp8, 10), MOE_METHOD(gemm_fp8, 8), MOE_METHOD(balance_loss, 7),
                         MOE_METHOD(balance_loss_backward, 11), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_moe_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__moe_ops(void) { return PyModule_Create(&module); }
