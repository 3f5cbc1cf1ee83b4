// Host side of the calls whose launch takes longer to describe than to run: the argument checks, the output
// allocations and the C ABI call of the residual norms and the gated projections in one native function each.
//
// Every function answers None where an argument is not what the kernels take (another type, host memory, a wrong
// shape, a size too small, an argument that the library refuses): the caller then takes its own path, which names
// the argument in its error.  Nothing has been launched in that case.  A failed launch is answered with the
// library's code instead: a kernel may have been queued before it, so the call must not be made again.  Four tokens of 7168 columns: 12.4 us per call with
// the checks and the allocations in Python.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/bsfp8.h"

namespace {

// The positional arguments of a call, taken in order; `ok` turns false at the first that does not fit.
struct Args {
  PyObject* const* at;
  Py_ssize_t left;
  bool ok = true;

  PyObject* next() {
    if (left <= 0) {
      ok = false;
      return Py_None;
    }
    --left;
    return *at++;
  }
  int64_t integer() {
    const long long v = PyLong_AsLongLong(next());
    if (v == -1 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return v;
  }
  double number() {
    const double v = PyFloat_AsDouble(next());
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return v;
  }
  bool truth() {
    const int v = PyObject_IsTrue(next());
    if (v < 0) {
      PyErr_Clear();
      ok = false;
    }
    return v == 1;
  }
  // a contiguous device tensor of one of two element types, or nullptr for None
  const at::Tensor* tensor(at::ScalarType a, at::ScalarType b) {
    PyObject* o = next();
    if (o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || (t.scalar_type() != a && t.scalar_type() != b) || !t.is_contiguous()) ok = false;
    return &t;
  }
  const at::Tensor* tensor(at::ScalarType a) { return tensor(a, a); }
  // the same with at least `bytes` bytes
  const at::Tensor* buffer(at::ScalarType a, at::ScalarType b, int64_t bytes) {
    const at::Tensor* t = tensor(a, b);
    if (t != nullptr && ok && (int64_t)t->nbytes() < bytes) ok = false;
    return t;
  }
  const at::Tensor* bytes(int64_t n) { return buffer(at::kByte, at::kByte, n); }
};

void* ptr(const at::Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }
bool shaped(const at::Tensor* t, int64_t n) { return t == nullptr || (t->dim() == 1 && t->size(0) == n); }
bool shaped(const at::Tensor* t, int64_t r, int64_t c) {
  return t == nullptr || (t->dim() == 2 && t->size(0) == r && t->size(1) == c);
}
int64_t gate_size(int kind, int64_t rows, int64_t cols) { return kind == BSFP8_GATE_TOKEN ? rows : cols; }

// An output: the tensor given, or a new one (kept in `own`) where `wanted`.
struct Out {
  const at::Tensor* given;
  at::Tensor own;
  bool wanted;
  template <class New>
  void* get(New make) {
    if (given == nullptr && wanted) {
      own = make();
      given = &own;
    }
    return ptr(given);
  }
  PyObject* object() const {
    if (given == nullptr) Py_RETURN_NONE;
    return THPVariable_Wrap(*given);
  }
};

// What a call that returned an error answers.
PyObject* refused(int rc) {
  if (rc == BSFP8_ERR_LAUNCH) return PyLong_FromLong(rc);
  Py_RETURN_NONE;
}

constexpr at::ScalarType F32 = at::kFloat, BF16 = at::kBFloat16;

// (x, y, post_weight, pre_weight, gate, gate_kind, x_scale, y_scale, eps, weight_offset, r, n, rstd_y, rstd_r,
// stream) -> (r, n, rstd_y, rstd_r)
PyObject* residual_norm(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  Args a{argv, argc};
  const at::Tensor* x = a.tensor(F32, BF16);
  const at::Tensor* y = a.tensor(BF16, at::kShort);
  const at::Tensor *post = a.tensor(F32), *pre = a.tensor(F32), *gate = a.tensor(F32);
  const int kind = (int)a.integer();
  const float xs = (float)a.number(), ys = (float)a.number(), eps = (float)a.number(), off = (float)a.number();
  if (!a.ok || x == nullptr || x->dim() != 2) Py_RETURN_NONE;
  Out r{a.tensor(x->scalar_type()), {}, true}, n{a.tensor(BF16, at::kShort), {}, pre != nullptr};
  Out ry{a.tensor(F32), {}, post != nullptr}, rr{a.tensor(F32), {}, pre != nullptr};
  const int64_t stream = a.integer(), rows = x->size(0), cols = x->size(1);
  if (!a.ok || a.left != 0 || !shaped(y, rows, cols) || !shaped(post, cols) || !shaped(pre, cols) ||
      !shaped(gate, gate_size(kind, rows, cols)) || !shaped(r.given, rows, cols) || !shaped(n.given, rows, cols) ||
      !shaped(ry.given, rows) || !shaped(rr.given, rows))
    Py_RETURN_NONE;
  const auto row = [&] { return at::empty({rows}, x->options().dtype(F32)); };
  void* pr = r.get([&] { return at::empty_like(*x); });
  void* pn = n.get([&] { return at::empty({rows, cols}, x->options().dtype(BF16)); });
  float *py = (float*)ry.get(row), *prr = (float*)rr.get(row);
  const int rc = bsfp8_residual_norm(rows, cols, ptr(x), x->scalar_type() == F32 ? BSFP8_F32 : BSFP8_BF16, ptr(y),
                                     (const float*)ptr(post), (const float*)ptr(pre), (const float*)ptr(gate), kind, xs,
                                     ys, eps, off, pr, pn, py, prr, (void*)stream);
  if (rc != BSFP8_OK) return refused(rc);
  return Py_BuildValue("(NNNN)", r.object(), n.object(), ry.object(), rr.object());
}

// (dn, dr, r, rstd_r, pre_weight, y, rstd_y, post_weight, gate, gate_kind, x_scale, y_scale, weight_offset, dx, dy,
// dpre_weight, dpost_weight, dgate, accumulate, workspace, stream) -> (dx, dy, dpre_weight, dpost_weight, dgate)
PyObject* residual_norm_grad(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  Args a{argv, argc};
  const at::Tensor *dn = a.tensor(BF16, at::kShort), *dr = a.tensor(F32, BF16), *r = a.tensor(F32, BF16);
  const at::Tensor *rr = a.tensor(F32), *pre = a.tensor(F32), *y = a.tensor(BF16, at::kShort), *ry = a.tensor(F32);
  const at::Tensor *post = a.tensor(F32), *gate = a.tensor(F32);
  const int kind = (int)a.integer();
  const float xs = (float)a.number(), ys = (float)a.number(), off = (float)a.number();
  const at::Tensor* ref = dr != nullptr ? dr : r;
  if (!a.ok || ref == nullptr || ref->dim() != 2) Py_RETURN_NONE;
  const at::ScalarType type = ref->scalar_type();
  Out dx{a.tensor(type), {}, true}, dy{a.tensor(BF16, at::kShort), {}, y != nullptr};
  Out dpre{a.tensor(F32), {}, pre != nullptr}, dpost{a.tensor(F32), {}, post != nullptr};
  Out dgate{a.tensor(F32), {}, gate != nullptr};
  const int accumulate = a.truth();
  const int64_t rows = ref->size(0), cols = ref->size(1), need = bsfp8_residual_norm_grad_workspace_bytes(rows, cols);
  PyObject* ws = a.next();
  at::Tensor work;
  if (ws == Py_None) {
    work = at::empty({need}, ref->options().dtype(at::kByte));
  } else {
    if (!THPVariable_Check(ws)) Py_RETURN_NONE;
    work = THPVariable_Unpack(ws);
    if (!work.is_cuda() || !work.is_contiguous() || (int64_t)work.nbytes() < need) Py_RETURN_NONE;
  }
  const int64_t stream = a.integer(), gates = gate_size(kind, rows, cols);
  const bool given = (pre == nullptr || dpre.given != nullptr) && (post == nullptr || dpost.given != nullptr) &&
                     (gate == nullptr || kind != BSFP8_GATE_CHANNEL || dgate.given != nullptr);
  if (!a.ok || a.left != 0 || (accumulate && !given) || (r != nullptr && r->scalar_type() != type) ||
      !shaped(dn, rows, cols) || !shaped(dr, rows, cols) || !shaped(r, rows, cols) || !shaped(y, rows, cols) ||
      !shaped(rr, rows) || !shaped(ry, rows) || !shaped(pre, cols) || !shaped(post, cols) || !shaped(gate, gates) ||
      !shaped(dx.given, rows, cols) || !shaped(dy.given, rows, cols) || !shaped(dpre.given, cols) ||
      !shaped(dpost.given, cols) || !shaped(dgate.given, gates))
    Py_RETURN_NONE;
  const auto like = [](const at::Tensor* t) { return [t] { return at::empty_like(*t); }; };
  void *pdx = dx.get(like(ref)), *pdy = dy.get(like(y));
  float *pp = (float*)dpre.get(like(pre)), *pq = (float*)dpost.get(like(post)), *pg = (float*)dgate.get(like(gate));
  const int rc = bsfp8_residual_norm_grad(
      rows, cols, type == F32 ? BSFP8_F32 : BSFP8_BF16, ptr(dn), ptr(dr), ptr(r), (const float*)ptr(rr),
      (const float*)ptr(pre), ptr(y), (const float*)ptr(ry), (const float*)ptr(post), (const float*)ptr(gate), kind, xs,
      ys, off, pdx, pdy, pp, pq, pg, accumulate, work.data_ptr(), (void*)stream);
  if (rc != BSFP8_OK) return refused(rc);
  return Py_BuildValue("(NNNNN)", dx.object(), dy.object(), dpre.object(), dpost.object(), dgate.object());
}

// The four quantized outputs of a gated projection [rows, cols] (None where a layout is not asked for).
struct Quantized {
  int which = 0;
  const at::Tensor *row_q, *row_s, *col_q, *col_s;
  Quantized(Args& a, int64_t rows, int64_t cols, int64_t groups) {
    const int64_t bound = rows > 0 ? bsfp8_colwise_rows_bound(rows, (int32_t)groups) : 0;
    row_q = a.bytes(rows * cols);
    row_s = a.bytes(rows * cols / 32);
    col_q = a.bytes(cols * bound);
    col_s = a.bytes(cols * bound / 32);
    which = (row_q != nullptr ? BSFP8_ROWWISE : 0) | (col_q != nullptr ? BSFP8_COLWISE : 0);
  }
};

// (x row_q, x row_s, rows, hidden, w row_q, w row_s, ffn, splits, recipe, y_dtype, probs, ab, y, four outputs, status,
// stream) -> True
PyObject* swiglu(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  Args a{argv, argc};
  if (argc != 19) Py_RETURN_NONE;
  // sizes first: they say how large the tensors have to be
  const auto size = [&](int i) {
    Args one{argv + i, 1};
    const int64_t v = one.integer();
    a.ok = a.ok && one.ok && v >= 0 && v <= (int64_t(1) << 40);
    return v;
  };
  const int64_t R = size(2), H = size(3), F = size(6);
  if (!a.ok || !THPVariable_Check(argv[7]) || H > (1 << 24) || F > (1 << 24) || R > (int64_t(1) << 31)) Py_RETURN_NONE;
  const int64_t E = THPVariable_Unpack(argv[7]).numel();
  if (E > BSFP8_MAX_GROUPS) Py_RETURN_NONE;
  const at::Tensor *xq = a.bytes(R * H), *xs = a.bytes(R * H / 32);
  a.next(), a.next();
  const at::Tensor *wq = a.bytes(E * 2 * F * H), *ws = a.bytes(E * 2 * F * H / 32);
  a.next();
  const at::Tensor* splits = a.tensor(at::kInt);
  const int recipe = (int)a.integer(), y_dtype = (int)a.integer();
  const bool f32 = y_dtype == BSFP8_OUT_F32;
  const at::Tensor* probs = a.buffer(F32, F32, R * 4);
  const at::Tensor* ab = a.buffer(BF16, at::kShort, R * F * 4);
  const at::Tensor* y = f32 ? a.buffer(F32, at::kInt, R * F * 4) : a.buffer(BF16, at::kShort, R * F * 2);
  const Quantized q(a, R, F, E);
  const at::Tensor* status = a.tensor(at::kInt);
  const int64_t stream = a.integer();
  if (!a.ok) Py_RETURN_NONE;
  const int rc = bsfp8_grouped_gemm_swiglu(
      (const uint8_t*)ptr(xq), (const uint8_t*)ptr(xs), R, H, (const uint8_t*)ptr(wq), (const uint8_t*)ptr(ws), F,
      (const float*)ptr(probs), (const int32_t*)ptr(splits), (int32_t)E, recipe, ptr(ab), ptr(y), y_dtype, q.which,
      (uint8_t*)ptr(q.row_q), (uint8_t*)ptr(q.row_s), (uint8_t*)ptr(q.col_q), (uint8_t*)ptr(q.col_s),
      (uint32_t*)ptr(status), (void*)stream);
  if (rc != BSFP8_OK) return refused(rc);
  Py_RETURN_TRUE;
}

// (dy row_q, dy row_s, rows, hidden, w col_q, w col_s, ffn, splits, recipe, ab, probs, dab, four outputs, dprobs,
// workspace, status, stream) -> True
PyObject* swiglu_grad(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  Args a{argv, argc};
  if (argc != 20) Py_RETURN_NONE;
  const auto size = [&](int i) {
    Args one{argv + i, 1};
    const int64_t v = one.integer();
    a.ok = a.ok && one.ok && v >= 0 && v <= (int64_t(1) << 40);
    return v;
  };
  const int64_t R = size(2), H = size(3), F = size(6);
  if (!a.ok || !THPVariable_Check(argv[7]) || H > (1 << 24) || F > (1 << 24) || R > (int64_t(1) << 31)) Py_RETURN_NONE;
  const int64_t E = THPVariable_Unpack(argv[7]).numel(), HP = (H + 127) / 128 * 128;
  if (E > BSFP8_MAX_GROUPS) Py_RETURN_NONE;
  const at::Tensor *dq = a.bytes(R * H), *ds = a.bytes(R * H / 32);
  a.next(), a.next();
  const at::Tensor *wq = a.bytes(F * E * HP), *ws = a.bytes(F * E * HP / 32);
  a.next();
  const at::Tensor* splits = a.tensor(at::kInt);
  const int recipe = (int)a.integer();
  const at::Tensor *ab = a.buffer(BF16, at::kShort, R * F * 4), *probs = a.buffer(F32, F32, R * 4);
  const at::Tensor* dab = a.buffer(BF16, at::kShort, R * F * 4);
  const Quantized q(a, R, 2 * F, E);
  const at::Tensor* dprobs = a.buffer(F32, F32, R * 4);
  const int64_t need = dprobs != nullptr ? (int64_t)bsfp8_grouped_gemm_swiglu_grad_workspace_bytes(R, F, (int32_t)E) : 0;
  PyObject* given = a.next();
  at::Tensor work;
  if (given != Py_None) {
    if (!THPVariable_Check(given)) Py_RETURN_NONE;
    work = THPVariable_Unpack(given);
    if (!work.is_cuda() || !work.is_contiguous() || (int64_t)work.nbytes() < need) Py_RETURN_NONE;
  }
  const at::Tensor* status = a.tensor(at::kInt);
  const int64_t stream = a.integer();
  if (!a.ok || splits == nullptr) Py_RETURN_NONE;
  if (!work.defined() && need > 0) work = at::empty({need}, splits->options().dtype(at::kByte));
  const int rc = bsfp8_grouped_gemm_swiglu_grad(
      (const uint8_t*)ptr(dq), (const uint8_t*)ptr(ds), R, H, (const uint8_t*)ptr(wq), (const uint8_t*)ptr(ws), F,
      ptr(ab), (const float*)ptr(probs), (const int32_t*)ptr(splits), (int32_t)E, recipe, ptr(dab), q.which,
      (uint8_t*)ptr(q.row_q), (uint8_t*)ptr(q.row_s), (uint8_t*)ptr(q.col_q), (uint8_t*)ptr(q.col_s),
      (float*)ptr(dprobs), work.defined() ? work.data_ptr() : nullptr, (uint32_t*)ptr(status), (void*)stream);
  if (rc != BSFP8_OK) return refused(rc);
  Py_RETURN_TRUE;
}

// A C++ exception (an allocation that fails) becomes None too: the caller's own path meets it again and reports it.
template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject* self, PyObject* const* argv, Py_ssize_t argc) {
  try {
    return F(self, argv, argc);
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

PyMethodDef kMethods[] = {
    {"residual_norm", (PyCFunction)(void (*)())guarded<residual_norm>, METH_FASTCALL, nullptr},
    {"residual_norm_grad", (PyCFunction)(void (*)())guarded<residual_norm_grad>, METH_FASTCALL, nullptr},
    {"swiglu", (PyCFunction)(void (*)())guarded<swiglu>, METH_FASTCALL, nullptr},
    {"swiglu_grad", (PyCFunction)(void (*)())guarded<swiglu_grad>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&kModule); }
