// Host side of the calls whose launch takes longer to describe than to run: the argument checks, the output
// allocations and the C ABI call of the residual norms, the gated projections and the tokens' way to their experts and
// back in one native function each.
//
// Every function answers None where an argument is not what the kernels take (another type, host memory, a wrong
// shape, a size too small, an argument that the library refuses): the caller then takes its own path, which names
// the argument in its error.  Nothing has been launched in that case.  A failed launch is answered with the
// library's code instead: a kernel may have been queued before it, so the call must not be made again.  Four tokens of
// 7168 columns: 12.4 us per call of the norms with the checks and the allocations in Python; four tokens' choices sorted
// 16.8 us there, 7.7 here, their rows' sum 10.1 and 4.9.
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
  int64_t device = -1;  // that tensors have to be on, where given

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
    if (!t.is_cuda() || (t.scalar_type() != a && t.scalar_type() != b) || !t.is_contiguous() ||
        (device >= 0 && t.get_device() != device))
      ok = false;
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

// The calls below begin with (current device, stream).
struct Call : Args {
  int64_t stream;
  Call(PyObject* const* argv, Py_ssize_t argc) : Args{argv, argc} {
    device = integer();
    stream = integer();
    if (device < 0) ok = false;
  }
  // a tensor that has to be there, [rows, cols]
  const at::Tensor* matrix(at::ScalarType a, at::ScalarType b) {
    const at::Tensor* t = tensor(a, b);
    if (t == nullptr || t->dim() != 2) ok = false;
    return ok ? t : nullptr;
  }
  // a workspace of at least `bytes` bytes: the tensor given, or a new one like `ref`
  at::Tensor workspace(int64_t bytes, const at::Tensor* ref) {
    PyObject* o = next();
    if (o == Py_None) return ok && bytes > 0 ? at::empty({bytes}, ref->options().dtype(at::kByte)) : at::Tensor();
    if (!THPVariable_Check(o)) {
      ok = false;
      return {};
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || !t.is_contiguous() || (int64_t)t.nbytes() < bytes || t.get_device() != device) ok = false;
    return t;
  }
  bool done() const { return ok && left == 0; }
};
void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
int dtype_of(const at::Tensor* t) { return t->scalar_type() == F32 ? BSFP8_F32 : BSFP8_BF16; }
constexpr at::ScalarType I32 = at::kInt, U8 = at::kByte;

// (.., logits, top_k, scoring, bias, renormalize, scale, probs, experts, score_sum, workspace) -> (probs, experts)
PyObject* route_topk(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  Call a(argv, argc);
  const at::Tensor* logits = a.matrix(F32, BF16);
  const int64_t K = a.integer(), scoring = a.integer();
  const at::Tensor* bias = a.tensor(F32);
  const int renormalize = a.truth();
  const float scale = (float)a.number();
  Out probs{a.tensor(F32), {}, true}, experts{a.tensor(I32), {}, true};
  const at::Tensor* sum = a.tensor(F32);
  if (!a.ok || K < 1 || K > BSFP8_MAX_TOP_K) Py_RETURN_NONE;
  const int64_t T = logits->size(0), E = logits->size(1);
  if (E > BSFP8_MAX_GROUPS) Py_RETURN_NONE;
  const at::Tensor work =
      a.workspace(sum != nullptr ? (int64_t)bsfp8_route_topk_workspace_bytes(T, (int32_t)E) : 0, logits);
  if (!a.done() || !shaped(bias, E) || !shaped(sum, E) || !shaped(probs.given, T, K) || !shaped(experts.given, T, K))
    Py_RETURN_NONE;
  float* pp = (float*)probs.get([&] { return at::empty({T, K}, logits->options().dtype(F32)); });
  int32_t* pe = (int32_t*)experts.get([&] { return at::empty({T, K}, logits->options().dtype(I32)); });
  const int rc = bsfp8_route_topk(ptr(logits), dtype_of(logits), T, (int32_t)E, (int32_t)K, (int)scoring,
                                  (const float*)ptr(bias), renormalize, scale, pp, pe, (float*)ptr(sum),
                                  sum != nullptr ? ptr(work) : nullptr, (void*)a.stream);
  if (rc != BSFP8_OK) return refused(rc);
  return Py_BuildValue("(NN)", probs.object(), experts.object());
}

// (.., dprobs, logits, experts, scoring, renormalize, scale, dscore_sum, dlogits) -> (dlogits,)
PyObject* route_topk_grad(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  Call a(argv, argc);
  const at::Tensor *dprobs = a.matrix(F32, F32), *logits = a.matrix(F32, BF16), *experts = a.matrix(I32, I32);
  const int64_t scoring = a.integer();
  const int renormalize = a.truth();
  const float scale = (float)a.number();
  const at::Tensor* dsum = a.tensor(F32);
  if (!a.ok) Py_RETURN_NONE;
  Out dl{a.tensor(logits->scalar_type()), {}, true};
  const int64_t T = logits->size(0), E = logits->size(1), K = experts->size(1);
  if (!a.done() || E > BSFP8_MAX_GROUPS || K > BSFP8_MAX_TOP_K || !shaped(dprobs, T, K) || !shaped(experts, T, K) ||
      !shaped(dsum, E) || !shaped(dl.given, T, E))
    Py_RETURN_NONE;
  void* out = dl.get([&] { return at::empty_like(*logits); });
  const int rc = bsfp8_route_topk_grad((const float*)ptr(dprobs), ptr(logits), dtype_of(logits),
                                       (const int32_t*)ptr(experts), T, (int32_t)E, (int32_t)K, (int)scoring, renormalize,
                                       scale, (const float*)ptr(dsum), out, (void*)a.stream);
  if (rc != BSFP8_OK) return refused(rc);
  return Py_BuildValue("(N)", dl.object());
}

// (.., experts, num_experts, probs, splits, rows, choices, row probs, workspace) -> (splits, rows, choices, row probs)
PyObject* dispatch_plan(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  Call a(argv, argc);
  const at::Tensor* experts = a.matrix(I32, I32);
  const int64_t E = a.integer();
  const at::Tensor* probs = a.tensor(F32);
  Out splits{a.tensor(I32), {}, true}, rows{a.tensor(I32), {}, true}, choices{a.tensor(I32), {}, true};
  Out row_probs{a.tensor(F32), {}, probs != nullptr};
  if (!a.ok || E < 1 || E > BSFP8_MAX_GROUPS) Py_RETURN_NONE;
  const int64_t T = experts->size(0), K = experts->size(1);
  if (K < 1 || K > BSFP8_MAX_TOP_K) Py_RETURN_NONE;
  const int64_t N = T * K;
  const at::Tensor work =
      a.workspace((int64_t)bsfp8_dispatch_plan_workspace_bytes(T, (int32_t)K, (int32_t)E), experts);
  if (!a.done() || !shaped(probs, T, K) || !shaped(splits.given, E) || !shaped(rows.given, T, K) ||
      !shaped(choices.given, N) || !shaped(row_probs.given, N) || (probs == nullptr && row_probs.given != nullptr))
    Py_RETURN_NONE;
  const auto whole = [&](int64_t n) { return [&, n] { return at::empty({n}, experts->options()); }; };
  int32_t *ps = (int32_t*)splits.get(whole(E)), *pr = (int32_t*)rows.get([&] { return at::empty_like(*experts); });
  int32_t* pc = (int32_t*)choices.get(whole(N));
  float* pp = (float*)row_probs.get([&] { return at::empty({N}, probs->options()); });
  const int rc = bsfp8_dispatch_plan((const int32_t*)ptr(experts), (const float*)ptr(probs), T, (int32_t)K, (int32_t)E, ps,
                                     pr, pc, pp, ptr(work), (void*)a.stream);
  if (rc != BSFP8_OK) return refused(rc);
  return Py_BuildValue("(NNNN)", splits.object(), rows.object(), choices.object(), row_probs.object());
}

// (.., x, rows, weights, out) -> (out,)
PyObject* dispatch(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  Call a(argv, argc);
  const at::Tensor *x = a.matrix(F32, BF16), *rows = a.matrix(I32, I32), *weights = a.tensor(F32);
  if (!a.ok) Py_RETURN_NONE;
  Out out{a.tensor(x->scalar_type()), {}, true};
  const int64_t T = rows->size(0), K = rows->size(1), C = x->size(1), N = T * K;
  if (!a.done() || K > BSFP8_MAX_TOP_K || !shaped(x, T, C) || !shaped(weights, T, K) || !shaped(out.given, N, C))
    Py_RETURN_NONE;
  void* po = out.get([&] { return at::empty({N, C}, x->options()); });
  const int rc = bsfp8_dispatch(ptr(x), dtype_of(x), T, C, (const int32_t*)ptr(rows), (int32_t)K, (const float*)ptr(weights),
                                po, N, (void*)a.stream);
  if (rc != BSFP8_OK) return refused(rc);
  return Py_BuildValue("(N)", out.object());
}

// Quantized buffers of a [rows, cols] operand with an MX recipe, as large as `which` asks for.
struct MxBuffers {
  const at::Tensor *row_q, *row_s, *col_q, *col_s;
  MxBuffers(Args& a, int64_t recipe, int64_t which, int64_t rows, int64_t cols, int64_t groups) {
    const bool row = which & BSFP8_ROWWISE, col = which & BSFP8_COLWISE;
    if ((recipe != BSFP8_RECIPE_MX_1X32_E8M0 && recipe != BSFP8_RECIPE_MXFP4_1X32_E8M0) || groups < 1 ||
        groups > BSFP8_MAX_GROUPS || cols > (1 << 24) || rows > (int64_t(1) << 31))
      a.ok = false;
    row_q = a.bytes(row && a.ok ? (int64_t)bsfp8_rowwise_data_bytes(rows, cols, (int)recipe) : 0);
    row_s = a.bytes(row && a.ok ? (int64_t)bsfp8_rowwise_scale_bytes(rows, cols) : 0);
    col_q = a.bytes(col && a.ok && rows > 0 ? (int64_t)bsfp8_colwise_data_bytes(rows, cols, (int32_t)groups, (int)recipe) : 0);
    col_s = a.bytes(col && a.ok && rows > 0 ? (int64_t)bsfp8_colwise_scale_bytes(rows, cols, (int32_t)groups, (int)recipe) : 0);
  }
};

// (.., x, rows, choices, splits, recipe, which, four outputs, weights, status) -> True
PyObject* dispatch_quantize(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  Call a(argv, argc);
  const at::Tensor *x = a.matrix(BF16, at::kShort), *rows = a.matrix(I32, I32);
  const at::Tensor *choices = a.tensor(I32), *splits = a.tensor(I32);
  const int64_t recipe = a.integer(), which = a.integer();
  if (!a.ok || choices == nullptr || splits == nullptr) Py_RETURN_NONE;
  const int64_t T = rows->size(0), K = rows->size(1), C = x->size(1), N = T * K, E = splits->numel();
  const MxBuffers q(a, recipe, which, N, C, E);
  const at::Tensor *weights = a.tensor(F32), *status = a.tensor(I32);
  if (!a.done() || K > BSFP8_MAX_TOP_K || !shaped(x, T, C) || !shaped(choices, N) || !shaped(weights, T, K)) Py_RETURN_NONE;
  const int rc = bsfp8_dispatch_quantize(
      ptr(x), T, C, (const int32_t*)ptr(choices), (int32_t)K, (const float*)ptr(weights), N, (const int32_t*)ptr(splits),
      (int32_t)E, (int)recipe, (int)which, (uint8_t*)ptr(q.row_q), (uint8_t*)ptr(q.row_s), (uint8_t*)ptr(q.col_q),
      (uint8_t*)ptr(q.col_s), (uint32_t*)ptr(status), (void*)a.stream);
  if (rc != BSFP8_OK) return refused(rc);
  Py_RETURN_TRUE;
}

// (.., y, rows, weights, add, out) -> (out,)
PyObject* combine(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  Call a(argv, argc);
  const at::Tensor *y = a.matrix(F32, BF16), *rows = a.matrix(I32, I32), *weights = a.tensor(F32);
  if (!a.ok) Py_RETURN_NONE;
  const at::Tensor* add = a.tensor(y->scalar_type());
  Out out{a.tensor(y->scalar_type()), {}, true};
  const int64_t T = rows->size(0), K = rows->size(1), C = y->size(1), N = T * K;
  if (!a.done() || K > BSFP8_MAX_TOP_K || !shaped(y, N, C) || !shaped(weights, T, K) || !shaped(add, T, C) ||
      !shaped(out.given, T, C))
    Py_RETURN_NONE;
  void* po = out.get([&] { return at::empty({T, C}, y->options()); });
  const int rc = bsfp8_combine(ptr(y), dtype_of(y), N, C, (const int32_t*)ptr(rows), T, (int32_t)K,
                               (const float*)ptr(weights), ptr(add), po, (void*)a.stream);
  if (rc != BSFP8_OK) return refused(rc);
  return Py_BuildValue("(N)", out.object());
}

// (.., dout, rows, y, weights, dy, whether dy is wanted, dweights) -> (dy, dweights)
PyObject* combine_grad(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  Call a(argv, argc);
  const at::Tensor *dout = a.matrix(F32, BF16), *rows = a.matrix(I32, I32);
  if (!a.ok) Py_RETURN_NONE;
  const at::ScalarType type = dout->scalar_type();
  const at::Tensor *y = a.tensor(type), *weights = a.tensor(F32);
  Out dy{a.tensor(type), {}, false};
  dy.wanted = a.truth();
  Out dw{a.tensor(F32), {}, weights != nullptr && y != nullptr};
  const int64_t T = rows->size(0), K = rows->size(1), C = dout->size(1), N = T * K;
  if (!a.done() || K > BSFP8_MAX_TOP_K || !shaped(dout, T, C) || !shaped(y, N, C) || !shaped(weights, T, K) ||
      !shaped(dy.given, N, C) || !shaped(dw.given, T, K) || (dw.given != nullptr && y == nullptr))
    Py_RETURN_NONE;
  void* pd = dy.get([&] { return at::empty({N, C}, dout->options()); });
  float* pw = (float*)dw.get([&] { return at::empty({T, K}, weights->options()); });
  const int rc = bsfp8_combine_grad(ptr(dout), dtype_of(dout), T, C, ptr(y), N, (const int32_t*)ptr(rows), (int32_t)K,
                                    (const float*)ptr(weights), pd, pw, (void*)a.stream);
  if (rc != BSFP8_OK) return refused(rc);
  return Py_BuildValue("(NN)", dy.object(), dw.object());
}

// (.., activation, h, probs, splits, recipe, which, four outputs, kept row_q, kept row_s, status) -> True
PyObject* act_checkpoint(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  Call a(argv, argc);
  const int64_t act = a.integer();
  const at::Tensor *h = a.matrix(BF16, at::kShort), *probs = a.tensor(F32), *splits = a.tensor(I32);
  const int64_t recipe = a.integer(), which = a.integer();
  if (!a.ok || splits == nullptr || (act != BSFP8_ACT_SRELU && act != BSFP8_ACT_SWIGLU)) Py_RETURN_NONE;
  const int64_t R = h->size(0), wide = h->size(1), F = act == BSFP8_ACT_SWIGLU ? wide / 2 : wide, E = splits->numel();
  const MxBuffers q(a, recipe, which, R, F, E);
  const at::Tensor *kq = a.bytes(R * wide), *ks = a.bytes(R * wide / 32), *status = a.tensor(I32);
  if (!a.done() || !shaped(probs, R) || (act == BSFP8_ACT_SWIGLU && wide % 2)) Py_RETURN_NONE;
  const int rc = bsfp8_grouped_act_checkpoint(
      (int)act, ptr(h), (const float*)ptr(probs), R, F, (const int32_t*)ptr(splits), (int32_t)E, (int)recipe, (int)which,
      (uint8_t*)ptr(q.row_q), (uint8_t*)ptr(q.row_s), (uint8_t*)ptr(q.col_q), (uint8_t*)ptr(q.col_s), (uint8_t*)ptr(kq),
      (uint8_t*)ptr(ks), (uint32_t*)ptr(status), (void*)a.stream);
  if (rc != BSFP8_OK) return refused(rc);
  Py_RETURN_TRUE;
}

// (.., activation, kept row_q, kept row_s, dy, probs, splits, recipe, which, four outputs, y col_q, y col_s, dprobs, workspace,
// status) -> True
PyObject* act_checkpoint_grad(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  Call a(argv, argc);
  const int64_t act = a.integer();
  const at::Tensor *kq = a.tensor(U8), *ks = a.tensor(U8);
  const at::Tensor *dy = a.matrix(BF16, at::kShort), *probs = a.tensor(F32), *splits = a.tensor(I32);
  const int64_t recipe = a.integer(), which = a.integer();
  if (!a.ok || splits == nullptr || kq == nullptr || ks == nullptr || (act != BSFP8_ACT_SRELU && act != BSFP8_ACT_SWIGLU))
    Py_RETURN_NONE;
  const int64_t R = dy->size(0), F = dy->size(1), wide = act == BSFP8_ACT_SWIGLU ? 2 * F : F, E = splits->numel();
  const MxBuffers q(a, recipe, which, R, wide, E);
  const int64_t bound = R > 0 ? bsfp8_colwise_rows_bound(R, (int32_t)E) / (recipe == BSFP8_RECIPE_MXFP4_1X32_E8M0 ? 2 : 1) : 0;
  const at::Tensor *yq = a.bytes(F * bound), *ys = a.bytes(R > 0 ? F * (bsfp8_colwise_rows_bound(R, (int32_t)E) / 32) : 0);
  const at::Tensor* dprobs = a.tensor(F32);
  const at::Tensor work =
      a.workspace(dprobs != nullptr ? (int64_t)bsfp8_grouped_act_checkpoint_grad_workspace_bytes(R, F) : 0, dy);
  const at::Tensor* status = a.tensor(I32);
  if (!a.done() || !shaped(probs, R) || !shaped(dprobs, R) || (int64_t)kq->nbytes() < R * wide ||
      (int64_t)ks->nbytes() < R * wide / 32)
    Py_RETURN_NONE;
  const int rc = bsfp8_grouped_act_checkpoint_grad(
      (int)act, (const uint8_t*)ptr(kq), (const uint8_t*)ptr(ks), (const float*)ptr(probs), ptr(dy), R, F,
      (const int32_t*)ptr(splits), (int32_t)E, (int)recipe, (int)which, (uint8_t*)ptr(q.row_q), (uint8_t*)ptr(q.row_s),
      (uint8_t*)ptr(q.col_q), (uint8_t*)ptr(q.col_s), (uint8_t*)ptr(yq), (uint8_t*)ptr(ys), (float*)ptr(dprobs),
      dprobs != nullptr ? ptr(work) : nullptr, (uint32_t*)ptr(status), (void*)a.stream);
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
    {"route_topk", (PyCFunction)(void (*)())guarded<route_topk>, METH_FASTCALL, nullptr},
    {"route_topk_grad", (PyCFunction)(void (*)())guarded<route_topk_grad>, METH_FASTCALL, nullptr},
    {"dispatch_plan", (PyCFunction)(void (*)())guarded<dispatch_plan>, METH_FASTCALL, nullptr},
    {"dispatch", (PyCFunction)(void (*)())guarded<dispatch>, METH_FASTCALL, nullptr},
    {"dispatch_quantize", (PyCFunction)(void (*)())guarded<dispatch_quantize>, METH_FASTCALL, nullptr},
    {"combine", (PyCFunction)(void (*)())guarded<combine>, METH_FASTCALL, nullptr},
    {"combine_grad", (PyCFunction)(void (*)())guarded<combine_grad>, METH_FASTCALL, nullptr},
    {"act_checkpoint", (PyCFunction)(void (*)())guarded<act_checkpoint>, METH_FASTCALL, nullptr},
    {"act_checkpoint_grad", (PyCFunction)(void (*)())guarded<act_checkpoint_grad>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&kModule); }
