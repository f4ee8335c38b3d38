// Native marshalling for the calls that a serving or training loop makes most:
// the norm, the 8-bit base's forward and backward, and the AdamW step over many
// tensors. The Python binding's checks of one such call, its allocations and the
// conversion of its arguments take three to five times as long as the launch
// itself (norm of one row: 17 us in Python); here they take about one launch's
// time, and a list of 448 tensors 20 us instead of 450.
//
// Each function checks its arguments by the rules of the Python binding and
// returns
//   None    when any of them does not hold (or the case is not one of the plain
//           ones): the caller goes on in Python, which says what is wrong, or
//           does it
//   int     a status of the C ABI other than QLORA_OK
//   tuple   the results
// Nothing is enqueued before every check has passed.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>

#include <algorithm>
#include <cstdint>
#include <utility>
#include <vector>

#include "qlora.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Refused {};  // thrown to the entry point: this call is Python's

// A tensor argument, or an undefined one for None.
Tensor tensor(PyObject *o) {
  if (o == Py_None) return Tensor();
  if (!THPVariable_Check(o)) throw Refused{};
  return THPVariable_Unpack(o);
}
void need(bool ok) {
  if (!ok) throw Refused{};
}
template <typename T = void>
T *ptr(const Tensor &t) {
  return t.defined() ? static_cast<T *>(t.data_ptr()) : nullptr;
}
// Defined tensors lie on the current device `dev`.
void on(int dev, std::initializer_list<const Tensor *> ts) {
  for (const Tensor *t : ts)
    if (t->defined()) need(t->is_cuda() && t->get_device() == dev);
}
void is(const Tensor &t, ScalarType type, at::IntArrayRef shape) {
  if (t.defined()) need(t.scalar_type() == type && t.sizes() == shape && t.is_contiguous());
}
int float_type(const Tensor &t) {
  if (t.scalar_type() == at::kFloat) return QLORA_F32;
  need(t.scalar_type() == at::kBFloat16);
  return QLORA_BF16;
}
int64_t groups(int64_t d) { return (d + QLORA_FP8_GROUP - 1) / QLORA_FP8_GROUP; }
ScalarType fp8_type(int fmt) { return fmt == QLORA_E5M2 ? at::kFloat8_e5m2 : at::kFloat8_e4m3fn; }
Tensor empty(at::IntArrayRef shape, ScalarType type, const Tensor &like) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}
// Rows of `d` dense values, any row stride of at least d; the stride.
int64_t rows(const Tensor &t, ScalarType type, int64_t T, int64_t d) {
  if (!t.defined()) return d;
  need(t.scalar_type() == type && t.dim() == 2 && t.size(0) == T && t.size(1) == d);
  need((d == 1 || t.stride(1) == 1) && (T == 1 || t.stride(0) >= d));
  return T == 1 ? d : t.stride(0);
}

int64_t as_int(PyObject *o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused{};
  }
  return v;
}
double as_float(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused{};
  }
  return v;
}
bool as_bool(PyObject *o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    throw Refused{};
  }
  return v == 1;
}
hipStream_t as_stream(PyObject *o) { return reinterpret_cast<hipStream_t>(as_int(o)); }

PyObject *results(std::initializer_list<Tensor> ts) {
  PyObject *out = PyTuple_New((Py_ssize_t)ts.size());
  Py_ssize_t i = 0;
  for (const Tensor &t : ts) {
    PyObject *o = t.defined() ? THPVariable_Wrap(t) : (Py_INCREF(Py_None), Py_None);
    PyTuple_SET_ITEM(out, i++, o);
  }
  return out;
}
PyObject *answer(int status, std::initializer_list<Tensor> ts) {
  return status == QLORA_OK ? results(ts) : PyLong_FromLong(status);
}

#define QLORA_ENTRY(N)                 \
  HANDLE_TH_ERRORS                     \
  if (n != N) Py_RETURN_NONE;          \
  try {
#define QLORA_EXIT                     \
  }                                    \
  catch (const Refused &) {            \
    Py_RETURN_NONE;                    \
  }                                    \
  END_HANDLE_TH_ERRORS

// (x, weight, residual, eps, want_y, fmt or 0, save_rstd, device, stream) -> (y, yq, ys, s, rstd)
PyObject *rmsnorm_forward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  QLORA_ENTRY(9)
  const Tensor x = tensor(a[0]), w = tensor(a[1]), res = tensor(a[2]);
  const float eps = (float)as_float(a[3]);
  const bool want_y = as_bool(a[4]), save_rstd = as_bool(a[6]);
  const int fmt = (int)as_int(a[5]), dev = (int)as_int(a[7]);
  need(x.defined() && x.dim() == 2);
  const int dt = float_type(x);
  const ScalarType type = x.scalar_type();
  const int64_t T = x.size(0), d = x.size(1);
  need(T > 0 && d >= 1 && d <= QLORA_NORM_MAX_DIM && (want_y || fmt));
  const int64_t ldx = rows(x, type, T, d), ldr = rows(res, type, T, d);
  const int wd = w.defined() ? float_type(w) : QLORA_F32;
  if (w.defined()) is(w, w.scalar_type(), {d});
  on(dev, {&x, &w, &res});
  Tensor y, yq, ys, s, rstd;
  if (want_y) y = empty({T, d}, type, x);
  if (res.defined()) s = empty({T, d}, type, x);
  if (fmt) {
    yq = empty({T, d}, fp8_type(fmt), x);
    ys = empty({T, groups(d)}, at::kFloat, x);
  }
  if (save_rstd) rstd = empty({T}, at::kFloat, x);
  return answer(qlora_rmsnorm_forward(ptr(x), ldx, ptr(res), ldr, dt, T, d, ptr(w), wd, eps, ptr(s), ptr(y),
                                      ptr<uint8_t>(yq), ptr<float>(ys), fmt, ptr<float>(rstd), as_stream(a[8])),
                {y, yq, ys, s, rstd});
  QLORA_EXIT
}

// (dy, s, weight, rstd, ds, need_dw, device, stream) -> (dx, dw)
PyObject *rmsnorm_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  QLORA_ENTRY(8)
  const Tensor dy = tensor(a[0]), s = tensor(a[1]), w = tensor(a[2]), rstd = tensor(a[3]), ds = tensor(a[4]);
  const bool need_dw = as_bool(a[5]);
  const int dev = (int)as_int(a[6]);
  need(dy.defined() && s.defined() && rstd.defined() && s.dim() == 2);
  const int dt = float_type(s);
  const ScalarType type = s.scalar_type();
  const int64_t T = s.size(0), d = s.size(1);
  need(T > 0 && d >= 1 && d <= QLORA_NORM_MAX_DIM);
  const int64_t lds = rows(s, type, T, d), ldy = rows(dy, type, T, d), ldd = rows(ds, type, T, d);
  const int wd = w.defined() ? float_type(w) : QLORA_F32;
  if (w.defined()) is(w, w.scalar_type(), {d});
  is(rstd, at::kFloat, {T});
  on(dev, {&dy, &s, &w, &rstd, &ds});
  const Tensor dx = empty({T, d}, type, s);
  Tensor dw, ws;
  size_t bytes = 0;
  if (need_dw) {
    dw = empty({d}, at::kFloat, s);
    bytes = qlora_rmsnorm_workspace_bytes(T, d);
    ws = empty({(int64_t)bytes}, at::kByte, s);
  }
  return answer(qlora_rmsnorm_backward(ptr(dy), ldy, ptr(s), lds, ptr(ds), ldd, dt, T, d, ptr(w), wd, ptr<float>(rstd),
                                       ptr(dx), ptr<float>(dw), ptr(ws), bytes, as_stream(a[7])),
                {dx, dw});
  QLORA_EXIT
}

struct Base {
  Tensor codes, scales;
  qlora_fp8_weight w;
};
Base base(PyObject *codes, PyObject *scales, PyObject *d_out, PyObject *d_in) {
  Base b{tensor(codes), tensor(scales), {}};
  const int64_t N = as_int(d_out), K = as_int(d_in);
  need(b.codes.defined() && b.scales.defined() && N >= 16 && K >= 16 && N % 16 == 0 && K % 16 == 0);
  is(b.codes, at::kFloat8_e4m3fn, {N, K});
  is(b.scales, at::kFloat, {groups(N), groups(K)});
  b.w = qlora_fp8_weight{N, K, ptr<uint8_t>(b.codes), ptr<float>(b.scales)};
  return b;
}
int adapter_rank(const Tensor &A, const Tensor &B, int64_t N, int64_t K) {
  need(A.defined() == B.defined());
  if (!A.defined()) return 0;
  need(A.dim() == 2);
  const int64_t r = A.size(0);
  need(r <= QLORA_MAX_RANK && r % 8 == 0);
  is(A, at::kBFloat16, {r, K});
  is(B, at::kBFloat16, {N, r});
  return (int)r;
}
// The device's cached workspace, where it is large enough.
void workspace(const Tensor &ws, size_t bytes) { need(ws.defined() && (size_t)ws.numel() >= bytes); }

// (codes, scales, d_out, d_in, x, A, B, alpha, xq, xs, fmt, save_u, ws, device, stream) -> (h, u)
PyObject *fp8_forward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  QLORA_ENTRY(15)
  const Base b = base(a[0], a[1], a[2], a[3]);
  const int64_t N = b.w.d_out, K = b.w.d_in;
  const Tensor x = tensor(a[4]), A = tensor(a[5]), B = tensor(a[6]), xq = tensor(a[8]), xs = tensor(a[9]), ws = tensor(a[12]);
  const float alpha = (float)as_float(a[7]);
  const int fmt = (int)as_int(a[10]), dev = (int)as_int(a[13]);
  const bool save_u = as_bool(a[11]);
  need(xq.defined() == xs.defined());
  const Tensor &lead = x.defined() ? x : xq;
  need(lead.defined() && lead.dim() == 2 && lead.size(0) >= 1);
  const int64_t T = lead.size(0);
  is(x, at::kBFloat16, {T, K});
  is(xq, fp8_type(fmt), {T, K});
  is(xs, at::kFloat, {T, groups(K)});
  const int r = adapter_rank(A, B, N, K);
  need(r == 0 || x.defined());
  on(dev, {&b.codes, &b.scales, &x, &A, &B, &xq, &xs, &ws});
  workspace(ws, qlora_fp8_workspace_bytes(N, K, T, r));
  const Tensor h = empty({T, N}, at::kBFloat16, b.codes);
  Tensor u;
  if (save_u && r > 0) u = empty({T, r}, at::kFloat, b.codes);
  return answer(qlora_fp8_forward(&b.w, ptr<uint8_t>(xq), ptr<float>(xs), fmt, ptr<uint16_t>(x), T, ptr<uint16_t>(A),
                                  ptr<uint16_t>(B), r, alpha, ptr<uint16_t>(h), ptr<float>(u), ptr(ws),
                                  (size_t)ws.numel(), as_stream(a[14])),
                {h, u});
  QLORA_EXIT
}

// (codes, scales, d_out, d_in, x, dY, A, B, alpha, u, need_dx, need_dA, need_dB, fmt, ws, device, stream) -> (dX, dA, dB)
PyObject *fp8_backward(PyObject *, PyObject *const *a, Py_ssize_t n) {
  QLORA_ENTRY(17)
  const Base b = base(a[0], a[1], a[2], a[3]);
  const int64_t N = b.w.d_out, K = b.w.d_in;
  const Tensor x = tensor(a[4]), dY = tensor(a[5]), A = tensor(a[6]), B = tensor(a[7]), u = tensor(a[9]), ws = tensor(a[14]);
  const float alpha = (float)as_float(a[8]);
  const int fmt = (int)as_int(a[13]), dev = (int)as_int(a[15]);
  need(dY.defined() && dY.dim() == 2 && dY.size(0) >= 1);
  const int64_t T = dY.size(0);
  is(dY, at::kBFloat16, {T, N});
  is(x, at::kBFloat16, {T, K});
  const int r = adapter_rank(A, B, N, K);
  need(r > 0 || !u.defined());
  is(u, at::kFloat, {T, r});
  const bool need_dA = r > 0 && as_bool(a[11]), need_dB = r > 0 && as_bool(a[12]);
  need(x.defined() || !(need_dA || (need_dB && !u.defined())));
  on(dev, {&b.codes, &b.scales, &x, &dY, &A, &B, &u, &ws});
  workspace(ws, qlora_fp8_workspace_bytes(N, K, T, r));
  Tensor dX, dA, dB;
  if (as_bool(a[10])) dX = empty({T, K}, at::kBFloat16, b.codes);
  if (need_dA) dA = empty({r, K}, at::kFloat, b.codes);
  if (need_dB) dB = empty({N, r}, at::kFloat, b.codes);
  return answer(qlora_fp8_backward(&b.w, ptr<uint16_t>(x), ptr<uint16_t>(dY), fmt, T, ptr<uint16_t>(A), ptr<uint16_t>(B),
                                   r, alpha, ptr<float>(u), ptr<uint16_t>(dX), ptr<float>(dA), ptr<float>(dB), ptr(ws),
                                   (size_t)ws.numel(), as_stream(a[16])),
                {dX, dA, dB});
  QLORA_EXIT
}

// (step, grads, params, m, v, m_scale, v_scale, master, lr, beta1, beta2, eps, weight_decay, max_norm or 0, seed, norm,
//  device, stream) -> (norm,); grads and params are lists
PyObject *adamw_many(PyObject *, PyObject *const *a, Py_ssize_t n) {
  QLORA_ENTRY(18)
  const int64_t step = as_int(a[0]);
  need(PyList_Check(a[1]) && PyList_Check(a[2]));
  const Py_ssize_t count = PyList_GET_SIZE(a[1]);
  need(count >= 1 && count == PyList_GET_SIZE(a[2]));
  const Tensor m = tensor(a[3]), v = tensor(a[4]), ms = tensor(a[5]), vs = tensor(a[6]), master = tensor(a[7]);
  Tensor norm = tensor(a[15]);
  const qlora_adamw_many_hparams hp{as_float(a[8]), as_float(a[9]), as_float(a[10]), as_float(a[11]), as_float(a[12])};
  const float max_norm = (float)as_float(a[13]);
  const int64_t seed = as_int(a[14]);
  const int dev = (int)as_int(a[16]);
  need(m.defined() && v.defined() && seed >= 0 && seed < ((int64_t)1 << 32));
  need(max_norm > 0.f || as_float(a[13]) == 0.0);  // (0: no clipping; what float32 turns into 0 is refused)
  std::vector<qlora_adamw_job> jobs((size_t)count);
  std::vector<std::pair<uintptr_t, uintptr_t>> spans, reads;  // what is written; the gradients
  spans.reserve((size_t)count + 6);
  reads.reserve((size_t)count);
  int gd = -1, pd = -1;
  int64_t total = 0;
  for (Py_ssize_t i = 0; i < count; ++i) {
    PyObject *go = PyList_GET_ITEM(a[1], i), *po = PyList_GET_ITEM(a[2], i);
    need(THPVariable_Check(po));
    const Tensor &p = THPVariable_Unpack(po);
    const Tensor g = tensor(go);  // None: the tensor is left as it is
    const int pt = float_type(p);
    if (pd < 0) pd = pt;
    const int64_t size = p.numel();
    need(pt == pd && p.is_contiguous());
    if (g.defined()) {
      const int gt = float_type(g);
      if (gd < 0) gd = gt;
      need(gt == gd && g.numel() == size && g.is_contiguous());
      if (size) {
        const uintptr_t at = reinterpret_cast<uintptr_t>(g.data_ptr());
        reads.emplace_back(at, at + (uintptr_t)size * g.element_size());
      }
    }
    on(dev, {&g, &p});
    jobs[(size_t)i] = qlora_adamw_job{ptr(g), p.data_ptr(), size};
    if (size) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(p.data_ptr());
      spans.emplace_back(at, at + (uintptr_t)size * p.element_size());
    }
    total += (size + QLORA_ADAMW_BLOCK - 1) / QLORA_ADAMW_BLOCK * QLORA_ADAMW_BLOCK;
  }
  for (const Tensor *t : std::initializer_list<const Tensor *>{&m, &v, &ms, &vs, &master, &norm})
    if (t->defined() && t->numel()) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(t->data_ptr());
      spans.emplace_back(at, at + (uintptr_t)t->numel() * t->element_size());
    }
  std::sort(spans.begin(), spans.end());
  for (size_t i = 1; i < spans.size(); ++i) need(spans[i - 1].second <= spans[i].first);
  for (const auto &g : reads) {  // (gradients may overlap each other)
    const auto next = std::lower_bound(spans.begin(), spans.end(), std::make_pair(g.second, (uintptr_t)0));
    need(next == spans.begin() || (next - 1)->second <= g.first);
  }
  if (gd < 0) gd = QLORA_F32;
  const bool bits8 = m.scalar_type() == at::kFloat8_e4m3fn;
  need(bits8 || m.scalar_type() == at::kFloat);
  is(m, m.scalar_type(), {total});
  is(v, m.scalar_type(), {total});
  need(bits8 == ms.defined() && bits8 == vs.defined() && (pd == QLORA_BF16) == master.defined());
  is(ms, at::kFloat, {total / QLORA_ADAMW_BLOCK});
  is(vs, at::kFloat, {total / QLORA_ADAMW_BLOCK});
  is(master, at::kFloat, {total});
  is(norm, at::kFloat, {1});
  need(max_norm > 0.f || !norm.defined());
  on(dev, {&m, &v, &ms, &vs, &master, &norm});
  const qlora_adamw_state st{bits8 ? QLORA_E4M3 : QLORA_F32, ptr(m), ptr(v), ptr<float>(ms), ptr<float>(vs),
                             ptr<float>(master)};
  Tensor ws;
  size_t bytes = 0;
  if (max_norm > 0.f) {
    if (!norm.defined()) norm = empty({1}, at::kFloat, m);
    bytes = qlora_adamw_many_workspace_bytes((int32_t)count);
    ws = empty({(int64_t)bytes}, at::kByte, m);
  }
  return answer(qlora_adamw_many(&hp, step, jobs.data(), (int32_t)count, gd, pd, &st, max_norm, ptr<float>(norm),
                                 (uint32_t)seed, ptr(ws), bytes, as_stream(a[17])),
                {norm});
  QLORA_EXIT
}

#define QLORA_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {QLORA_METHOD(rmsnorm_forward), QLORA_METHOD(rmsnorm_backward), QLORA_METHOD(fp8_forward),
                         QLORA_METHOD(fp8_backward), QLORA_METHOD(adamw_many), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal(void) { return PyModule_Create(&module_def); }
