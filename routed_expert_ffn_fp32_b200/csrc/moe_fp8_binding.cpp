// Argument marshalling of the 8-bit operators' Python binding: reads sizes,
// types, devices and pointers out of the tensors, checks them against one
// another and calls the C entry point (include/moe.h) on the current stream of
// the tensors' device.  A decode step makes many of these calls and each is as
// short as a launch: 3.0 us for the norm or a dense product, 4.1 for the gate /
// up pair (6.9 to 10.9 us with the same checks written in Python over ctypes).
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdint>
#include <exception>
#include <limits>
#include <optional>
#include <stdexcept>
#include <string>

#include "moe.h"

namespace {

decltype(&moe_rmsnorm_quant_fp8) p_norm = nullptr;
decltype(&moe_gemm_fp8) p_gemm = nullptr;
decltype(&moe_grouped_gemm_fp8) p_grouped = nullptr;
decltype(&moe_grouped_swiglu_fp8) p_swiglu = nullptr;

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
void need(bool ok, const char* what) {
  if (!ok) throw Refused(what);
}

using Opt = const at::Tensor*;  // nullptr: None

Opt optional_tensor(PyObject* o) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw std::invalid_argument("expected a torch.Tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o) {
  Opt t = optional_tensor(o);
  if (t == nullptr) throw std::invalid_argument("expected a torch.Tensor, not None");
  return *t;
}

int64_t b128(int64_t n) { return (n + 127) / 128; }
int32_t i32(int64_t v) {
  need(v >= std::numeric_limits<int32_t>::min() && v <= std::numeric_limits<int32_t>::max(),
       "expected sizes and integers below 2^31");
  return int32_t(v);
}
bool codes(const at::Tensor& q) { return q.scalar_type() == at::kFloat8_e4m3fn || q.scalar_type() == at::kByte; }

int32_t dtype_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return MOE_DTYPE_BF16;
    case at::kHalf: return MOE_DTYPE_F16;
    case at::kFloat: return MOE_DTYPE_F32;
    default: throw Refused("expected bfloat16, float16 or float32 values");
  }
}

void rows8(const at::Tensor& q, const at::Tensor& s) {
  need(codes(q) && s.scalar_type() == at::kFloat, "rows: expected E4M3 codes and float32 scales");
  need(q.dim() == 2 && s.dim() == 2 && s.size(0) == q.size(0) && s.size(1) == b128(q.size(1)),
       "rows: expected codes [rows, K] and scales [rows, ceil(K / 128)]");
}
void mats8(const at::Tensor& q, const at::Tensor& s, int64_t K) {
  need(codes(q) && s.scalar_type() == at::kFloat, "weights: expected E4M3 codes and float32 scales");
  need(q.dim() == 3 && q.size(2) == K && s.dim() == 3 && s.size(0) == q.size(0) && s.size(1) == b128(q.size(1)) &&
           s.size(2) == b128(K),
       "weights: expected codes [E, N, K] and scales [E, ceil(N / 128), ceil(K / 128)]");
}
void groups(Opt offsets, Opt entries, int64_t E, int64_t P) {
  need(offsets == nullptr || (offsets->scalar_type() == at::kInt && offsets->numel() == E + 1),
       "offsets: expected E + 1 int32 values");
  need(entries == nullptr || (entries->scalar_type() == at::kInt && entries->numel() == P),
       "entries: expected one int32 value per pair");
}

// The tensors' one CUDA device, current while this lives, and their pointers.
struct Call {
  int dev = -2;
  void* stream = nullptr;
  std::optional<c10::cuda::CUDAGuard> guard;

  void* ptr(const at::Tensor& t) {
    const int d = t.is_cuda() ? t.get_device() : -1;
    if (dev == -2) {
      need(d >= 0, "expected CUDA tensors");
      dev = d;
    }
    need(d == dev, "expected tensors on one device");
    need(t.is_contiguous(), "expected contiguous tensors");
    return t.data_ptr();
  }
  void* ptr(Opt t) { return t ? ptr(*t) : nullptr; }
  // after the pointers: device and stream (None: the device's current one)
  void open(PyObject* o) {
    c10::DeviceIndex now = -1;
    if (c10::cuda::GetDevice(&now) != cudaSuccess || now != dev) guard.emplace(static_cast<c10::DeviceIndex>(dev));
    if (o == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    } else {
      stream = PyLong_AsVoidPtr(o);
      if (stream == nullptr && PyErr_Occurred()) throw std::invalid_argument("stream: expected an address");
    }
  }
};

template <typename F>
PyObject* run(Py_ssize_t given, Py_ssize_t wanted, F&& f) {
  try {
    if (given != wanted) throw std::invalid_argument("wrong number of arguments");
    return PyLong_FromLong(f());
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_TypeError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw std::invalid_argument("expected a number");
  }
  return float(v);
}
int32_t integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw std::invalid_argument("expected an integer");
  }
  return i32(v);
}

// x, weight, eps, q_out, s_out, residual, residual_out, y_out, stream
PyObject* norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 9, [&] {
    const at::Tensor &x = tensor(a[0]), &w = tensor(a[1]), &q = tensor(a[3]), &s = tensor(a[4]);
    const Opt res = optional_tensor(a[5]), ro = optional_tensor(a[6]), y = optional_tensor(a[7]);
    const int32_t dt = dtype_of(x);
    rows8(q, s);
    need(x.sizes() == q.sizes() && w.dim() == 1 && w.size(0) == x.size(1) && w.scalar_type() == at::kFloat,
         "expected x, q_out [rows, H] and a float32 weight [H]");
    for (Opt t : {res, ro, y})
      need(t == nullptr || (t->sizes() == x.sizes() && t->scalar_type() == x.scalar_type()),
           "residual, residual_out, y_out: expected the shape and type of x");
    const float eps = number(a[2]);
    Call c;
    void *px = c.ptr(x), *pr = c.ptr(res), *pw = c.ptr(w), *pro = c.ptr(ro), *py = c.ptr(y), *pq = c.ptr(q),
         *ps = c.ptr(s);
    c.open(a[8]);
    return p_norm(px, pr, static_cast<const float*>(pw), i32(x.size(0)), i32(x.size(1)), dt, eps, pro, py,
                  static_cast<uint8_t*>(pq), static_cast<float*>(ps), c.stream);
  });
}

// a_q, a_s, w_q, w_s, out, ws, stream
PyObject* gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 7, [&] {
    const at::Tensor &aq = tensor(a[0]), &as = tensor(a[1]), &wq = tensor(a[2]), &wsc = tensor(a[3]),
                     &out = tensor(a[4]), &ws = tensor(a[5]);
    const int32_t dt = dtype_of(out);
    rows8(aq, as);
    const int64_t rows = aq.size(0), K = aq.size(1);
    need(codes(wq) && wsc.scalar_type() == at::kFloat && wq.dim() == 2 && wq.size(1) == K && wsc.dim() == 2 &&
             wsc.size(0) == b128(wq.size(0)) && wsc.size(1) == b128(K),
         "w_q, w_s: expected codes [N, K] and float32 scales [ceil(N / 128), ceil(K / 128)]");
    const int64_t N = wq.size(0);
    need(out.dim() == 2 && out.size(0) == rows && out.size(1) == N, "out: expected [rows, N]");
    Call c;
    void *pa = c.ptr(aq), *pas = c.ptr(as), *pw = c.ptr(wq), *pws = c.ptr(wsc), *po = c.ptr(out), *pk = c.ptr(ws);
    c.open(a[6]);
    return p_gemm(static_cast<const uint8_t*>(pa), static_cast<const float*>(pas), static_cast<const uint8_t*>(pw),
                  static_cast<const float*>(pws), i32(rows), i32(N), i32(K), dt, po, pk, ws.nbytes(), c.stream);
  });
}

// a_q, a_s, w_q, w_s, offsets, entries, out, ws, a_div, scatter, stream
PyObject* grouped(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 11, [&] {
    const at::Tensor &aq = tensor(a[0]), &as = tensor(a[1]), &wq = tensor(a[2]), &wsc = tensor(a[3]),
                     &out = tensor(a[6]), &ws = tensor(a[7]);
    const Opt off = optional_tensor(a[4]), ent = optional_tensor(a[5]);
    const int32_t dt = dtype_of(out);
    rows8(aq, as);
    const int64_t K = aq.size(1);
    mats8(wq, wsc, K);
    const int64_t E = wq.size(0), N = wq.size(1);
    need(out.dim() == 2 && out.size(1) == N, "out: expected [n_pairs, N]");
    const int64_t P = out.size(0);
    groups(off, ent, E, P);
    const int32_t div = integer(a[8]);
    const int scatter = PyObject_IsTrue(a[9]);
    if (scatter < 0) {
      PyErr_Clear();
      throw std::invalid_argument("scatter: expected a truth value");
    }
    Call c;
    void *pa = c.ptr(aq), *pas = c.ptr(as), *pw = c.ptr(wq), *pws = c.ptr(wsc), *pf = c.ptr(off), *pe = c.ptr(ent),
         *po = c.ptr(out), *pk = c.ptr(ws);
    c.open(a[10]);
    return p_grouped(static_cast<const uint8_t*>(pa), static_cast<const float*>(pas), i32(aq.size(0)),
                     static_cast<const uint8_t*>(pw), static_cast<const float*>(pws), static_cast<const int32_t*>(pf),
                     static_cast<const int32_t*>(pe), i32(P), i32(E), i32(N), i32(K), div, scatter, dt, po, pk,
                     ws.nbytes(), c.stream);
  });
}

// a_q, a_s, gate_q, gate_s, up_q, up_s, offsets, entries, q_out, s_out, ws, a_div, stream
PyObject* swiglu(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return run(n, 13, [&] {
    const at::Tensor &aq = tensor(a[0]), &as = tensor(a[1]), &gq = tensor(a[2]), &gs = tensor(a[3]),
                     &uq = tensor(a[4]), &us = tensor(a[5]), &q = tensor(a[8]), &s = tensor(a[9]),
                     &ws = tensor(a[10]);
    const Opt off = optional_tensor(a[6]), ent = optional_tensor(a[7]);
    rows8(aq, as);
    const int64_t H = aq.size(1);
    mats8(gq, gs, H);
    mats8(uq, us, H);
    need(uq.sizes() == gq.sizes(), "up_q: expected the shape of gate_q");
    const int64_t E = gq.size(0), I = gq.size(1);
    rows8(q, s);
    need(q.size(1) == I, "q_out: expected [n_pairs, I]");
    const int64_t P = q.size(0);
    groups(off, ent, E, P);
    const int32_t div = integer(a[11]);
    Call c;
    void *pa = c.ptr(aq), *pas = c.ptr(as), *pg = c.ptr(gq), *pgs = c.ptr(gs), *pu = c.ptr(uq), *pus = c.ptr(us),
         *pf = c.ptr(off), *pe = c.ptr(ent), *pq = c.ptr(q), *ps = c.ptr(s), *pk = c.ptr(ws);
    c.open(a[12]);
    return p_swiglu(static_cast<const uint8_t*>(pa), static_cast<const float*>(pas), i32(aq.size(0)),
                    static_cast<const uint8_t*>(pg), static_cast<const float*>(pgs), static_cast<const uint8_t*>(pu),
                    static_cast<const float*>(pus), static_cast<const int32_t*>(pf), static_cast<const int32_t*>(pe),
                    i32(P), i32(E), i32(I), i32(H), div, static_cast<uint8_t*>(pq), static_cast<float*>(ps), pk,
                    ws.nbytes(), c.stream);
  });
}

// addresses of the library's entry points: norm, gemm, grouped gemm, swiglu
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "expected four addresses");
    return nullptr;
  }
  void* p[4];
  for (int i = 0; i < 4; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "expected four addresses");
      return nullptr;
    }
  }
  p_norm = reinterpret_cast<decltype(p_norm)>(p[0]);
  p_gemm = reinterpret_cast<decltype(p_gemm)>(p[1]);
  p_grouped = reinterpret_cast<decltype(p_grouped)>(p[2]);
  p_swiglu = reinterpret_cast<decltype(p_swiglu)>(p[3]);
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyObject* bound(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  if (p_norm == nullptr) {
    PyErr_SetString(PyExc_RuntimeError, "the library's entry points are not bound");
    return nullptr;
  }
  return F(self, a, n);
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef kMethods[] = {method<bind>("bind"),
                          method<bound<norm>>("norm"),
                          method<bound<gemm>>("gemm"),
                          method<bound<grouped>>("grouped"),
                          method<bound<swiglu>>("swiglu"),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fp8_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr,
                       nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp8_binding() { return PyModule_Create(&kModule); }
