// gdr_binding.cpp -- the operators' Python binding: checks of device, type, shape
// and layout, allocation of outputs on the current stream, and the call of the
// library (include/gdr.h) with the interpreter's lock released.  A failed check
// raises ValueError with nothing enqueued.  Compiled, because the smallest calls
// are bound by the host: one sequence's delta-rule step takes 4.5 us a call (13.5 through
// checks in Python and ctypes), a norm between two blocks 6.8 (19.7).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <memory>
#include <stdexcept>
#include <string>

#include "../../include/gdr.h"

namespace {

using at::Tensor;
using c10::ScalarType;
using Shape = c10::IntArrayRef;

PyObject* g_check = nullptr;  // raises for a status

struct Refused : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct PyError {};  // a Python exception is set

std::string str(ScalarType t) {
  switch (t) {
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Half: return "torch.float16";
    case ScalarType::Float: return "torch.float32";
    default: return c10::toString(t);
  }
}
std::string str(Shape s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

int code_of(ScalarType t) {
  return t == ScalarType::BFloat16 ? GDR_DTYPE_BF16 : t == ScalarType::Half ? GDR_DTYPE_F16 : t == ScalarType::Float ? GDR_DTYPE_F32 : -1;
}

// One call: its name and its device.
struct Call {
  const char* where;
  int dev = 0;
  cudaStream_t stream = nullptr;
  at::TensorOptions options;

  [[noreturn]] void fail(const std::string& what) const { throw Refused(std::string(where) + ": " + what); }

  // The current device, which must hold t.
  void on(const Tensor& t) {
    if (!t.is_cuda()) fail("tensors must be on a CUDA device, got " + t.device().str());
    dev = t.get_device();
    if (dev != c10::cuda::current_device())
      fail("tensors are on " + t.device().str() + ", the current device is cuda:" + std::to_string(c10::cuda::current_device()));
    stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    options = at::TensorOptions().device(t.device());
  }
  const Tensor& tensor(const char* name, PyObject* o) const {
    if (!THPVariable_Check(o)) fail(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
  }
  void same_device(const char* name, const Tensor& t) const {
    if (!t.is_cuda() || t.get_device() != dev)
      fail(std::string(name) + " is on " + t.device().str() + ", expected cuda:" + std::to_string(dev));
  }
  // The address of a dense tensor of exactly this type and shape.
  void* dense(const char* name, const Tensor& t, ScalarType type, Shape shape) const {
    if (t.scalar_type() != type || t.sizes() != shape)
      fail(std::string(name) + " is " + str(t.scalar_type()) + " " + str(t.sizes()) + ", expected " + str(type) + " " + str(shape));
    if (!t.is_contiguous()) fail(std::string(name) + " must be contiguous");
    same_device(name, t);
    return t.data_ptr();
  }
  void* dense(const char* name, PyObject* o, ScalarType type, Shape shape) const {  // None: null
    return o == Py_None ? nullptr : dense(name, tensor(name, o), type, shape);
  }
  Tensor empty(Shape shape, ScalarType type) const { return at::empty(shape, options.dtype(type)); }
  // `given`, or a new tensor where it is None; *p: its address.
  Tensor output(const char* name, PyObject* given, Shape shape, ScalarType type, void** p) const {
    Tensor t;
    if (given == Py_None) {
      t = empty(shape, type);
      *p = t.data_ptr();
    } else {
      t = tensor(name, given);
      *p = dense(name, t, type, shape);
    }
    return t;
  }
  Tensor scratch(PyObject* given, size_t need, void** p, size_t* bytes) const {
    Tensor t;
    if (given == Py_None) {
      t = empty({(int64_t)(need > 256 ? need : 256)}, ScalarType::Byte);
    } else {
      t = tensor("scratch", given);
      if (!t.is_contiguous() || !t.is_cuda() || t.get_device() != dev)
        fail("scratch must be contiguous and on cuda:" + std::to_string(dev));
    }
    *p = t.data_ptr();
    *bytes = (size_t)t.numel() * t.element_size();
    return t;
  }
  // A size that the library takes as 32 bits.
  int32_t size(const char* name, int64_t n) const {
    if (n > INT32_MAX) fail(std::string(name) + " " + std::to_string(n) + " is past 2^31 - 1");
    return (int32_t)n;
  }
  void status(gdr_status code) const {
    if (code == GDR_OK) return;
    PyObject* r = PyObject_CallFunction(g_check, "is", (int)code, where);
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, where);
    throw PyError();
  }
  template <typename F>
  void run(F f) const {
    gdr_status code;
    Py_BEGIN_ALLOW_THREADS code = f();
    Py_END_ALLOW_THREADS status(code);
  }
};

// cu_seqlens on the device and on the host (a C-contiguous int32 array, held for
// the call).
struct Pack {
  Py_buffer view{};
  const int32_t* host = nullptr;
  const int32_t* cu = nullptr;
  int n = 0;
  Pack(const Call& c, PyObject* device, PyObject* array) {
    if (PyObject_GetBuffer(array, &view, PyBUF_FORMAT | PyBUF_ND | PyBUF_C_CONTIGUOUS) != 0) throw PyError();
    if (view.ndim != 1 || view.shape[0] < 1 || view.itemsize != 4) {
      PyBuffer_Release(&view);
      c.fail("cu_seqlens_host must be one-dimensional with at least one entry");
    }
    host = static_cast<const int32_t*>(view.buf);
    n = (int)view.shape[0] - 1;
    try {
      cu = static_cast<const int32_t*>(c.dense("cu_seqlens", device, ScalarType::Int, {(int64_t)n + 1}));
    } catch (...) {
      PyBuffer_Release(&view);
      throw;
    }
  }
  Pack(const Pack&) = delete;
  ~Pack() { PyBuffer_Release(&view); }
};

bool truth(PyObject* o) {
  const int r = PyObject_IsTrue(o);
  if (r < 0) throw PyError();
  return r != 0;
}
double number(PyObject* o) {
  const double r = PyFloat_AsDouble(o);
  if (r == -1.0 && PyErr_Occurred()) throw PyError();
  return r;
}
PyObject* wrap(const Tensor& t) { return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None); }
PyObject* two(const Tensor& a, const Tensor& b) {
  PyObject* r = PyTuple_New(2);
  if (!r) throw PyError();
  PyTuple_SET_ITEM(r, 0, wrap(a));
  PyTuple_SET_ITEM(r, 1, wrap(b));
  return r;
}

// The dict of gradients: the caller's tensors, or new ones beside them.
struct Grads {
  PyObject* d;
  explicit Grads(PyObject* given) : d(given == Py_None ? PyDict_New() : PyDict_Copy(given)) {
    if (!d) throw PyError();
  }
  Grads(const Grads&) = delete;
  ~Grads() { Py_XDECREF(d); }
  PyObject* get(const char* name) const {  // null: none given
    PyObject* o = PyDict_GetItemString(d, name);
    return o == Py_None ? nullptr : o;
  }
  void set(const char* name, PyObject* v) {  // takes v
    const int e = v ? PyDict_SetItemString(d, name, v) : -1;
    Py_XDECREF(v);
    if (e) throw PyError();
  }
  void* tensor(const Call& c, const char* name, Shape shape, ScalarType type) {
    if (PyObject* o = get(name)) return c.dense(name, o, type, shape);
    Tensor t = c.empty(shape, type);
    set(name, wrap(t));
    return t.data_ptr();
  }
  PyObject* release() {
    PyObject* r = d;
    d = nullptr;
    return r;
  }
};

// --- short causal convolution ---------------------------------------------------
struct Conv {
  int dt, wdt, W;
  int64_t T, C;
  ScalarType type;
  const Tensor& x;
  void *w, *bias;
  Conv(Call& c, PyObject* xo, PyObject* weight, PyObject* bo) : x(c.tensor("x", xo)) {
    c.on(x);
    type = x.scalar_type();
    dt = code_of(type);
    if (x.dim() != 2) c.fail("x has shape " + str(x.sizes()) + ", expected [tokens, channels]");
    if (dt < 0) c.fail("x is " + str(type) + "; bfloat16, float16 and float32 are supported");
    T = x.size(0);
    C = c.size("channels", x.size(1));
    const Tensor& wt = c.tensor("weight", weight);
    if (wt.dim() != 2 || wt.size(0) != C || wt.size(1) < 2 || wt.size(1) > 4)
      c.fail("weight has shape " + str(wt.sizes()) + ", expected [" + std::to_string(C) + ", 2 to 4]");
    const ScalarType wtype = wt.scalar_type();
    if (wtype != type && wtype != ScalarType::Float) c.fail("weight is " + str(wtype) + ", expected " + str(type) + " or float32");
    W = (int)wt.size(1);
    w = c.dense("weight", wt, wtype, wt.sizes());
    bias = c.dense("bias", bo, wtype, {C});
    wdt = code_of(wtype);
  }
  // Row stride of a tensor of x's shape with dense rows.
  int64_t rows(const Call& c, const char* name, const Tensor& t) const {
    if (t.stride(1) != 1 && C > 1) c.fail(std::string(name) + " must have dense rows");
    return T > 1 ? t.stride(0) : C;
  }
};

PyObject* sconv_fwd_(PyObject* const* a) {  // x weight bias cu cuh s0 silu out st want_st
  Call c{"sconv_fwd"};
  const Conv v(c, a[0], a[1], a[2]);
  const Pack p(c, a[3], a[4]);
  const int64_t state[3] = {p.n, v.W - 1, v.C}, shape[2] = {v.T, v.C};
  const int64_t ldx = v.rows(c, "x", v.x);
  const void* s0 = c.dense("s0", a[5], v.type, state);
  const bool silu = truth(a[6]);
  void *op, *sp = nullptr;
  const Tensor out = c.output("out", a[7], shape, v.type, &op);
  const Tensor st = a[8] == Py_None && !truth(a[9]) ? Tensor() : c.output("st", a[8], state, v.type, &sp);
  c.run([&] {
    return sconv_fwd(v.dt, v.x.data_ptr(), ldx, v.w, v.bias, v.wdt, p.cu, p.host, p.n, v.T, (int32_t)v.C, v.W, silu, s0, op,
                     sp, c.stream);
  });
  return two(out, st);
}

PyObject* sconv_bwd_(PyObject* const* a) {  // x weight bias cu cuh dout s0 dst want_ds0 silu scratch grads
  Call c{"sconv_bwd"};
  const Conv v(c, a[0], a[1], a[2]);
  const Pack p(c, a[3], a[4]);
  const int64_t state[3] = {p.n, v.W - 1, v.C}, shape[2] = {v.T, v.C}, taps[2] = {v.C, v.W};
  const Tensor& dout = c.tensor("dout", a[5]);
  if (dout.scalar_type() != v.type || dout.sizes() != v.x.sizes())
    c.fail("dout is " + str(dout.scalar_type()) + " " + str(dout.sizes()) + ", expected " + str(v.type) + " " + str(v.x.sizes()));
  c.same_device("dout", dout);
  const int64_t ldx = v.rows(c, "x", v.x), ldo = v.rows(c, "dout", dout);
  const void *s0 = c.dense("s0", a[6], v.type, state), *dst = c.dense("dst", a[7], v.type, state);
  const bool silu = truth(a[9]);
  Grads g(a[11]);
  void* dx = g.tensor(c, "dx", shape, v.type);
  float* dw = static_cast<float*>(g.tensor(c, "dweight", taps, ScalarType::Float));
  float* db = nullptr;
  if (a[2] == Py_None) g.set("dbias", Py_NewRef(Py_None));
  else db = static_cast<float*>(g.tensor(c, "dbias", {v.C}, ScalarType::Float));
  void* ds0 = nullptr;
  if (truth(a[8]) || g.get("ds0")) ds0 = g.tensor(c, "ds0", state, v.type);
  size_t need = 0, bytes = 0;
  c.status(sconv_workspace_bytes(v.T, (int32_t)v.C, v.W, &need));
  void* sp;
  const Tensor scratch = c.scratch(a[10], need, &sp, &bytes);
  c.run([&] {
    return sconv_bwd(v.dt, v.x.data_ptr(), ldx, v.w, v.bias, v.wdt, p.cu, p.host, p.n, v.T, (int32_t)v.C, v.W, silu, s0,
                     dout.data_ptr(), ldo, dst, dx, dw, db, ds0, sp, bytes, c.stream);
  });
  return g.release();
}

PyObject* sconv_step_(PyObject* const* a) {  // x weight bias state slots silu out
  Call c{"sconv_step"};
  const Conv v(c, a[0], a[1], a[2]);
  const Tensor& st = c.tensor("state", a[3]);
  const int64_t S = c.size("states", st.dim() > 0 ? st.size(0) : 0), state[3] = {S, v.W - 1, v.C}, shape[2] = {v.T, v.C};
  const int32_t rows = c.size("batch", v.T);
  void* sp = c.dense("state", st, v.type, state);
  const int64_t ldx = v.rows(c, "x", v.x);
  const int32_t* slots = static_cast<const int32_t*>(c.dense("slots", a[4], ScalarType::Int, {v.T}));
  const bool silu = truth(a[5]);
  void* op;
  const Tensor out = c.output("out", a[6], shape, v.type, &op);
  c.run([&] {
    return sconv_step(v.dt, v.x.data_ptr(), ldx, v.w, v.bias, v.wdt, sp, slots, rows, (int32_t)S, (int32_t)v.C, v.W,
                      silu, op, c.stream);
  });
  return wrap(out);
}

// --- selective scan ---------------------------------------------------------------
struct Scan {
  const Tensor& x;
  const Tensor& dt;
  const Tensor& B;
  const Tensor& C;
  int64_t T, H, P, G, NS, ldx, ldb, ldc, lddt;
  int dt_code;
  const float *A, *D, *bias;
  // Token stride of a [T, heads, dim] tensor whose (heads, dim) are dense.
  static int64_t heads(const Call& c, const char* name, const Tensor& t, int64_t T) {
    if (t.dim() != 3 || t.size(0) != T)
      c.fail(std::string(name) + " has shape " + str(t.sizes()) + ", expected [" + std::to_string(T) + ", heads, dim]");
    if (t.scalar_type() != ScalarType::BFloat16) c.fail(std::string(name) + " is " + str(t.scalar_type()) + ", expected bfloat16");
    c.same_device(name, t);
    const int64_t h = t.size(1), d = t.size(2);
    if ((d > 1 && t.stride(2) != 1) || (h > 1 && t.stride(1) != d)) c.fail(std::string(name) + " must be dense within a token");
    return T > 1 ? t.stride(0) : h * d;
  }
  Scan(Call& c, PyObject* const* a)  // x dt A B C D dt_bias
      : x(c.tensor("x", a[0])), dt(c.tensor("dt", a[1])), B(c.tensor("B", a[3])), C(c.tensor("C", a[4])) {
    c.on(x);
    if (x.dim() != 3) c.fail("x has shape " + str(x.sizes()) + ", expected [tokens, heads, head dim]");
    T = x.size(0);
    H = c.size("heads", x.size(1));
    P = c.size("head dim", x.size(2));
    ldx = heads(c, "x", x, T);
    ldb = heads(c, "B", B, T);
    ldc = heads(c, "C", C, T);
    if (B.sizes() != C.sizes()) c.fail("B has shape " + str(B.sizes()) + " and C " + str(C.sizes()));
    G = c.size("groups", B.size(1));
    NS = c.size("state size", B.size(2));
    dt_code = code_of(dt.scalar_type());
    if (dt.dim() != 2 || dt.size(0) != T || dt.size(1) != H || (dt_code != GDR_DTYPE_BF16 && dt_code != GDR_DTYPE_F32) ||
        (H > 1 && dt.stride(1) != 1))
      c.fail("dt is " + str(dt.scalar_type()) + " " + str(dt.sizes()) + ", expected bfloat16 or float32 [" + std::to_string(T) +
             ", " + std::to_string(H) + "] with dense rows");
    c.same_device("dt", dt);
    lddt = T > 1 ? dt.stride(0) : H;
    if (G < 1 || H % G) c.fail(std::to_string(H) + " heads do not share " + std::to_string(G) + " groups of B and C evenly");
    A = static_cast<const float*>(c.dense("A", c.tensor("A", a[2]), ScalarType::Float, {H}));
    D = static_cast<const float*>(c.dense("D", a[5], ScalarType::Float, {H}));
    bias = static_cast<const float*>(c.dense("dt_bias", a[6], ScalarType::Float, {H}));
  }
  const gdr_bf16* bf(const Tensor& t) const { return static_cast<const gdr_bf16*>(t.data_ptr()); }
};

PyObject* ssm_fwd_(PyObject* const* a) {  // x dt A B C D dt_bias softplus cu cuh h0 out ht want_ht scratch
  Call c{"ssm_fwd"};
  const Scan v(c, a);
  const bool softplus = truth(a[7]);
  const Pack p(c, a[8], a[9]);
  const int64_t state[4] = {p.n, v.H, v.NS, v.P}, shape[3] = {v.T, v.H, v.P};
  const float* h0 = static_cast<const float*>(c.dense("h0", a[10], ScalarType::Float, state));
  size_t need = 0, bytes = 0;
  c.status(ssm_workspace_bytes(v.T, (int32_t)v.H, (int32_t)v.P, (int32_t)v.G, (int32_t)v.NS, p.n, p.host, &need));
  void *op, *hp = nullptr, *sp = nullptr;
  const Tensor out = c.output("out", a[11], shape, ScalarType::BFloat16, &op);
  const Tensor ht = a[12] == Py_None && !truth(a[13]) ? Tensor() : c.output("ht", a[12], state, ScalarType::Float, &hp);
  const Tensor scratch = a[14] == Py_None && need == 0 ? Tensor() : c.scratch(a[14], need, &sp, &bytes);
  c.run([&] {
    return ssm_fwd(v.bf(v.x), v.ldx, v.dt.data_ptr(), v.dt_code, v.lddt, v.A, v.bf(v.B), v.ldb, v.bf(v.C), v.ldc, v.D, v.bias,
                   softplus, p.cu, p.host, p.n, v.T, (int32_t)v.H, (int32_t)v.P, (int32_t)v.G, (int32_t)v.NS, h0,
                   static_cast<gdr_bf16*>(op), static_cast<float*>(hp), sp, bytes, c.stream);
  });
  return two(out, ht);
}

PyObject* ssm_step_(PyObject* const* a) {  // x dt A B C D dt_bias softplus state slots out
  Call c{"ssm_step"};
  const Scan v(c, a);
  const bool softplus = truth(a[7]);
  const Tensor& st = c.tensor("state", a[8]);
  const int64_t S = c.size("states", st.dim() > 0 ? st.size(0) : 0), state[4] = {S, v.H, v.NS, v.P}, shape[3] = {v.T, v.H, v.P};
  const int32_t rows = c.size("batch", v.T);
  float* sp = static_cast<float*>(c.dense("state", st, ScalarType::Float, state));
  const int32_t* slots = static_cast<const int32_t*>(c.dense("slots", a[9], ScalarType::Int, {v.T}));
  void* op;
  const Tensor out = c.output("out", a[10], shape, ScalarType::BFloat16, &op);
  c.run([&] {
    return ssm_step(v.bf(v.x), v.ldx, v.dt.data_ptr(), v.dt_code, v.lddt, v.A, v.bf(v.B), v.ldb, v.bf(v.C), v.ldc, v.D, v.bias,
                    softplus, sp, slots, rows, (int32_t)S, (int32_t)v.H, (int32_t)v.P, (int32_t)v.G, (int32_t)v.NS,
                    static_cast<gdr_bf16*>(op), c.stream);
  });
  return wrap(out);
}

// --- one token of the gated delta rule -----------------------------------------------
PyObject* delta_step(const char* where, bool kda, PyObject* const* a) {  // q k v g beta state scale slots out l2
  Call c{where};
  const Tensor &q = c.tensor("q", a[0]), &v = c.tensor("v", a[2]), &st = c.tensor("state", a[5]);
  c.on(q);
  if (q.dim() != 3 || v.dim() != 3 || q.size(2) != 128)
    c.fail("q has shape " + str(q.sizes()) + " and v " + str(v.sizes()) + ", expected [batch, heads, 128]");
  const int64_t B = c.size("batch", q.size(0)), Hqk = c.size("heads", q.size(1)), HV = c.size("heads", v.size(1)),
                S = c.size("states", st.dim() > 0 ? st.size(0) : 0);
  if (kda && Hqk != HV)
    c.fail("q and k have " + std::to_string(Hqk) + " heads and v has " + std::to_string(HV) + "; KDA needs the same count");
  if (Hqk < 1 || HV % Hqk)
    c.fail(std::to_string(HV) + " value heads do not share " + std::to_string(Hqk) + " q/k heads evenly");
  const int64_t keys[3] = {B, Hqk, 128}, vals[3] = {B, HV, 128}, state[4] = {S, HV, 128, 128};
  const auto bf = ScalarType::BFloat16, f32 = ScalarType::Float;
  const auto* qp = static_cast<const gdr_bf16*>(c.dense("q", q, bf, keys));
  const auto* kp = static_cast<const gdr_bf16*>(c.dense("k", c.tensor("k", a[1]), bf, keys));
  const auto* vp = static_cast<const gdr_bf16*>(c.dense("v", v, bf, vals));
  const auto* gp = static_cast<const float*>(c.dense("g", c.tensor("g", a[3]), f32, Shape(vals, kda ? 3 : 2)));
  const void* bp = c.dense("beta", c.tensor("beta", a[4]), kda ? bf : f32, Shape(vals, 2));
  float* sp = static_cast<float*>(c.dense("state", st, f32, state));
  const float scale = (float)number(a[6]);
  const auto* slots = static_cast<const int32_t*>(c.dense("slots", a[7], ScalarType::Int, {B}));
  const bool l2 = truth(a[9]);
  void* op;
  const Tensor out = c.output("out", a[8], vals, bf, &op);
  c.run([&] {
    return kda ? kda_step(qp, kp, vp, gp, static_cast<const gdr_bf16*>(bp), sp, slots, (int32_t)B, (int32_t)S, (int32_t)HV,
                          scale, l2, static_cast<gdr_bf16*>(op), c.stream)
               : gdn_step(qp, kp, vp, gp, static_cast<const float*>(bp), sp, slots, (int32_t)B, (int32_t)S, (int32_t)Hqk,
                          (int32_t)HV, scale, l2, static_cast<gdr_bf16*>(op), c.stream);
  });
  return wrap(out);
}
PyObject* kda_step_(PyObject* const* a) { return delta_step("kda_step", true, a); }
PyObject* gdn_step_(PyObject* const* a) { return delta_step("gdn_step", false, a); }

// --- norms around a block --------------------------------------------------------------
struct RowPtr {
  const void* p = nullptr;
  int64_t s0 = 0, s1 = 0;
};
// Address and strides of a tensor shaped like x: [..., D] as [R0, R1, D] with dense rows.
RowPtr row_ptr(const Call& c, const char* name, PyObject* o, const Tensor& x) {
  if (o == Py_None) return {};
  const Tensor& t = c.tensor(name, o);
  const int64_t nd = t.dim(), D = x.size(x.dim() - 1);
  if (t.sizes() != x.sizes() || t.scalar_type() != x.scalar_type())
    c.fail(std::string(name) + " is " + str(t.scalar_type()) + " " + str(t.sizes()) + ", expected " + str(x.scalar_type()) + " " + str(x.sizes()));
  c.same_device(name, t);
  if (t.stride(nd - 1) != 1 && D > 1) c.fail(std::string(name) + " must have dense rows");
  if (nd == 3) return {t.data_ptr(), t.stride(0), t.stride(1)};
  if (nd == 2) return {t.data_ptr(), t.stride(0), D};
  if (nd > 3 && !t.is_contiguous())
    c.fail(std::string(name) + " has " + std::to_string(nd) + " dimensions and must be contiguous");
  return {t.data_ptr(), nd == 1 ? D : D * t.size(nd - 2), D};
}
struct Norm {
  const Tensor& x;
  ScalarType type;
  int dt, wdt, act, R1;
  int64_t R0, D;
  RowPtr xr, gate, res;
  bool has_weight, has_post, has_gate, has_res;
  const void *w, *wp;
  float alpha, eps;
  RowPtr rows(const Call& c, const char* name, PyObject* o) const { return row_ptr(c, name, o, x); }
  Norm(Call& c, PyObject* const* a) : x(c.tensor("x", a[0])) {  // x weight post_weight gate act residual res_scale eps
    c.on(x);
    type = x.scalar_type();
    dt = code_of(type);
    if (dt < 0) c.fail("x is " + str(type) + "; bfloat16, float16 and float32 are supported");
    const int64_t nd = x.dim();
    if (nd < 1 || x.size(nd - 1) < 1 || x.size(nd - 1) > GDR_NORM_MAX_D)
      c.fail("x has shape " + str(x.sizes()) + "; rows of 1 to 16384 elements are supported");
    const char* name = PyUnicode_Check(a[4]) ? PyUnicode_AsUTF8(a[4]) : nullptr;
    act = !name ? -1 : std::string(name) == "silu" ? GDR_ACT_SILU : std::string(name) == "sigmoid" ? GDR_ACT_SIGMOID : -1;
    if (act < 0) c.fail("act must be 'silu' or 'sigmoid'");
    has_weight = a[1] != Py_None;
    has_post = a[2] != Py_None;
    has_gate = a[3] != Py_None;
    has_res = a[5] != Py_None;
    if (!has_weight && !has_post && !has_res) c.fail("one of weight, post_weight and residual is needed");
    D = x.size(nd - 1);
    const int64_t inner = nd >= 3 ? x.size(nd - 2) : 1;
    R0 = inner ? x.numel() / (inner * D) : 0;
    R1 = c.size("rows of the inner dimension", inner ? inner : 1);
    const ScalarType wtype = has_weight ? c.tensor("weight", a[1]).scalar_type()
                             : has_post ? c.tensor("post_weight", a[2]).scalar_type()
                                        : type;
    if (wtype != type && wtype != ScalarType::Float) c.fail("weights are " + str(wtype) + ", expected " + str(type) + " or float32");
    wdt = code_of(wtype);
    xr = rows(c, "x", a[0]);
    gate = rows(c, "gate", a[3]);
    res = rows(c, "residual", a[5]);
    w = c.dense("weight", a[1], wtype, {D});
    wp = c.dense("post_weight", a[2], wtype, {D});
    alpha = (float)number(a[6]);
    eps = (float)number(a[7]);
  }
};

PyObject* norm_fwd_(PyObject* const* a) {  // ... h y
  Call c{"norm_fwd"};
  const Norm v(c, a);
  void *hp = nullptr, *yp = nullptr;
  Tensor h, y;
  if (a[8] != Py_None || v.has_res || !v.has_weight) h = c.output("h", a[8], v.x.sizes(), v.type, &hp);
  if (a[9] != Py_None || v.has_weight) y = c.output("y", a[9], v.x.sizes(), v.type, &yp);
  c.run([&] {
    return norm_fwd(v.dt, v.R0, v.R1, (int32_t)v.D, v.xr.p, v.xr.s0, v.xr.s1, v.gate.p, v.gate.s0, v.gate.s1, v.act, v.res.p,
                    v.res.s0, v.res.s1, v.alpha, v.wp, v.w, v.wdt, v.eps, hp, yp, c.stream);
  });
  return two(h, y);
}

PyObject* norm_bwd_(PyObject* const* a) {  // ... dh dy scratch grads
  Call c{"norm_bwd"};
  const Norm v(c, a);
  if (a[8] == Py_None && a[9] == Py_None) c.fail("one of dh and dy is needed");
  if (a[9] != Py_None && !v.has_weight) c.fail("dy without weight");
  const RowPtr dh = v.rows(c, "dh", a[8]), dy = v.rows(c, "dy", a[9]);
  // where u = x and res_scale = 1, dx and dresidual are one tensor
  const bool same = v.has_res && !v.has_post && !v.has_gate && v.alpha == 1.f && (a[11] == Py_None || PyDict_Size(a[11]) == 0);
  Grads g(a[11]);
  void *dgate = nullptr, *dres = nullptr;
  float *dw = nullptr, *dwp = nullptr;
  void* dx = g.tensor(c, "dx", v.x.sizes(), v.type);
  if (v.has_gate || g.get("dgate")) dgate = g.tensor(c, "dgate", v.x.sizes(), v.type);
  if (same) g.set("dresidual", Py_NewRef(g.get("dx")));
  else if (v.has_res || g.get("dresidual")) dres = g.tensor(c, "dresidual", v.x.sizes(), v.type);
  if (v.has_weight || g.get("dweight")) dw = static_cast<float*>(g.tensor(c, "dweight", {v.D}, ScalarType::Float));
  if (v.has_post || g.get("dpost_weight")) dwp = static_cast<float*>(g.tensor(c, "dpost_weight", {v.D}, ScalarType::Float));
  size_t need = 0, bytes = 0;
  c.status(norm_workspace_bytes((int32_t)v.D, &need));
  void* sp;
  const Tensor scratch = c.scratch(a[10], need, &sp, &bytes);
  c.run([&] {
    return norm_bwd(v.dt, v.R0, v.R1, (int32_t)v.D, v.xr.p, v.xr.s0, v.xr.s1, v.gate.p, v.gate.s0, v.gate.s1, v.act, v.res.p,
                    v.res.s0, v.res.s1, v.alpha, v.wp, v.w, v.wdt, v.eps, dh.p, dh.s0, dh.s1, dy.p, dy.s0, dy.s1, dx, dgate, dres,
                    dw, dwp, sp, bytes, c.stream);
  });
  return g.release();
}

// --- layer norm in front of a block ------------------------------------------------------
struct LayerNorm {
  const Tensor& x;
  ScalarType type;
  int dt, wdt, R1;
  int64_t R0, D;
  RowPtr xr, res;
  bool has_res;
  const void *w, *b;
  float alpha, eps;
  LayerNorm(Call& c, PyObject* const* a) : x(c.tensor("x", a[0])) {  // x weight bias residual res_scale eps
    c.on(x);
    type = x.scalar_type();
    dt = code_of(type);
    if (dt < 0) c.fail("x is " + str(type) + "; bfloat16, float16 and float32 are supported");
    const int64_t nd = x.dim();
    if (nd < 1 || x.size(nd - 1) < 1 || x.size(nd - 1) > GDR_NORM_MAX_D)
      c.fail("x has shape " + str(x.sizes()) + "; rows of 1 to 16384 elements are supported");
    D = x.size(nd - 1);
    const int64_t inner = nd >= 3 ? x.size(nd - 2) : 1;
    R0 = inner ? x.numel() / (inner * D) : 0;
    R1 = c.size("rows of the inner dimension", inner ? inner : 1);
    const ScalarType wtype = a[1] != Py_None   ? c.tensor("weight", a[1]).scalar_type()
                             : a[2] != Py_None ? c.tensor("bias", a[2]).scalar_type()
                                               : type;
    if (wtype != type && wtype != ScalarType::Float) c.fail("weights are " + str(wtype) + ", expected " + str(type) + " or float32");
    wdt = code_of(wtype);
    xr = row_ptr(c, "x", a[0], x);
    res = row_ptr(c, "residual", a[3], x);
    has_res = a[3] != Py_None;
    w = c.dense("weight", a[1], wtype, {D});
    b = c.dense("bias", a[2], wtype, {D});
    alpha = (float)number(a[4]);
    eps = (float)number(a[5]);
  }
};

PyObject* lnorm_fwd_(PyObject* const* a) {  // ... h y
  Call c{"lnorm_fwd"};
  const LayerNorm v(c, a);
  void *hp = nullptr, *yp;
  Tensor h;
  if (a[6] != Py_None || v.has_res) h = c.output("h", a[6], v.x.sizes(), v.type, &hp);
  const Tensor y = c.output("y", a[7], v.x.sizes(), v.type, &yp);
  c.run([&] {
    return lnorm_fwd(v.dt, v.R0, v.R1, (int32_t)v.D, v.xr.p, v.xr.s0, v.xr.s1, v.res.p, v.res.s0, v.res.s1, v.alpha, v.w, v.b,
                     v.wdt, v.eps, hp, yp, c.stream);
  });
  return two(h, y);
}

PyObject* lnorm_bwd_(PyObject* const* a) {  // ... dh dy scratch grads
  Call c{"lnorm_bwd"};
  const LayerNorm v(c, a);
  if (a[7] == Py_None) c.fail("dy is needed");
  const RowPtr dh = row_ptr(c, "dh", a[6], v.x), dy = row_ptr(c, "dy", a[7], v.x);
  // where res_scale = 1, dx and dresidual are one tensor
  const bool same = v.has_res && v.alpha == 1.f && (a[9] == Py_None || PyDict_Size(a[9]) == 0);
  Grads g(a[9]);
  void *dres = nullptr, *dx = g.tensor(c, "dx", v.x.sizes(), v.type);
  float *dw = nullptr, *db = nullptr;
  if (same) g.set("dresidual", Py_NewRef(g.get("dx")));
  else if (v.has_res || g.get("dresidual")) dres = g.tensor(c, "dresidual", v.x.sizes(), v.type);
  if (v.w || g.get("dweight")) dw = static_cast<float*>(g.tensor(c, "dweight", {v.D}, ScalarType::Float));
  if (v.b || g.get("dbias")) db = static_cast<float*>(g.tensor(c, "dbias", {v.D}, ScalarType::Float));
  size_t need = 0, bytes = 0;
  c.status(lnorm_workspace_bytes((int32_t)v.D, &need));
  void* sp;
  const Tensor scratch = c.scratch(a[8], need, &sp, &bytes);
  c.run([&] {
    return lnorm_bwd(v.dt, v.R0, v.R1, (int32_t)v.D, v.xr.p, v.xr.s0, v.xr.s1, v.res.p, v.res.s0, v.res.s1, v.alpha, v.w, v.wdt,
                     v.eps, dh.p, dh.s0, dh.s1, dy.p, dy.s0, dy.s1, dx, dres, dw, db, sp, bytes, c.stream);
  });
  return g.release();
}

// --- [tokens, heads, dim] with dense heads ---------------------------------------------------
struct Heads {
  void* p = nullptr;
  int64_t T = 0, H = 0, D = 0, s0 = 0, s1 = 0;
  Heads() = default;
  Heads(const Call& c, const char* name, const Tensor& t, ScalarType type) {
    if (t.dim() != 3) c.fail(std::string(name) + " has shape " + str(t.sizes()) + ", expected [tokens, heads, dim]");
    if (t.scalar_type() != type) c.fail(std::string(name) + " is " + str(t.scalar_type()) + ", expected " + str(type));
    c.same_device(name, t);
    T = t.size(0);
    H = t.size(1);
    D = t.size(2);
    if (D > 1 && t.stride(2) != 1) c.fail(std::string(name) + " must have dense heads");
    s1 = H > 1 ? t.stride(1) : D;
    s0 = T > 1 ? t.stride(0) : H * D;
    p = t.data_ptr();
  }
  const gdr_bf16* bf() const { return static_cast<const gdr_bf16*>(p); }
};

// --- rotary positions --------------------------------------------------------------------
PyObject* rope_(PyObject* const* a) {  // q k freqs positions cu interleaved amplitude q_out k_out inverse
  const bool back = truth(a[9]);
  Call c{back ? "rope_bwd" : "rope_fwd"};
  if (a[0] == Py_None && a[1] == Py_None) c.fail("one of q and k is needed");
  const Tensor& first = c.tensor(a[0] != Py_None ? "q" : "k", a[a[0] != Py_None ? 0 : 1]);
  c.on(first);
  const ScalarType type = first.scalar_type();
  const int dt = code_of(type);
  if (dt < 0) c.fail("rows are " + str(type) + "; bfloat16, float16 and float32 are supported");
  Heads in[2], out[2];
  Tensor res[2];
  const char* names[2][2] = {{"q", "q_out"}, {"k", "k_out"}};
  int64_t T = 0, D = 0;
  for (int i = 0; i < 2; ++i) {
    if (a[i] == Py_None) {
      if (a[7 + i] != Py_None) c.fail(std::string(names[i][1]) + " without " + names[i][0]);
      continue;
    }
    const Tensor& t = c.tensor(names[i][0], a[i]);
    in[i] = Heads(c, names[i][0], t, type);
    if (i == 1 && a[0] != Py_None && (in[1].T != T || in[1].D != D))
      c.fail("k has shape " + str(t.sizes()) + ", expected [" + std::to_string(T) + ", heads, " + std::to_string(D) + "]");
    T = in[i].T;
    D = in[i].D;
    if (a[7 + i] == Py_None) {
      res[i] = c.empty(t.sizes(), type);
    } else {
      res[i] = c.tensor(names[i][1], a[7 + i]);
      if (res[i].sizes() != t.sizes()) c.fail(std::string(names[i][1]) + " has shape " + str(res[i].sizes()) + ", expected " + str(t.sizes()));
    }
    out[i] = Heads(c, names[i][1], res[i], type);
  }
  const Tensor& freqs = c.tensor("freqs", a[2]);
  const int64_t R = freqs.dim() == 1 ? 2 * freqs.size(0) : -1;
  if (R < 0 || R > D) c.fail("freqs has shape " + str(freqs.sizes()) + ", expected [pairs] of heads of " + std::to_string(D));
  const float* fp = static_cast<const float*>(c.dense("freqs", freqs, ScalarType::Float, {R / 2}));
  const void* pos = nullptr;
  bool wide = false;
  const int32_t* cu = nullptr;
  int32_t N = 0;
  if (a[3] != Py_None) {
    const Tensor& p = c.tensor("positions", a[3]);
    wide = p.scalar_type() == ScalarType::Long;
    pos = c.dense("positions", p, wide ? ScalarType::Long : ScalarType::Int, {T});
  } else if (a[4] != Py_None) {
    const Tensor& u = c.tensor("cu_seqlens", a[4]);
    if (u.dim() != 1 || u.size(0) < 1) c.fail("cu_seqlens has shape " + str(u.sizes()) + ", expected [documents + 1]");
    N = c.size("documents", u.size(0) - 1);
    cu = static_cast<const int32_t*>(c.dense("cu_seqlens", u, ScalarType::Int, {u.size(0)}));
  } else {
    c.fail("one of positions and cu_seqlens is needed");
  }
  const bool inter = truth(a[5]);
  const float amp = (float)number(a[6]);
  const int32_t HQ = c.size("heads", in[0].H), HK = c.size("heads", in[1].H), d = c.size("head dim", D);
  c.run([&] {
    return rope_turn(dt, in[0].p, in[0].s0, in[0].s1, HQ, out[0].p, out[0].s0, out[0].s1, in[1].p, in[1].s0, in[1].s1, HK, out[1].p,
                     out[1].s0, out[1].s1, T, d, (int32_t)R, fp, pos, wide, cu, N, inter, amp, back, c.stream);
  });
  return two(res[0], res[1]);
}

// --- softmax attention ---------------------------------------------------------------------
struct Attention {
  Heads q, k, v;
  Pack pack;
  std::unique_ptr<Pack> keys;
  float scale;
  bool causal;
  int32_t window;
  Attention(Call& c, PyObject* const* a)  // q k v cu cuh cu_keys cu_keys_host scale causal window
      : q((c.on(c.tensor("q", a[0])), Heads(c, "q", c.tensor("q", a[0]), ScalarType::BFloat16))),
        k(c, "k", c.tensor("k", a[1]), ScalarType::BFloat16), v(c, "v", c.tensor("v", a[2]), ScalarType::BFloat16),
        pack(c, a[3], a[4]) {
    if (k.T != v.T || k.H != v.H || k.D != v.D || k.D != q.D)
      c.fail("q has shape " + str(c.tensor("q", a[0]).sizes()) + ", k " + str(c.tensor("k", a[1]).sizes()) + " and v " +
             str(c.tensor("v", a[2]).sizes()));
    if (k.H < 1 || q.H < 1 || q.H % k.H) c.fail(std::to_string(q.H) + " heads do not share " + std::to_string(k.H) + " key heads evenly");
    if (q.D < 1 || q.D > GDR_ATTN_MAX_D) c.fail("head dim " + std::to_string(q.D) + "; 1 to 256 are supported");
    c.size("heads", q.H);
    if ((a[5] == Py_None) != (a[6] == Py_None)) c.fail("cu_keys and cu_keys_host come together");
    if (a[5] != Py_None) {
      keys = std::make_unique<Pack>(c, a[5], a[6]);
      if (keys->n != pack.n) c.fail("cu_keys has " + std::to_string(keys->n) + " documents, cu_seqlens " + std::to_string(pack.n));
    } else if (k.T != q.T) {
      c.fail("k has " + std::to_string(k.T) + " tokens and q " + std::to_string(q.T) + "; other keys need cu_keys");
    }
    scale = a[7] == Py_None ? (float)(1.0 / std::sqrt((double)q.D)) : (float)number(a[7]);
    if (!(scale > 0) || !std::isfinite(scale)) c.fail("scale must be positive and finite");
    causal = truth(a[8]);
    const long w = PyLong_AsLong(a[9]);
    if (w == -1 && PyErr_Occurred()) throw PyError();
    if (w < 0) c.fail("window must not be negative");
    if (w > 0 && !causal) c.fail("a window needs causal");
    window = w > INT32_MAX ? 0 : (int32_t)w;  // (sees everything)
  }
  const int32_t* cuk() const { return keys ? keys->cu : nullptr; }
  const int32_t* cuk_host() const { return keys ? keys->host : nullptr; }
  void workspace(const Call& c, size_t* fwd, size_t* bwd) const {
    c.status(attn_workspace_bytes(q.T, k.T, (int32_t)q.H, (int32_t)k.H, (int32_t)q.D, pack.n, pack.host, cuk_host(), causal, window,
                                  fwd, bwd));
  }
};

PyObject* attn_fwd_(PyObject* const* a) {  // ... out lse scratch
  Call c{"attn_fwd"};
  const Attention v(c, a);
  size_t need = 0, bytes = 0;
  v.workspace(c, &need, nullptr);
  void *op, *lp, *sp = nullptr;
  const Tensor out = c.output("out", a[10], {v.q.T, v.q.H, v.q.D}, ScalarType::BFloat16, &op);
  const Tensor lse = c.output("lse", a[11], {v.q.H, v.q.T}, ScalarType::Float, &lp);
  const Tensor scratch = a[12] == Py_None && need == 0 ? Tensor() : c.scratch(a[12], need, &sp, &bytes);
  c.run([&] {
    return attn_fwd(v.q.bf(), v.q.s0, v.q.s1, v.k.bf(), v.k.s0, v.k.s1, v.v.bf(), v.v.s0, v.v.s1, v.pack.cu, v.pack.host, v.cuk(),
                    v.cuk_host(), v.pack.n, v.q.T, v.k.T, (int32_t)v.q.H, (int32_t)v.k.H, (int32_t)v.q.D, v.scale, v.causal,
                    v.window, static_cast<gdr_bf16*>(op), static_cast<float*>(lp), sp, bytes, c.stream);
  });
  return two(out, lse);
}

PyObject* attn_bwd_(PyObject* const* a) {  // ... out lse dout scratch grads
  Call c{"attn_bwd"};
  const Attention v(c, a);
  const auto bf = ScalarType::BFloat16;
  const int64_t qs[3] = {v.q.T, v.q.H, v.q.D}, ks[3] = {v.k.T, v.k.H, v.k.D};
  const auto* out = static_cast<const gdr_bf16*>(c.dense("out", c.tensor("out", a[10]), bf, qs));
  const auto* lse = static_cast<const float*>(c.dense("lse", c.tensor("lse", a[11]), ScalarType::Float, {v.q.H, v.q.T}));
  const Tensor& dt = c.tensor("dout", a[12]);
  const Heads dout(c, "dout", dt, bf);
  if (dt.sizes() != Shape(qs, 3)) c.fail("dout has shape " + str(dt.sizes()) + ", expected " + str(Shape(qs, 3)));
  size_t need = 0, bytes = 0;
  v.workspace(c, nullptr, &need);
  Grads g(a[14]);
  auto* dq = static_cast<gdr_bf16*>(g.tensor(c, "dq", qs, bf));
  auto* dk = static_cast<gdr_bf16*>(g.tensor(c, "dk", ks, bf));
  auto* dv = static_cast<gdr_bf16*>(g.tensor(c, "dv", ks, bf));
  void* sp;
  const Tensor scratch = c.scratch(a[13], need, &sp, &bytes);
  c.run([&] {
    return attn_bwd(v.q.bf(), v.q.s0, v.q.s1, v.k.bf(), v.k.s0, v.k.s1, v.v.bf(), v.v.s0, v.v.s1, out, lse, dout.bf(), dout.s0, dout.s1,
                    v.pack.cu, v.pack.host, v.cuk(), v.cuk_host(), v.pack.n, v.q.T, v.k.T, (int32_t)v.q.H, (int32_t)v.k.H,
                    (int32_t)v.q.D, v.scale, v.causal, v.window, dq, dk, dv, sp, bytes, c.stream);
  });
  return g.release();
}

// --- the module --------------------------------------------------------------------------
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected, got %zd", N, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const PyError&) {
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::bad_alloc&) {
    PyErr_NoMemory();
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}
PyObject* set_check(PyObject*, PyObject* f) {
  Py_XSETREF(g_check, Py_NewRef(f));
  Py_RETURN_NONE;
}

}  // namespace

PyMODINIT_FUNC PyInit__gdr_ops() {
#define GDR_ENTRY(f, n) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(call<f##_, n>)), METH_FASTCALL, nullptr}
  static PyMethodDef table[] = {
      {"set_check", set_check, METH_O, nullptr},
      GDR_ENTRY(sconv_fwd, 10), GDR_ENTRY(sconv_bwd, 12), GDR_ENTRY(sconv_step, 7), GDR_ENTRY(ssm_fwd, 15),
      GDR_ENTRY(ssm_step, 11), GDR_ENTRY(kda_step, 10), GDR_ENTRY(gdn_step, 10), GDR_ENTRY(norm_fwd, 10),
      GDR_ENTRY(norm_bwd, 12), GDR_ENTRY(lnorm_fwd, 8), GDR_ENTRY(lnorm_bwd, 10), GDR_ENTRY(rope, 10), GDR_ENTRY(attn_fwd, 13),
      GDR_ENTRY(attn_bwd, 15), {nullptr, nullptr, 0, nullptr}};
#undef GDR_ENTRY
  static PyModuleDef def = {PyModuleDef_HEAD_INIT, "_gdr_ops", nullptr, -1, table, nullptr, nullptr, nullptr, nullptr};
  return PyModule_Create(&def);
}
