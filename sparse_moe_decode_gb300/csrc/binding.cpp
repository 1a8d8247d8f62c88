// binding.cpp -- the tensor-level calls of the Python package whose kernels
// take a few microseconds (the gated delta rule, the norms around a block):
// argument checks, output allocation and the call of the C ABI without the
// interpreter's cost per attribute.  A CPython extension module; the library's
// functions come in through `init`, so that it links against torch alone.
//
// Every call returns its tensors, or the moe_status it was refused with, or
// kOtherDevice, nothing done, where another device than its tensors' is current.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>

#include "moe_gb300.h"

namespace {

decltype(&moe_delta_chunk) g_chunk;
decltype(&moe_delta_step) g_step;
decltype(&moe_norm_gate_residual) g_norm;

struct Refused {
  int status;
};

constexpr int kOtherDevice = -1;

void require(bool ok) {
  if (!ok) throw Refused{MOE_ERR_INVALID_ARG};
}

const at::Tensor &tensor(PyObject *o) {
  require(THPVariable_Check(o));
  return THPVariable_Unpack(o);
}

// Runs a call; C++ exceptions end here.
template <class F>
PyObject *guarded(F f) {
  try {
    return f();
  } catch (const Refused &r) {
    return PyLong_FromLong(r.status);
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

int64_t integer(PyObject *o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    require(false);
  }
  return v;
}

float real(PyObject *o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    require(false);
  }
  return static_cast<float>(v);
}

void *address(PyObject *o) { return reinterpret_cast<void *>(static_cast<uintptr_t>(integer(o))); }

// The stream of a call: the one whose address is given, or with None the
// current one of `device`.  It is current while this lasts, so that memory made
// for the results comes from its pool and is not still in use by another's work.
class OnStream {
 public:
  OnStream(PyObject *given, int64_t device) {
    const c10::DeviceIndex d = static_cast<c10::DeviceIndex>(device);
    if (c10::cuda::current_device() != d) throw Refused{kOtherDevice};
    const cudaStream_t now = c10::cuda::getCurrentCUDAStream(d).stream();
    stream_ = given == Py_None ? now : static_cast<cudaStream_t>(address(given));
    if (stream_ != now) guard_.reset_stream(c10::cuda::getStreamFromExternal(stream_, d));
  }
  void *get() const { return stream_; }

 private:
  cudaStream_t stream_;
  c10::cuda::OptionalCUDAStreamGuard guard_;
};

void place(const at::Tensor &x, at::ScalarType type, int64_t device) {
  require(x.scalar_type() == type && x.is_cuda() && x.get_device() == device &&
          x.layout() == at::kStrided);
}

// The first stride of x, whose rows have the sizes `row` and lie whole: only
// the first stride is free (a single row has none of its own).
int64_t row_stride(const at::Tensor &x, at::ScalarType type, int64_t device, int64_t rows,
                   at::IntArrayRef row) {
  place(x, type, device);
  const int64_t d = static_cast<int64_t>(row.size());
  require(x.dim() == d + 1 && x.size(0) == rows);
  int64_t whole = 1;
  bool inner = true;
  for (int64_t i = d; i >= 1; --i) {
    require(x.size(i) == row[i - 1]);
    inner = inner && (x.size(i) == 1 || x.stride(i) == whole);
    whole *= row[i - 1];
  }
  require(inner || rows == 0);
  return rows > 1 ? x.stride(0) : whole;
}

// A caller's tensor that a kernel was told to write: autograd sees that what it
// may have kept of it is no longer there.
void written(PyObject *o) {
  if (o == Py_None) return;
  const at::Tensor &x = THPVariable_Unpack(o);
  if (!x.is_inference()) x.unsafeGetTensorImpl()->bump_version();
}

at::Tensor fresh(at::IntArrayRef sizes, int64_t device) {
  return at::empty(sizes, at::TensorOptions()
                              .dtype(at::kBFloat16)
                              .device(at::kCUDA, static_cast<c10::DeviceIndex>(device)));
}

// ------------------------------------------------------------- delta rule

struct Delta {
  moe_delta_dims dims;
  void *workspace;
  size_t ws_bytes;
  int64_t device;
};

constexpr const char *kDelta = "sparse_moe_decode_gb300.delta";

void delta_free(PyObject *capsule) {
  delete static_cast<Delta *>(PyCapsule_GetPointer(capsule, kDelta));
}

// delta(address of a moe_delta_dims, workspace, ws_bytes, device) -> handle
PyObject *delta_handle(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    require(n == 4);
    Delta *h = new Delta{*static_cast<const moe_delta_dims *>(address(a[0])), address(a[1]),
                         static_cast<size_t>(integer(a[2])), integer(a[3])};
    return PyCapsule_New(h, kDelta, delta_free);
  });
}

// What both forms share: the inputs q, k, v, g, beta at a[0..4].
moe_delta_inputs delta_inputs(const Delta &h, PyObject *const *a, int64_t &rows) {
  const moe_delta_dims &d = h.dims;
  const at::Tensor &q = tensor(a[0]), &k = tensor(a[1]), &v = tensor(a[2]), &g = tensor(a[3]),
                   &beta = tensor(a[4]);
  require(q.dim() == 3);
  rows = q.size(0);
  const int64_t qk[2] = {d.qk_heads, d.qk_dim}, vv[2] = {d.v_heads, d.v_dim}, gate[1] = {d.v_heads};
  moe_delta_inputs in;
  in.q_ld = row_stride(q, at::kBFloat16, h.device, rows, qk);
  in.k_ld = row_stride(k, at::kBFloat16, h.device, rows, qk);
  in.v_ld = row_stride(v, at::kBFloat16, h.device, rows, vv);
  in.g_ld = row_stride(g, at::kFloat, h.device, rows, gate);
  in.beta_ld = row_stride(beta, at::kFloat, h.device, rows, gate);
  in.q = static_cast<const moe_bf16 *>(q.const_data_ptr());
  in.k = static_cast<const moe_bf16 *>(k.const_data_ptr());
  in.v = static_cast<const moe_bf16 *>(v.const_data_ptr());
  in.g = static_cast<const float *>(g.const_data_ptr());
  in.beta = static_cast<const float *>(beta.const_data_ptr());
  return in;
}

struct DeltaStates {
  const int32_t *slots = nullptr;
  int64_t n_slots;
  const float *in = nullptr;
  float *out = nullptr;
};

float *delta_state(const Delta &h, const at::Tensor &x, int64_t &n_slots) {
  const moe_delta_dims &d = h.dims;
  place(x, at::kFloat, h.device);
  require(x.dim() == 4 && x.size(1) == d.v_heads && x.size(2) == d.v_dim &&
          x.size(3) == d.qk_dim && x.is_contiguous());
  n_slots = x.size(0);
  return static_cast<float *>(x.mutable_data_ptr());
}

// state_in, state_out and slots (each None or a tensor) at a[0..2]
DeltaStates delta_states(const Delta &h, PyObject *const *a, int64_t B) {
  DeltaStates s;
  s.n_slots = B;
  if (a[0] != Py_None) s.in = delta_state(h, tensor(a[0]), s.n_slots);
  if (a[1] != Py_None) {
    const int64_t before = s.n_slots;
    s.out = delta_state(h, tensor(a[1]), s.n_slots);
    require(a[0] == Py_None || before == s.n_slots);
  }
  if (a[2] != Py_None) {
    const at::Tensor &x = tensor(a[2]);
    place(x, at::kInt, h.device);
    require(x.dim() == 1 && x.size(0) == B && x.is_contiguous());
    s.slots = static_cast<const int32_t *>(x.const_data_ptr());
    // without states there is none to be out of
    if (a[0] == Py_None && a[1] == Py_None) s.n_slots = 1 << 30;
  }
  require(s.n_slots <= INT32_MAX);
  return s;
}

const Delta &delta_of(PyObject *o) {
  const void *p = PyCapsule_GetPointer(o, kDelta);
  if (!p) {
    PyErr_Clear();
    require(false);
  }
  const Delta &h = *static_cast<const Delta *>(p);
  require(h.device >= 0);  // CUDA memory only
  return h;
}

at::Tensor delta_out(const Delta &h, PyObject *o, int64_t rows, int64_t &ld) {
  const int64_t row[2] = {h.dims.v_heads, h.dims.v_dim};
  if (o == Py_None) {
    ld = row[0] * row[1];
    return fresh({rows, row[0], row[1]}, h.device);
  }
  at::Tensor out = tensor(o);
  ld = row_stride(out, at::kBFloat16, h.device, rows, row);
  return out;
}

// a: state_in, state_out, slots, out as they were given
PyObject *delta_result(moe_status st, const at::Tensor &out, PyObject *const *a) {
  if (st != MOE_OK) return PyLong_FromLong(st);
  written(a[1]), written(a[3]);
  return THPVariable_Wrap(out);
}

// chunk(handle, q, k, v, g, beta, state_in, state_out, slots, out, cu_seqlens, stream)
PyObject *delta_chunk(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    require(n == 12);
    const Delta &h = delta_of(a[0]);
    int64_t rows, B = 1, ld;
    const moe_delta_inputs in = delta_inputs(h, a + 1, rows);
    const int32_t *cu = nullptr;
    if (a[10] != Py_None) {
      const at::Tensor &x = tensor(a[10]);
      place(x, at::kInt, h.device);
      require(x.dim() == 1 && x.size(0) >= 1 && x.is_contiguous());
      B = x.size(0) - 1;
      cu = static_cast<const int32_t *>(x.const_data_ptr());
    }
    require(rows <= INT32_MAX && B <= INT32_MAX);
    const DeltaStates s = delta_states(h, a + 6, B);
    const OnStream stream(a[11], h.device);
    const at::Tensor out = delta_out(h, a[9], rows, ld);
    return delta_result(g_chunk(&h.dims, &in, static_cast<int>(rows), cu, static_cast<int>(B),
                                s.slots, static_cast<int>(s.n_slots), s.in, s.out,
                                static_cast<moe_bf16 *>(out.mutable_data_ptr()), ld, h.workspace,
                                h.ws_bytes, stream.get()),
                        out, a + 6);
  });
}

// step(handle, q, k, v, g, beta, state_in, state_out, slots, out, tokens, stream)
PyObject *delta_step(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    require(n == 12);
    const Delta &h = delta_of(a[0]);
    int64_t rows, B, tokens, ld;
    const moe_delta_inputs in = delta_inputs(h, a + 1, rows);
    if (a[10] != Py_None) {
      tokens = integer(a[10]);
      B = tokens > 0 ? rows / tokens : 0;
    } else {
      // as many sequences as slots, or else states; one row each without both
      PyObject *lead = a[8] != Py_None ? a[8] : a[6] != Py_None ? a[6] : a[7];
      if (lead != Py_None) require(tensor(lead).dim() >= 1);
      B = lead == Py_None ? rows : tensor(lead).size(0);
      tokens = B ? rows / B : 0;
    }
    require(B * tokens == rows && rows <= INT32_MAX);
    const DeltaStates s = delta_states(h, a + 6, B);
    const OnStream stream(a[11], h.device);
    const at::Tensor out = delta_out(h, a[9], rows, ld);
    return delta_result(g_step(&h.dims, &in, static_cast<int>(B), static_cast<int>(tokens), s.slots,
                               static_cast<int>(s.n_slots), s.in, s.out,
                               static_cast<moe_bf16 *>(out.mutable_data_ptr()), ld, h.workspace,
                               h.ws_bytes, stream.get()),
                        out, a + 6);
  });
}

// ------------------------------------------------------------------- norm

// norm(x, gamma_post, gate, gate_act, resid, res_scale, gamma_pre, eps,
// resid_out, x_next, stream) -> (resid_out, x_next or None)
PyObject *norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    require(n == 11);
    const at::Tensor &x = tensor(a[0]);
    const int64_t d = x.dim();
    require(x.is_cuda() && (d == 2 || d == 3));
    const int64_t device = x.get_device(), rows = x.size(0), width = x.size(d - 1);
    const int64_t inner = d == 3 ? x.size(1) : 1;
    require(width > 0 && inner > 0 && width <= INT32_MAX && inner <= INT32_MAX);
    const at::IntArrayRef row = x.sizes().slice(1);
    const int64_t channel[1] = {width};
    const auto ptr = [](const at::Tensor &t) {
      return static_cast<moe_bf16 *>(t.mutable_data_ptr());
    };
    const auto ld_of = [&](const at::Tensor &t) {
      return row_stride(t, at::kBFloat16, device, rows, row);
    };
    const auto per_channel = [&](const at::Tensor &t) {
      place(t, at::kBFloat16, device);
      require(t.dim() == 1 && t.size(0) == width && t.is_contiguous());
      return ptr(t);
    };
    moe_norm_args m = {};
    m.rows = rows * inner, m.width = static_cast<int32_t>(width);
    m.inner = static_cast<int32_t>(inner);
    m.x = ptr(x), m.x_ld = ld_of(x);
    if (a[1] != Py_None) m.gamma_post = per_channel(tensor(a[1]));
    if (a[2] != Py_None) {
      const at::Tensor &gate = tensor(a[2]);
      if (gate.sizes() == at::IntArrayRef(channel)) {
        m.gate = per_channel(gate), m.gate_kind = MOE_GATE_CHANNEL;
      } else if (gate.sizes() == x.sizes()) {
        m.gate = ptr(gate), m.gate_ld = ld_of(gate), m.gate_kind = MOE_GATE_ELEMENT;
      } else {
        int64_t one[2] = {1, 1};
        one[0] = d == 3 ? inner : 1;
        m.gate_ld = row_stride(gate, at::kBFloat16, device, rows, at::IntArrayRef(one, d - 1));
        m.gate = ptr(gate), m.gate_kind = MOE_GATE_ROW;
      }
    }
    m.gate_act = static_cast<int32_t>(integer(a[3]));
    if (a[4] != Py_None) m.resid_in = ptr(tensor(a[4])), m.resid_in_ld = ld_of(tensor(a[4]));
    m.res_scale = real(a[5]), m.eps = real(a[7]);
    const OnStream stream(a[10], device);
    const at::Tensor resid = a[8] == Py_None ? fresh(x.sizes(), device) : tensor(a[8]);
    m.resid_out = ptr(resid), m.resid_out_ld = ld_of(resid);
    at::Tensor next;
    require(a[6] != Py_None || a[9] == Py_None);
    if (a[6] != Py_None) {
      m.gamma_pre = per_channel(tensor(a[6]));
      next = a[9] == Py_None ? fresh(x.sizes(), device) : tensor(a[9]);
      m.x_next = ptr(next), m.x_next_ld = ld_of(next);
    }
    const moe_status st = g_norm(&m, stream.get());
    if (st != MOE_OK) return PyLong_FromLong(st);
    written(a[8]), written(a[9]);
    PyObject *both = PyTuple_New(2);
    if (!both) return nullptr;
    PyObject *r = THPVariable_Wrap(resid), *x2 = Py_None;
    if (m.x_next) x2 = THPVariable_Wrap(next);
    else Py_INCREF(Py_None);
    PyTuple_SET_ITEM(both, 0, r);
    PyTuple_SET_ITEM(both, 1, x2);
    return both;
  });
}

// init(moe_delta_chunk, moe_delta_step, moe_norm_gate_residual): addresses
PyObject *init(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> PyObject * {
    require(n == 3);
    g_chunk = reinterpret_cast<decltype(g_chunk)>(address(a[0]));
    g_step = reinterpret_cast<decltype(g_step)>(address(a[1]));
    g_norm = reinterpret_cast<decltype(g_norm)>(address(a[2]));
    Py_RETURN_NONE;
  });
}

#define METHOD(name, f) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}

PyMethodDef kMethods[] = {METHOD("init", init),
                          METHOD("delta", delta_handle),
                          METHOD("delta_chunk", delta_chunk),
                          METHOD("delta_step", delta_step),
                          METHOD("norm", norm),
                          {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&kModule); }
