// The layer operators' calls on torch tensors: checks of the arguments,
// allocation of outputs, and the C entry point (gdn.h), in one native call.
// The steps run a few microseconds on the GPU, so what a call costs on the
// host is most of its time; the same checks in Python take as long again as
// the launch.  layer.py documents the calls and passes their arguments on by
// position; the entry points' addresses come from the loaded library (init).
#include <ATen/core/Tensor.h>
#include <ATen/hip/EmptyTensor.h>
#include <c10/core/DeviceGuard.h>
#include <c10/core/StreamGuard.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "gdn.h"

namespace {

using at::Tensor;
using c10::IntArrayRef;
using c10::ScalarType;

decltype(&gdn_conv_forward) f_conv_forward;
decltype(&gdn_conv_step) f_conv_step;
decltype(&gdn_ssm_workspace_bytes) f_ssm_workspace;
decltype(&gdn_ssm_forward) f_ssm_forward;
decltype(&gdn_ssm_step) f_ssm_step;
decltype(&gdn_rotary) f_rotary;
decltype(&gdn_step) f_step;
PyObject* gdn_error;  // the package's exception, made from a status

struct Refused {  // becomes a Python exception
  PyObject* type;
  std::string what;
};
struct Failed {
  int status;
};
[[noreturn]] void refuse(std::string what) { throw Refused{PyExc_ValueError, std::move(what)}; }

std::string text(IntArrayRef s) {
  std::string t = "[";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + "]";
}
const char* text(ScalarType t) {
  return t == at::kFloat ? "float32" : t == at::kBFloat16 ? "bfloat16" : t == at::kInt ? "int32" : t == at::kDouble ? "float64" : t == at::kByte ? "uint8" : "?";
}

// an argument: a tensor, or null for None
const Tensor* tensor(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, std::string(name) + " must be a tensor"};
  const Tensor& t = THPVariable_Unpack(o);
  if (t.is_neg()) refuse(std::string(name) + " is a negated view: its memory holds other values (resolve_neg)");
  return &t;
}
const Tensor& given(PyObject* o, const char* name) {
  const Tensor* t = tensor(o, name);
  if (!t) refuse(std::string(name) + " must be given");
  return *t;
}

// numbers, checked before anything is launched
int64_t whole(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused{PyExc_TypeError, std::string(name) + " must be a whole number (of 64 bits)"};
  }
  return v;
}
float real(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused{PyExc_TypeError, std::string(name) + " must be a number"};
  }
  return (float)v;
}

int kind_of(const Tensor& x, const char* name) {
  const ScalarType t = x.scalar_type();
  if (t != at::kFloat && t != at::kBFloat16) throw Refused{PyExc_TypeError, std::string(name) + " must be float32 or bfloat16"};
  if (!x.is_cuda()) refuse(std::string(name) + " must be a CUDA tensor");
  return t == at::kFloat ? GDN_DTYPE_F32 : GDN_DTYPE_BF16;
}

void want(const Tensor& t, IntArrayRef shape, ScalarType type, const Tensor& like, const char* name) {
  if (t.scalar_type() != type || t.sizes() != shape || !t.is_contiguous() || t.device() != like.device())
    refuse(std::string(name) + " must be contiguous " + text(type) + " " + text(shape) + " on " + like.device().str());
}
template <typename T = const float>
T* param(const Tensor* t, IntArrayRef shape, ScalarType type, const Tensor& like, const char* name) {
  if (!t) return nullptr;
  want(*t, shape, type, like, name);
  return static_cast<T*>(t->data_ptr());
}

// rows whose last dimension is contiguous
void rows(const Tensor& t, IntArrayRef shape, const Tensor& like, const char* name) {
  if (t.scalar_type() != like.scalar_type() || t.sizes() != shape || t.device() != like.device())
    refuse(std::string(name) + " must be " + text(like.scalar_type()) + " " + text(shape) + " on " + like.device().str());
  if (shape.back() != 1 && t.stride(-1) != 1 && t.numel()) refuse(std::string(name) + ": the last dimension must be contiguous");
}

void* ptr(const Tensor* t) { return t ? t->data_ptr() : nullptr; }

// (its rows of no sequence hold nothing yet)
int32_t unused_rows(const Tensor* out) { return out ? 0 : GDN_LAYER_OPT_ZERO_UNUSED; }

// The stream of a call: the current one of the tensors' device, or the
// caller's.  What the call allocates belongs to it: a block of another stream's
// memory may still be read or written by that stream's earlier work.  Tensors
// that the caller gets back are meant for the current stream too, which keeps
// their blocks from reuse when they are freed.
struct Stream {
  void* raw;
  bool other = false;
  c10::Stream stream;
  c10::Device device;
  Stream(PyObject* o, const Tensor& x) : raw(nullptr), stream(c10::Stream::DEFAULT, x.device()), device(x.device()) {
    const c10::hip::HIPStream now = c10::hip::getCurrentHIPStream(x.get_device());
    raw = now.stream();
    if (o == Py_None) return;
    const long long v[4] = {number(o, "cuda_stream"), number(o, "stream_id"), number(o, "device_index"), number(o, "device_type")};
    if (v[2] != x.get_device()) refuse("stream must be one of " + x.device().str());
    other = reinterpret_cast<void*>(v[0]) != raw;
    raw = reinterpret_cast<void*>(v[0]);
    stream = c10::Stream::unpack3(v[1], (c10::DeviceIndex)v[2], (c10::DeviceType)v[3]);
  }
  static long long number(PyObject* o, const char* name) {
    PyObject* a = PyObject_GetAttrString(o, name);
    const long long v = a ? PyLong_AsLongLong(a) : -1;
    Py_XDECREF(a);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      throw Refused{PyExc_TypeError, "stream must be a torch.cuda.Stream"};
    }
    return v;
  }
  // (without the dispatcher's part of a call, 0.3 us)
  Tensor fresh(IntArrayRef sizes, ScalarType type, bool returned = true) const {
    if (!other) return at::detail::empty_cuda(sizes, type, device, std::nullopt);
    Tensor t;
    {
      const c10::StreamGuard guard(stream);
      t = at::detail::empty_cuda(sizes, type, device, std::nullopt);
    }
    if (returned) t.record_stream(c10::impl::VirtualGuardImpl(device.type()).getStream(device));
    return t;
  }
};

Tensor output(const Stream& s, const Tensor* out, const Tensor& like, const char* name = "out") {
  if (!out) return s.fresh(like.sizes(), like.scalar_type());
  rows(*out, like.sizes(), like, name);
  return *out;
}

void check(gdn_status_t st) {
  if (st != GDN_OK) throw Failed{(int)st};
}

// (sequences, tokens) of x: [B, T, D], or [T, D] with offsets
void lead(const Tensor& x, const Tensor* off, int64_t* B, int64_t* T) {
  if (!off) {
    if (x.dim() != 3) refuse("x must be [B, T, D] (or [T, D] with seq_offsets)");
    *B = x.size(0);
    *T = x.size(1);
    return;
  }
  if (x.dim() != 2) refuse("x must be [T, D] with seq_offsets");
  if (off->scalar_type() != at::kInt || off->dim() != 1 || off->size(0) < 2 || !off->is_contiguous() || off->device() != x.device())
    refuse("seq_offsets must be contiguous int32 [B + 1] on " + x.device().str());
  *B = off->size(0) - 1;
  *T = x.size(0);
}

// A prompt's states [slots, d1, d2]: checked; a final state is allocated if
// one is wanted and none given.
struct States {
  int64_t slots;
  Tensor out;  // undefined: none
  States(const Stream& s, int64_t B, int64_t d1, int64_t d2, ScalarType type, const Tensor& x, const Tensor* in, const Tensor* given_out,
         const Tensor* index, bool wanted)
      : slots(B) {
    if (index) want(*index, {B}, at::kInt, x, "state_index");
    if (const Tensor* g = in ? in : given_out) {
      slots = g->dim() ? g->size(0) : 0;
      if (!index && slots != B) refuse("a state of " + std::to_string(slots) + " slots needs state_index for " + std::to_string(B) + " sequences");
    }
    if (in) want(*in, {slots, d1, d2}, type, x, "state_in");
    if (given_out) {
      want(*given_out, {slots, d1, d2}, type, x, "state_out");
      out = *given_out;
    } else if (wanted) {
      if (index) refuse("state_out must be given with state_index (or want_state=False)");
      out = s.fresh({B, d1, d2}, type);
    }
  }
  void* address() const { return out.defined() ? out.data_ptr() : nullptr; }
};

// a step's state: [slots, ...tail], advanced in place
int64_t step_slots(const Tensor& state, IntArrayRef tail, ScalarType type, const Tensor& x, const Tensor* index, int64_t B) {
  if (state.dim() != (int64_t)tail.size() + 1 || state.sizes().slice(1) != tail || state.scalar_type() != type ||
      state.device() != x.device() || !state.is_contiguous())
    refuse(std::string("state must be contiguous ") + text(type) + " [slots, ...] with " + text(tail) + " on " + x.device().str());
  if (index) want(*index, {B}, at::kInt, x, "state_index");
  else if (state.size(0) != B)
    refuse("a state of " + std::to_string(state.size(0)) + " slots needs state_index for " + std::to_string(B) + " sequences");
  return state.size(0);
}

PyObject* pair(const Tensor& a, const Tensor& b) {
  PyObject* x = THPVariable_Wrap(a);
  PyObject* y = b.defined() ? THPVariable_Wrap(b) : Py_NewRef(Py_None);
  return Py_BuildValue("(NN)", x, y);
}

// ---- the calls (arguments by position; see layer.py) ----

// x, weight, bias, state_in, act, seq_offsets, state_index, out, state_out, want_state, stream
PyObject* conv(PyObject* const* a) {
  const Tensor &x = given(a[0], "x"), &w = given(a[1], "weight");
  const Tensor *bias = tensor(a[2], "bias"), *in = tensor(a[3], "state_in"), *off = tensor(a[5], "seq_offsets");
  const Tensor *index = tensor(a[6], "state_index"), *out = tensor(a[7], "out"), *so = tensor(a[8], "state_out");
  gdn_conv_problem_t p = {};
  p.dtype = kind_of(x, "x");
  lead(x, off, &p.B, &p.T);
  const int64_t D = x.size(-1), W = w.dim() == 2 ? w.size(1) : 0;
  rows(x, x.sizes(), x, "x");
  const float* pw = param(&w, {D, W}, at::kFloat, x, "weight");
  const float* pb = param(bias, {D}, at::kFloat, x, "bias");
  const Stream s(a[10], x);
  const States st(s, p.B, W - 1, D, x.scalar_type(), x, in, so, index, a[9] == Py_True);
  const Tensor y = output(s, out, x);
  p.D = D;
  p.x_stride_b = off ? 0 : x.stride(0);
  p.x_stride_t = x.stride(-2);
  p.out_stride_b = off ? 0 : y.stride(0);
  p.out_stride_t = y.stride(-2);
  p.slots = st.slots;
  p.width = (int32_t)W;
  p.activation = (int32_t)whole(a[4], "activation");
  p.options = unused_rows(out);
  p.seq_offsets = static_cast<const int32_t*>(ptr(off));
  p.state_index = static_cast<const int32_t*>(ptr(index));
  p.stream = s.raw;
  const c10::DeviceGuard guard(x.device());
  check(f_conv_forward(&p, x.data_ptr(), pw, pb, ptr(in), st.address(), y.data_ptr()));
  return pair(y, st.out);
}

// x, weight, bias, state, act, state_index, out, stream
PyObject* conv_step(PyObject* const* a) {
  const Tensor &x = given(a[0], "x"), &w = given(a[1], "weight"), &state = given(a[3], "state");
  const Tensor *bias = tensor(a[2], "bias"), *index = tensor(a[5], "state_index"), *out = tensor(a[6], "out");
  gdn_conv_problem_t p = {};
  p.dtype = kind_of(x, "x");
  if (x.dim() != 2) refuse("x must be [B, D]");
  p.B = x.size(0);
  const int64_t D = x.size(1), W = w.dim() == 2 ? w.size(1) : 0;
  rows(x, x.sizes(), x, "x");
  const float* pw = param(&w, {D, W}, at::kFloat, x, "weight");
  const float* pb = param(bias, {D}, at::kFloat, x, "bias");
  p.slots = step_slots(state, {W - 1, D}, x.scalar_type(), x, index, p.B);
  const Stream s(a[7], x);
  const Tensor y = output(s, out, x);
  p.T = 1;
  p.D = D;
  p.x_stride_b = x.stride(0);
  p.out_stride_b = y.stride(0);
  p.width = (int32_t)W;
  p.activation = (int32_t)whole(a[4], "activation");
  p.options = unused_rows(out);
  p.state_index = static_cast<const int32_t*>(ptr(index));
  p.stream = s.raw;
  const c10::DeviceGuard guard(x.device());
  check(f_conv_step(&p, x.data_ptr(), pw, pb, state.data_ptr(), y.data_ptr()));
  return THPVariable_Wrap(y);
}

// x, dt, A, B, C, D, z, dt_bias at a[0..7]: checked, and everything of the
// problem that prompts and steps share
struct Ssm {
  gdn_ssm_problem_t p = {};
  const Tensor &x, &dt, &A, &B, &C;
  const Tensor* z;
  const float* rates;
  explicit Ssm(PyObject* const* a)
      : x(given(a[0], "x")), dt(given(a[1], "dt")), A(given(a[2], "A")), B(given(a[3], "B")), C(given(a[4], "C")),
        z(tensor(a[6], "z")) {
    p.dtype = kind_of(x, "x");
    if (A.dim() != 2) refuse("A must be [D, N]");
    if (x.dim() < 2) refuse("x must have rows");
    const int64_t D = x.size(-1), N = A.size(1);
    const bool grouped = B.dim() == x.dim() + 1;
    const int64_t G = grouped ? B.size(-2) : 1;
    c10::SmallVector<int64_t, 5> tail(x.sizes().begin(), x.sizes().end() - 1);
    if (grouped) tail.push_back(G);
    tail.push_back(N);
    rows(x, x.sizes(), x, "x");
    rows(dt, x.sizes(), x, "dt");
    rows(B, tail, x, "B");
    rows(C, tail, x, "C");
    if (z) rows(*z, x.sizes(), x, "z");
    if (G < 1 || D % G) refuse(std::to_string(G) + " groups do not divide " + std::to_string(D) + " channels");
    if (G != 1 && B.numel() && (B.stride(-2) != N || C.stride(-2) != N)) refuse("B, C: the last two dimensions must be contiguous");
    rates = param(&A, {D, N}, at::kFloat, x, "A");
    p.skip = param(tensor(a[5], "D"), {D}, at::kFloat, x, "D");
    p.dt_bias = param(tensor(a[7], "dt_bias"), {D}, at::kFloat, x, "dt_bias");
    p.options = a[8] == Py_True ? GDN_SSM_OPT_SOFTPLUS : 0;
    p.D = D;
    p.N = N;
    p.G = G;
    p.z = ptr(z);
  }
  // token and sequence strides: of dimensions `t` and `b` (b < 0: none)
  void strides(const Tensor& y, int b, int t) {
    auto of = [](const Tensor& r, int i) { return i < 0 ? 0 : r.stride(i); };
    p.x_stride_b = of(x, b), p.x_stride_t = of(x, t);
    p.dt_stride_b = of(dt, b), p.dt_stride_t = of(dt, t);
    if (z) p.z_stride_b = of(*z, b), p.z_stride_t = of(*z, t);
    p.b_stride_b = of(B, b), p.b_stride_t = of(B, t);
    p.c_stride_b = of(C, b), p.c_stride_t = of(C, t);
    p.out_stride_b = of(y, b), p.out_stride_t = of(y, t);
  }
};

// x, dt, A, B, C, D, z, dt_bias, softplus, state_in, seq_offsets, state_index, out, state_out, want_state, workspace, stream
PyObject* ssm(PyObject* const* a) {
  Ssm q(a);
  gdn_ssm_problem_t& p = q.p;
  const Tensor& x = q.x;
  const Tensor *in = tensor(a[9], "state_in"), *off = tensor(a[10], "seq_offsets"), *index = tensor(a[11], "state_index");
  const Tensor *out = tensor(a[12], "out"), *so = tensor(a[13], "state_out"), *ws = tensor(a[15], "workspace");
  lead(x, off, &p.B, &p.T);
  const Stream s(a[16], x);
  const States st(s, p.B, p.D, p.N, at::kFloat, x, in, so, index, a[14] == Py_True);
  const Tensor y = output(s, out, x);
  q.strides(y, off ? -1 : 0, off ? 0 : 1);
  p.options |= unused_rows(out);
  p.slots = st.slots;
  p.seq_offsets = static_cast<const int32_t*>(ptr(off));
  p.state_index = static_cast<const int32_t*>(ptr(index));
  Tensor mine;  // freed when the call returns: later work of its stream may have it
  if (const int64_t size = (int64_t)f_ssm_workspace(&p)) {
    if (ws && (ws->scalar_type() != at::kByte || ws->device() != x.device() || !ws->is_contiguous()))
      refuse("workspace must be a contiguous uint8 tensor on " + x.device().str());
    if (!ws || ws->numel() < size) mine = s.fresh({size}, at::kByte, false);
    const Tensor& w = mine.defined() ? mine : *ws;
    p.workspace = w.data_ptr();
    p.workspace_bytes = (size_t)w.numel();
  }
  p.stream = s.raw;
  const c10::DeviceGuard guard(x.device());
  check(f_ssm_forward(&p, x.data_ptr(), q.dt.data_ptr(), q.rates, q.B.data_ptr(), q.C.data_ptr(),
                      static_cast<const float*>(ptr(in)), static_cast<float*>(st.address()), y.data_ptr()));
  return pair(y, st.out);
}

// x, dt, A, B, C, D, z, dt_bias, softplus, state, state_index, out, stream
PyObject* ssm_step(PyObject* const* a) {
  Ssm q(a);
  gdn_ssm_problem_t& p = q.p;
  const Tensor &x = q.x, &state = given(a[9], "state");
  const Tensor *index = tensor(a[10], "state_index"), *out = tensor(a[11], "out");
  if (x.dim() != 2) refuse("x must be [S, D]");
  p.B = x.size(0);
  p.T = 1;
  p.slots = step_slots(state, {p.D, p.N}, at::kFloat, x, index, p.B);
  const Stream s(a[12], x);
  const Tensor y = output(s, out, x);
  q.strides(y, 0, -1);
  p.options |= unused_rows(out);
  p.state_index = static_cast<const int32_t*>(ptr(index));
  p.stream = s.raw;
  const c10::DeviceGuard guard(x.device());
  check(f_ssm_step(&p, x.data_ptr(), q.dt.data_ptr(), q.rates, q.B.data_ptr(), q.C.data_ptr(),
                   static_cast<float*>(state.data_ptr()), y.data_ptr()));
  return THPVariable_Wrap(y);
}

// q, k, inv_freq, positions, options, sections, scale, position0, q_out, k_out, stream
PyObject* rotary(PyObject* const* a) {
  const Tensor &q = given(a[0], "q"), &f = given(a[2], "inv_freq");
  const Tensor *k = tensor(a[1], "k"), *pos = tensor(a[3], "positions"), *qo = tensor(a[8], "q_out"), *ko = tensor(a[9], "k_out");
  gdn_rotary_problem_t p = {};
  p.dtype = kind_of(q, "q");
  if (q.dim() != 4) refuse("q must be [B, T, H, d]");
  if (f.dim() != 1) refuse("inv_freq must be [rot / 2]");
  p.B = q.size(0), p.T = q.size(1), p.Hq = q.size(2), p.d = q.size(3);
  const int64_t pairs = f.size(0);
  p.rot = 2 * pairs;
  want(f, {pairs}, at::kDouble, q, "inv_freq");
  rows(q, q.sizes(), q, "q");
  if (k) {
    if (k->dim() != 4) refuse("k must be [B, T, H, d]");
    p.Hk = k->size(2);
    rows(*k, {p.B, p.T, p.Hk, p.d}, q, "k");
  } else if (ko) {
    refuse("k_out without k");
  }
  p.axes = 1;
  if (pos) {
    const ScalarType t = pos->scalar_type();
    if ((t != at::kInt && t != at::kLong) || pos->device() != q.device() || !pos->is_contiguous())
      refuse("positions must be contiguous int32 or int64 on " + q.device().str());
    if ((pos->dim() != 2 && pos->dim() != 3) || pos->size(-2) != p.B || pos->size(-1) != p.T)
      refuse("positions must be " + text({p.B, p.T}) + " or [axes, ...]");
    if (pos->dim() == 3) {
      if (pos->size(0) < 1 || pos->size(0) > 4) refuse("positions have 1 to 4 axes");
      p.axes = (int32_t)pos->size(0);
    }
    p.position_bits = t == at::kLong ? 64 : 32;
  }
  if (a[5] == Py_None) {
    if (p.axes != 1) refuse("several axes need sections");
    p.section[0] = (int32_t)pairs;
  } else {
    PyObject* seq = PySequence_Fast(a[5], "");
    const Py_ssize_t n = seq ? PySequence_Fast_GET_SIZE(seq) : -1;
    long long v[4] = {0, 0, 0, 0};
    for (Py_ssize_t i = 0; i < n && i < 4; ++i) v[i] = PyLong_AsLongLong(PySequence_Fast_GET_ITEM(seq, i));
    Py_XDECREF(seq);
    if (PyErr_Occurred()) {
      PyErr_Clear();
      throw Refused{PyExc_TypeError, "sections must be whole numbers"};
    }
    for (int i = 0; i < 4; ++i) {
      if (v[i] < 0 || v[i] > pairs) refuse("sections must be between 0 and the number of pairs");
      p.section[i] = (int32_t)v[i];
    }
    if (n != p.axes) refuse("sections must give the pairs of each of " + std::to_string(p.axes) + " axes");
    if (n == 1 && p.section[0] != pairs) refuse("sections must add up to " + std::to_string(pairs) + " pairs");
  }
  const Stream s(a[10], q);
  const Tensor y = output(s, qo, q, "q_out");
  Tensor yk;
  if (k) {
    yk = output(s, ko, *k, "k_out");
    p.k_stride_b = k->stride(0), p.k_stride_t = k->stride(1), p.k_stride_h = k->stride(2);
    p.k_out_stride_b = yk.stride(0), p.k_out_stride_t = yk.stride(1), p.k_out_stride_h = yk.stride(2);
  }
  p.q_stride_b = q.stride(0), p.q_stride_t = q.stride(1), p.q_stride_h = q.stride(2);
  p.q_out_stride_b = y.stride(0), p.q_out_stride_t = y.stride(1), p.q_out_stride_h = y.stride(2);
  p.options = (int32_t)whole(a[4], "options");
  p.scale = real(a[6], "scale");
  p.position0 = whole(a[7], "position0");
  p.stream = s.raw;
  const c10::DeviceGuard guard(q.device());
  check(f_rotary(&p, q.data_ptr(), ptr(k), static_cast<const double*>(f.data_ptr()), ptr(pos), y.data_ptr(),
                 yk.defined() ? yk.data_ptr() : nullptr));
  return pair(y, yk);
}

// q, k, v, log_alpha, beta, state, state_index, options, gate, norm_weight, norm_eps, out, stream
PyObject* delta_step(PyObject* const* a) {
  const Tensor &q = given(a[0], "q"), &k = given(a[1], "k"), &v = given(a[2], "v"), &la = given(a[3], "log_alpha");
  const Tensor &beta = given(a[4], "beta"), &state = given(a[5], "state");
  const Tensor *index = tensor(a[6], "state_index"), *gate = tensor(a[8], "gate"), *nw = tensor(a[9], "norm_weight"), *out = tensor(a[11], "out");
  gdn_step_problem_t p = {};
  p.dtype = kind_of(q, "q");
  if (q.dim() != 3 || v.dim() != 3) refuse("q, k must be [B, H, dk] and v [B, H, dv]");
  const ScalarType type = q.scalar_type();
  p.B = q.size(0), p.H = q.size(1), p.dk = q.size(2), p.dv = v.size(2);
  want(q, q.sizes(), type, q, "q");
  want(k, q.sizes(), type, q, "k");
  want(v, {p.B, p.H, p.dv}, type, q, "v");
  want(la, {p.B, p.H}, at::kFloat, q, "log_alpha");
  want(beta, {p.B, p.H}, at::kFloat, q, "beta");
  p.slots = step_slots(state, {p.H, p.dv, p.dk}, at::kFloat, q, index, p.B);
  if (gate) {
    p.gate = param<void>(gate, {p.B, p.H, p.dv}, type, q, "gate");
    if (!nw) refuse("norm_weight must be given with gate");
    p.norm_weight = param(nw, {p.dv}, at::kFloat, q, "norm_weight");
  }
  const Stream s(a[12], q);
  Tensor y;
  if (out) {
    want(*out, {p.B, p.H, p.dv}, at::kFloat, q, "out");
    y = *out;
  } else {
    y = s.fresh({p.B, p.H, p.dv}, at::kFloat);
  }
  p.options = (int32_t)whole(a[7], "options") | unused_rows(out);
  p.norm_eps = real(a[10], "norm_eps");
  p.state_index = static_cast<const int32_t*>(ptr(index));
  p.stream = s.raw;
  const c10::DeviceGuard guard(q.device());
  check(f_step(&p, q.data_ptr(), k.data_ptr(), v.data_ptr(), static_cast<const float*>(la.data_ptr()),
               static_cast<const float*>(beta.data_ptr()), static_cast<float*>(state.data_ptr()), static_cast<float*>(y.data_ptr())));
  return THPVariable_Wrap(y);
}

// torch's own exception for it (which its C++ interface does not export)
void raise_out_of_memory(const char* what) {
  PyObject* torch = PyImport_ImportModule("torch");
  PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
  if (type) PyErr_SetString(type, what);
  Py_XDECREF(type);
  Py_XDECREF(torch);
}

// No exception leaves a call but as a Python one.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments expected", N);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& e) {
    PyErr_SetString(e.type, e.what.c_str());
  } catch (const Failed& e) {
    PyObject* status = PyLong_FromLong(e.status);
    PyErr_SetObject(gdn_error, status);
    Py_XDECREF(status);
  } catch (const c10::OutOfMemoryError& e) {
    raise_out_of_memory(e.what_without_backtrace());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// the exception class, then the entry points' addresses in this order
PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "8 arguments expected");
    return nullptr;
  }
  void* f[7];
  for (int i = 0; i < 7; ++i) f[i] = PyLong_AsVoidPtr(a[i + 1]);
  if (PyErr_Occurred()) return nullptr;
  f_conv_forward = reinterpret_cast<decltype(f_conv_forward)>(f[0]);
  f_conv_step = reinterpret_cast<decltype(f_conv_step)>(f[1]);
  f_ssm_workspace = reinterpret_cast<decltype(f_ssm_workspace)>(f[2]);
  f_ssm_forward = reinterpret_cast<decltype(f_ssm_forward)>(f[3]);
  f_ssm_step = reinterpret_cast<decltype(f_ssm_step)>(f[4]);
  f_rotary = reinterpret_cast<decltype(f_rotary)>(f[5]);
  f_step = reinterpret_cast<decltype(f_step)>(f[6]);
  Py_INCREF(a[0]);
  Py_XSETREF(gdn_error, a[0]);
  Py_RETURN_NONE;
}

#define GDN_CALL(name, F, N) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {
    {"init", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(init)), METH_FASTCALL, nullptr},
    GDN_CALL("causal_conv", conv, 11),
    GDN_CALL("causal_conv_step", conv_step, 8),
    GDN_CALL("selective_scan", ssm, 17),
    GDN_CALL("selective_step", ssm_step, 13),
    GDN_CALL("rotary", rotary, 11),
    GDN_CALL("delta_step", delta_step, 13),
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
