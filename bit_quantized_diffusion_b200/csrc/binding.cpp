// binding.cpp -- the Python binding of the 8-bit linear and of rotary positions: checks of
// tensors, their addresses and strides, the current stream, and the call of the C ABI.
//
// These calls run once per layer and token in a decoding loop, several in a row on the same
// stream, where the device work is a few microseconds. The same checks in Python through
// ctypes took 8.7 us per call, these take 2.9, launch included; what is checked and raised is the same. Tensors
// the caller does not give are allocated from the pool of the stream that the call runs on.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdint>
#include <optional>
#include <string>

#include "../../include/svdq.h"

namespace {

using at::ScalarType;
using at::Tensor;

constexpr int64_t kIntMax = 2147483647;

// Where a call runs: the current device, and the stream that was given or its current one.
struct Place {
  c10::DeviceIndex device;
  cudaStream_t stream;
  bool given;

  // `first` is any tensor of the call: without a CUDA tensor there may be no device to ask.
  Place(const Tensor& first, const char* name, PyObject* s) : given(s != Py_None) {
    TORCH_CHECK_VALUE(first.is_cuda(), name, ": expected a CUDA tensor");
    device = c10::cuda::current_device();
    if (!given) {
      stream = c10::cuda::getCurrentCUDAStream(device).stream();
    } else {
      PyObject* handle = PyLong_Check(s) ? Py_NewRef(s) : PyObject_GetAttrString(s, "cuda_stream");
      if (handle == nullptr) throw python_error();
      stream = static_cast<cudaStream_t>(PyLong_AsVoidPtr(handle));
      Py_DECREF(handle);
      if (PyErr_Occurred()) throw python_error();
    }
  }

  Tensor empty(at::IntArrayRef shape, ScalarType type) const {
    std::optional<c10::cuda::CUDAStreamGuard> guard;
    if (given) guard.emplace(c10::cuda::getStreamFromExternal(stream, device));
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, device));
  }
};

const Tensor& tensor(PyObject* o, const char* name) {
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  return THPVariable_Unpack(o);
}

void check(const Tensor& t, at::IntArrayRef shape, ScalarType type, const Place& p, const char* name) {
  TORCH_CHECK_VALUE(t.scalar_type() == type && t.sizes() == shape, name, " must be ", type, " ", shape, ", not ",
                    t.scalar_type(), " ", t.sizes());
  TORCH_CHECK_VALUE(t.is_cuda(), name, ": expected a CUDA tensor");
  TORCH_CHECK_VALUE(t.get_device() == p.device, name, " on ", t.device(), ", but the current device is cuda:",
                    static_cast<int>(p.device), ": call under torch.cuda.device(", t.device(), ")");
}

// A contiguous tensor of one shape and type.
void* flat(const Tensor& t, at::IntArrayRef shape, ScalarType type, const Place& p, const char* name) {
  check(t, shape, type, p, name);
  TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
  return t.data_ptr();
}
void* flat(PyObject* o, at::IntArrayRef shape, ScalarType type, const Place& p, const char* name) {
  return o == Py_None ? nullptr : flat(tensor(o, name), shape, type, p, name);
}

// A matrix whose rows are contiguous.
struct Rows {
  void* at = nullptr;
  int ld = 0;
  Rows() = default;
  Rows(const Tensor& t, int64_t rows, int64_t cols, ScalarType type, const Place& p, const char* name) {
    check(t, {rows, cols}, type, p, name);
    const int64_t stride = rows > 1 ? t.stride(0) : cols;
    TORCH_CHECK_VALUE(t.stride(1) == 1 && stride >= 0 && stride <= kIntMax, name,
                      ": rows must be contiguous, their stride below 2^31");
    at = t.data_ptr();
    ld = static_cast<int>(stride);
  }
};

// [M, heads, D] whose heads are contiguous.
struct Heads {
  void* at;
  int ld, ldh;
  Heads(const Tensor& t, at::IntArrayRef shape, ScalarType type, const Place& p, const char* name) {
    check(t, shape, type, p, name);
    // (one row or one head has no step to the next)
    const int64_t h = shape[1] > 1 ? t.stride(1) : shape[2], m = shape[0] > 1 ? t.stride(0) : shape[2];
    TORCH_CHECK_VALUE(t.stride(2) == 1 && h >= 0 && m >= 0 && h <= kIntMax && m <= kIntMax, name,
                      ": heads must be contiguous, strides below 2^31");
    at = t.data_ptr();
    ld = static_cast<int>(m);
    ldh = static_cast<int>(h);
  }
};

svdq_out out_type(ScalarType t, const char* what) {
  TORCH_CHECK_VALUE(t == ScalarType::BFloat16 || t == ScalarType::Float, what, " must be bfloat16 or float32");
  return t == ScalarType::Float ? SVDQ_OUT_F32 : SVDQ_OUT_BF16;
}

svdq_act activation(PyObject* o) {
  if (o == Py_None) return SVDQ_ACT_NONE;
  const char* s = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
  if (s != nullptr) {
    const std::string name(s);
    if (name == "none") return SVDQ_ACT_NONE;
    if (name == "gelu") return SVDQ_ACT_GELU;
    if (name == "silu") return SVDQ_ACT_SILU;
  }
  PyErr_Clear();
  TORCH_CHECK_VALUE(false, "activation must be None, 'gelu' or 'silu'");
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

// The library's call without the interpreter's lock; its status raised as SvdqError.
template <typename F>
void call(const char* where, F&& f) {
  svdq_status st;
  Py_BEGIN_ALLOW_THREADS
  st = f();
  Py_END_ALLOW_THREADS
  if (st == SVDQ_OK) return;
  PyObject* native = PyImport_ImportModule("bit_quantized_diffusion_b200._native");
  if (native != nullptr) {
    Py_XDECREF(PyObject_CallMethod(native, "check", "is", static_cast<int>(st), where));
    Py_DECREF(native);
  }
  throw python_error();
}

PyObject* owned(PyObject* given, const Tensor& t) { return given != Py_None ? Py_NewRef(given) : THPVariable_Wrap(t); }

void arity(const char* name, Py_ssize_t n, Py_ssize_t want) {
  TORCH_CHECK_TYPE(n == want, name, ": ", want, " arguments, got ", n);
}

// what both quantizers take: X, codes, scale
struct Quantize {
  Tensor X, codes, scale;
  int64_t M, K;
  Place place;
  svdq_out type;
  Rows x;
  void *pc, *ps;

  Quantize(PyObject* ox, PyObject* oc, PyObject* os, PyObject* stream)
      : X(tensor(ox, "X")), M(shape(X)), K(X.size(1)), place(X, "X", stream), type(out_type(X.scalar_type(), "X")),
        x(X, M, K, X.scalar_type(), place, "X") {
    codes = oc == Py_None ? place.empty({M, K}, ScalarType::Float8_e4m3fn) : tensor(oc, "codes");
    scale = os == Py_None ? place.empty({M}, ScalarType::Float) : tensor(os, "scale");
    pc = flat(codes, {M, K}, ScalarType::Float8_e4m3fn, place, "codes");
    ps = flat(scale, {M}, ScalarType::Float, place, "scale");
  }
  static int64_t shape(const Tensor& X) {
    TORCH_CHECK_VALUE(X.dim() == 2, "X must be a 2-D bf16 or float32 tensor");
    const int64_t M = X.size(0), K = X.size(1);
    out_type(X.scalar_type(), "X");
    TORCH_CHECK_VALUE(M >= 1 && M <= kIntMax && K >= 16 && K % 16 == 0 && K <= 32768,
                      "X must be [M >= 1, K] with K a multiple of 16, at most 32768");
    return M;
  }
};

// X, codes, scale, stream -> (codes, scale)
PyObject* quantize_act(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity("w8a8_quantize_act", n, 4);
  Quantize q(a[0], a[1], a[2], a[3]);
  call("w8a8_quantize_act", [&] {
    return w8a8_quantize_act(q.M, q.K, q.x.at, q.x.ld, q.type, q.pc, static_cast<float*>(q.ps), q.place.stream);
  });
  return Py_BuildValue("NN", owned(a[1], q.codes), owned(a[2], q.scale));
  END_HANDLE_TH_ERRORS
}

// X, weight, residual, eps, codes, scale, residual_out, stream -> (codes, scale, residual_out)
PyObject* rmsnorm_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity("w8a8_rmsnorm_quantize", n, 8);
  Quantize q(a[0], a[4], a[5], a[7]);
  const ScalarType type = q.X.scalar_type();
  const void* weight = flat(a[1], {q.K}, ScalarType::BFloat16, q.place, "weight");
  Rows r, o;
  Tensor sum;
  if (a[2] != Py_None) {
    sum = a[6] == Py_None ? q.place.empty({q.M, q.K}, type) : tensor(a[6], "residual_out");
    r = Rows(tensor(a[2], "residual"), q.M, q.K, type, q.place, "residual");
    o = Rows(sum, q.M, q.K, type, q.place, "residual_out");
  } else {
    TORCH_CHECK_VALUE(a[6] == Py_None, "residual_out without a residual");
  }
  const float eps = static_cast<float>(number(a[3]));
  call("w8a8_rmsnorm_quantize", [&] {
    return w8a8_rmsnorm_quantize(q.M, q.K, q.x.at, q.x.ld, r.at, r.ld, weight, eps, o.at, o.ld, q.type, q.pc,
                                 static_cast<float*>(q.ps), q.place.stream);
  });
  return Py_BuildValue("NNN", owned(a[4], q.codes), owned(a[5], q.scale),
                       a[2] == Py_None ? Py_NewRef(Py_None) : owned(a[6], sum));
  END_HANDLE_TH_ERRORS
}

// a_codes, a_scale, w_codes, w_scale, bias, residual, activation, out_dtype, Y, stream -> Y; gated without residual
PyObject* linear(const char* name, bool gated, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(name, n, gated ? 9 : 10);
  PyObject *bias = a[4], *residual = gated ? Py_None : a[5];
  PyObject* const* rest = a + (gated ? 5 : 6);  // activation, out_dtype, Y, stream
  const Tensor &ac = tensor(a[0], "a_codes"), &wc = tensor(a[2], "w_codes");
  TORCH_CHECK_VALUE(ac.dim() == 2 && wc.dim() == 2, "a_codes and w_codes must be [M, K] and [N, K]");
  const int64_t M = ac.size(0), K = ac.size(1), rows = wc.size(0), N = gated ? rows / 2 : rows;
  TORCH_CHECK_VALUE(M >= 1 && M <= kIntMax && K >= 16 && K % 16 == 0 && K <= kIntMax && N >= 16 && N % 16 == 0 &&
                        rows <= kIntMax && (!gated || rows % 2 == 0) && wc.size(1) == K,
                    "a_codes [M, K] and w_codes must share K, at least one row, K and the output's width multiples of 16");
  const svdq_act act = activation(rest[0]);
  TORCH_CHECK_VALUE(THPDtype_Check(rest[1]), "out_dtype must be bfloat16 or float32");
  const ScalarType type = reinterpret_cast<THPDtype*>(rest[1])->scalar_type;
  const svdq_out out = out_type(type, "out_dtype");
  const Place place(ac, "a_codes", rest[3]);
  const Tensor Y = rest[2] == Py_None ? place.empty({M, N}, type) : tensor(rest[2], "Y");
  const Rows y(Y, M, N, type, place, "Y");
  const void* pa = flat(ac, {M, K}, ScalarType::Float8_e4m3fn, place, "a_codes");
  const void* pw = flat(wc, {rows, K}, ScalarType::Float8_e4m3fn, place, "w_codes");
  const auto* sa = static_cast<const float*>(flat(tensor(a[1], "a_scale"), {M}, ScalarType::Float, place, "a_scale"));
  const auto* sw = static_cast<const float*>(flat(tensor(a[3], "w_scale"), {rows}, ScalarType::Float, place, "w_scale"));
  const void* b = flat(bias, {rows}, ScalarType::BFloat16, place, "bias");
  Rows r;
  if (residual != Py_None) r = Rows(tensor(residual, "residual"), M, N, type, place, "residual");
  call(name, [&] {
    return gated ? w8a8_gated_linear(M, N, K, pa, sa, pw, sw, b, act, y.at, y.ld, out, place.stream)
                 : w8a8_linear(M, N, K, pa, sa, pw, sw, b, act, r.at, r.ld, y.at, y.ld, out, place.stream);
  });
  return owned(rest[2], Y);
  END_HANDLE_TH_ERRORS
}
PyObject* linear_plain(PyObject*, PyObject* const* a, Py_ssize_t n) { return linear("w8a8_linear", false, a, n); }
PyObject* linear_gated(PyObject*, PyObject* const* a, Py_ssize_t n) { return linear("w8a8_gated_linear", true, a, n); }

// what the rotation and its tables share: positions, freq, axis, scale
struct Angles {
  int64_t M, axes, P;
  Place place;
  const void* positions;
  int bytes;
  const double* freq;
  const int* axis;
  float scale;

  Angles(PyObject* op, PyObject* of, PyObject* oa, PyObject* os, PyObject* stream) : Angles(tensor(op, "positions"), tensor(of, "freq"), oa, os, stream) {}
  Angles(const Tensor& p, const Tensor& f, PyObject* oa, PyObject* os, PyObject* stream)
      : M(shape(p)), axes(p.dim() == 2 ? p.size(1) : 1), P(pairs(f)), place(p, "positions", stream) {
    positions = flat(p, p.sizes(), p.scalar_type(), place, "positions");
    bytes = p.scalar_type() == ScalarType::Long ? 8 : 4;
    freq = static_cast<const double*>(flat(f, {P}, ScalarType::Double, place, "freq"));
    axis = static_cast<const int*>(flat(oa, {P}, ScalarType::Int, place, "axis"));
    scale = static_cast<float>(number(os));
  }
  static int64_t shape(const Tensor& p) {
    TORCH_CHECK_VALUE((p.scalar_type() == ScalarType::Int || p.scalar_type() == ScalarType::Long) &&
                          (p.dim() == 1 || p.dim() == 2) && p.size(0) >= 1 && p.size(0) <= kIntMax &&
                          (p.dim() == 1 || (p.size(1) >= 1 && p.size(1) <= kIntMax)),
                      "positions must be int32 or int64, [M] or [M, axes]");
    return p.size(0);
  }
  static int64_t pairs(const Tensor& f) {
    TORCH_CHECK_VALUE(f.dim() == 1 && f.scalar_type() == ScalarType::Double && f.size(0) >= 1 && f.size(0) <= 512,
                      "freq must be float64 [pairs], at most 512");
    return f.size(0);
  }
};

// X, positions, freq, axis, scale, interleaved, Y, stream -> Y
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity("svdq_rope", n, 8);
  const Tensor& X = tensor(a[0], "X");
  TORCH_CHECK_VALUE(X.dim() == 3, "X must be bf16 or float32 [M, heads, D]");
  const svdq_out type = out_type(X.scalar_type(), "X");
  const Angles g(a[1], a[2], a[3], a[4], a[7]);
  const int64_t H = X.size(1), D = X.size(2);
  TORCH_CHECK_VALUE(X.size(0) == g.M, "positions must be [", X.size(0), "] or [", X.size(0), ", axes]");
  TORCH_CHECK_VALUE(H >= 1 && H <= kIntMax && D <= kIntMax && D % 2 == 0 && 2 * g.P <= D,
                    "D must be even and hold 2 * len(freq) columns");
  const Tensor Y = a[6] == Py_None ? g.place.empty(X.sizes(), X.scalar_type()) : tensor(a[6], "Y");
  const Heads x(X, X.sizes(), X.scalar_type(), g.place, "X"), y(Y, X.sizes(), X.scalar_type(), g.place, "Y");
  const bool interleaved = truth(a[5]);
  call("svdq_rope", [&] {
    return svdq_rope(g.M, H, D, g.P, g.axes, g.positions, g.bytes, g.freq, g.axis, g.scale, interleaved, type, x.at,
                     x.ld, x.ldh, y.at, y.ld, y.ldh, g.place.stream);
  });
  return owned(a[6], Y);
  END_HANDLE_TH_ERRORS
}

// positions, freq, axis, scale, angle_major, cos, sin, stream -> (cos, sin)
PyObject* rope_table(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity("svdq_rope_table", n, 8);
  const Angles g(a[0], a[1], a[2], a[3], a[7]);
  const bool angle_major = truth(a[4]);
  const int64_t first = angle_major ? g.P : g.M, second = angle_major ? g.M : g.P;
  const Tensor cos = a[5] == Py_None ? g.place.empty({first, second}, ScalarType::Float) : tensor(a[5], "cos");
  const Tensor sin = a[6] == Py_None ? g.place.empty({first, second}, ScalarType::Float) : tensor(a[6], "sin");
  auto* pc = static_cast<float*>(flat(cos, {first, second}, ScalarType::Float, g.place, "cos"));
  auto* ps = static_cast<float*>(flat(sin, {first, second}, ScalarType::Float, g.place, "sin"));
  call("svdq_rope_table", [&] {
    return svdq_rope_table(g.M, g.P, g.axes, g.positions, g.bytes, g.freq, g.axis, g.scale, angle_major, pc, ps,
                           g.place.stream);
  });
  return Py_BuildValue("NN", owned(a[5], cos), owned(a[6], sin));
  END_HANDLE_TH_ERRORS
}

#define METHOD(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD("w8a8_quantize_act", quantize_act),
                         METHOD("w8a8_rmsnorm_quantize", rmsnorm_quantize),
                         METHOD("w8a8_linear", linear_plain),
                         METHOD("w8a8_gated_linear", linear_gated),
                         METHOD("svdq_rope", rope),
                         METHOD("svdq_rope_table", rope_table),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// the interpreter and the torch that this was compiled for (build.py looks for the text, and gives it)
PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "built_for", SVDQ_BUILT_FOR) != 0) Py_CLEAR(m);
  return m;
}
