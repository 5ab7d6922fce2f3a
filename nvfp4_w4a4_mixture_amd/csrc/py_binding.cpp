// Argument marshalling of the MXFP4 and MXFP8 operators, the block norms and the combine
// for Python, compiled: checks of the tensors, allocation of missing outputs,
// the C-ABI call.
//
// A single-token call lasts 2 to 5 us on the device and its launch about 3 us
// on the host; the same checks and allocations written in Python took another
// 4 to 8 us a call.  Of one token, norm_in went from 7.6 to 3.4 us, norm_out
// from 11.4 to 4.5, and quantising and projecting 6144 to 6144 from 16.7 to 7.6.
//
// The functions take every argument by position; ops.py gives them their
// names, defaults and documentation.  The library's entry points are passed in
// by address (bind), so that both bindings call the same loaded library.
#include <ATen/EmptyTensor.h>
#include <ATen/hip/HIPContextLight.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <initializer_list>
#include <optional>
#include <string>

#include "../../include/moe_nvfp4.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Entry {
  decltype(&mxfp4_quantize) quantize;
  decltype(&mxfp4_dequantize) dequantize;
  decltype(&mxfp4_linear) linear;
  decltype(&mxfp4_ffn_workspace_bytes) ffn_ws;
  decltype(&mxfp4_grouped_ffn) ffn;
  decltype(&moe_norm_in) norm_in;
  decltype(&moe_norm_out) norm_out;
  decltype(&moe_combine) combine;
  decltype(&mxfp8_quantize) quantize8;
  decltype(&mxfp8_dequantize) dequantize8;
  decltype(&mxfp8_linear) linear8;
  decltype(&mxfp8_ffn_workspace_bytes) ffn8_ws;
  decltype(&mxfp8_grouped_ffn) ffn8;
  decltype(&moe_norm_in_mxfp8) norm_in8;
  decltype(&moe_norm_out_mxfp8) norm_out8;
  decltype(&mxfp8_moe_layer_workspace_bytes) layer_ws;
  decltype(&mxfp8_moe_layer) layer;
} g_entry;
PyObject* g_check = nullptr;  // check(status, name): raises for a status other than MOE_OK

[[noreturn]] __attribute__((format(printf, 2, 3))) void raise(PyObject* type, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  PyErr_SetString(type, buf);
  throw python_error();
}

void check(moe_status st, const char* fn) {
  if (st == MOE_OK) return;
  PyObject* r = PyObject_CallFunction(g_check, "is", (int)st, fn);
  Py_XDECREF(r);
  throw python_error();
}

std::string type_name(ScalarType t) {
  switch (t) {
    case ScalarType::BFloat16: return "torch.bfloat16";
    case ScalarType::Float: return "torch.float32";
    case ScalarType::Half: return "torch.float16";
    case ScalarType::Byte: return "torch.uint8";
    case ScalarType::Int: return "torch.int32";
    default: return std::string("torch.") + at::toString(t);
  }
}

std::string shape_name(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

bool given(PyObject* o) { return o != Py_None; }

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a torch.Tensor", name);
  return THPVariable_Unpack(o);
}

// The device of this call's tensors: that of the first one checked (-1: none yet)
thread_local c10::DeviceIndex t_device = -1;

void on_device(const Tensor& t, const char* name) {
  if (!t.is_cuda()) raise(PyExc_ValueError, "%s must be on a GPU device", name);
  const c10::DeviceIndex d = t.get_device();
  if (t_device < 0) t_device = d;
  if (d != t_device)
    raise(PyExc_ValueError, "%s must be on cuda:%d with the other tensors, got cuda:%d", name, (int)t_device, (int)d);
}

const Tensor& typed(PyObject* o, const char* name, ScalarType type) {
  const Tensor& t = tensor(o, name);
  if (t.scalar_type() != type)
    raise(PyExc_TypeError, "%s must be %s, got %s", name, type_name(type).c_str(), type_name(t.scalar_type()).c_str());
  on_device(t, name);
  return t;
}

// A contiguous GPU tensor of this type and shape.
const Tensor& need(PyObject* o, const char* name, ScalarType type, at::IntArrayRef shape) {
  const Tensor& t = typed(o, name, type);
  if (t.sizes() != shape)
    raise(PyExc_ValueError, "%s must have shape %s, got %s", name, shape_name(shape).c_str(), shape_name(t.sizes()).c_str());
  if (!t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
  return t;
}

// A GPU matrix with unit column stride and any row stride, BF16 (or FP32, if `f32`).
struct Rows {
  const Tensor& t;
  int64_t rows, cols, ld;
};
Rows matrix(PyObject* o, const char* name, bool f32 = false) {
  const Tensor& t = tensor(o, name);
  if (t.scalar_type() != ScalarType::BFloat16 && !(f32 && t.scalar_type() == ScalarType::Float))
    raise(PyExc_TypeError, "%s must be a tensor of torch.bfloat16%s, got %s", name, f32 ? " or torch.float32" : "",
                           type_name(t.scalar_type()).c_str());
  on_device(t, name);
  if (t.dim() != 2 || (t.size(1) > 1 && t.size(0) > 0 && t.stride(1) != 1))
    raise(PyExc_ValueError, "%s must be [rows, cols] with unit column stride", name);
  const int64_t rows = t.size(0), cols = t.size(1);
  return {t, rows, cols, rows > 1 ? t.stride(0) : (cols > 1 ? cols : 1)};
}

// An uninitialized tensor on the call's device, the current one (see OnStream), straight
// from its allocator: without the dispatcher an output costs 0.3 us, not 0.6.
Tensor fresh(ScalarType type, at::IntArrayRef shape) {
  return at::detail::empty_generic(shape, at::cuda::getCUDADeviceAllocator(), c10::DispatchKeySet(c10::DispatchKey::CUDA),
                                   type, std::nullopt);
}

// An output matrix and its row stride: a given one checked, a missing one allocated.
struct Out {
  Tensor t;
  int64_t ld;
};
Out output(PyObject* o, const char* name, ScalarType type, int64_t rows, int64_t cols) {
  if (!given(o)) return {fresh(type, {rows, cols}), cols};
  const Rows m = matrix(o, name, true);
  if (m.t.scalar_type() != type)
    raise(PyExc_TypeError, "%s must be %s, got %s", name, type_name(type).c_str(), type_name(m.t.scalar_type()).c_str());
  if (m.rows != rows || m.cols != cols)
    raise(PyExc_ValueError, "%s must have shape %s, got %s", name, shape_name({rows, cols}).c_str(),
                            shape_name(m.t.sizes()).c_str());
  return {m.t, m.ld};
}

Tensor buffer(PyObject* o, const char* name, ScalarType type, at::IntArrayRef shape) {
  return given(o) ? need(o, name, type, shape) : fresh(type, shape);
}

// A workspace of at least one byte; the library checks a given one's size.
Tensor workspace(PyObject* o, size_t bytes) {
  if (!given(o)) return fresh(ScalarType::Byte, {(int64_t)(bytes ? bytes : 1)});
  const Tensor& t = typed(o, "workspace", ScalarType::Byte);
  if (!t.is_contiguous()) raise(PyExc_ValueError, "workspace must be contiguous");
  return t;
}

template <typename T>
T* ptr(const Tensor& t) {
  return t.defined() ? static_cast<T*>(t.data_ptr()) : nullptr;
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}
void* address(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p && PyErr_Occurred()) throw python_error();
  return p;
}

// The device of the call's tensors made the current one, if it is not.
class OnDevice {
 public:
  explicit OnDevice(c10::DeviceIndex d) : before_(c10::hip::current_device()), other_(before_ != d) {
    if (other_) c10::hip::set_device(d);
  }
  OnDevice(const OnDevice&) = delete;
  ~OnDevice() {
    if (other_) c10::hip::set_device(before_);
  }

 private:
  c10::DeviceIndex before_;
  bool other_;
};

// The stream that a call is enqueued on: a given torch stream, or the current
// one of the tensors' device, which is the current device while this object lives (a
// kernel launched on another one would reach for memory that may not be mapped
// there).  A given stream is the current one of the tensors' device while this
// object lives, so that missing outputs and workspaces come from its pool: the
// allocator hands a block on in the order of its own stream's work, and a
// workspace is dropped here while the kernels that use it are still queued.
// Constructed after the tensors are checked: without a GPU it raises.
class OnStream {
 public:
  OnStream(PyObject* o, const Tensor& like) : device_(like.get_device()) {
    if (!given(o)) return;
    PyObject* r = PyObject_GetAttrString(o, "cuda_stream");
    if (!r) throw python_error();
    hipStream_t s = static_cast<hipStream_t>(PyLong_AsVoidPtr(r));
    Py_DECREF(r);
    if (!s && PyErr_Occurred()) throw python_error();
    given_ = s;
    before_ = c10::hip::getCurrentHIPStream(like.get_device());
    c10::hip::setCurrentHIPStream(c10::hip::getStreamFromExternal(s, like.get_device()));
  }
  OnStream(const OnStream&) = delete;
  ~OnStream() {
    if (before_) c10::hip::setCurrentHIPStream(*before_);
  }
  void* get() const { return before_ ? given_ : c10::hip::getCurrentHIPStream().stream(); }

 private:
  OnDevice device_;
  hipStream_t given_ = nullptr;
  std::optional<c10::hip::HIPStream> before_;
};

int64_t padded(int64_t cols) { return (cols + 255) / 256 * 256; }

// The codes and scales of [rows, cols] in the padded row form.
struct Codes {
  Tensor codes, scales;
};
// `bits` of an element: 4 (MXFP4) or 8 (MXFP8).
Codes mx_output(PyObject* codes, PyObject* scales, int64_t rows, int64_t cols, int bits) {
  const int64_t c = padded(cols);
  return {buffer(codes, "codes", ScalarType::Byte, {rows, c * bits / 8}),
          buffer(scales, "scales", ScalarType::Byte, {rows, c / 32})};
}
// Given ones of `cols` columns; returns the rows.
int64_t mx_input(PyObject* codes, PyObject* scales, int64_t cols, int bits) {
  const int64_t c = padded(cols);
  const Tensor& t = tensor(codes, "x_codes");
  const int64_t rows = t.dim() == 2 ? t.size(0) : 0;
  need(codes, "x_codes", ScalarType::Byte, {rows, c * bits / 8});
  need(scales, "x_scales", ScalarType::Byte, {rows, c / 32});
  return rows;
}

ScalarType float_type(int64_t code) { return code ? ScalarType::Float : ScalarType::BFloat16; }

PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}

PyObject* tuple_of(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New((Py_ssize_t)ts.size());
  if (!r) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) PyTuple_SET_ITEM(r, i++, wrap(t));
  return r;
}

// Every function: METH_FASTCALL with exactly N arguments, C++ and torch exceptions turned into Python's.
template <int N, PyObject* (*F)(PyObject* const*)>
PyObject* call(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != N) raise(PyExc_TypeError, "expected %d arguments, got %d", N, (int)n);
  t_device = -1;
  return F(a);
  END_HANDLE_TH_ERRORS
}

// x, codes, scales, stream
template <int BITS>
PyObject* quantize(PyObject* const* a) {
  const Rows x = matrix(a[0], "x", true);
  const OnStream st(a[3], x.t);
  const Codes q = mx_output(a[1], a[2], x.rows, x.cols, BITS);
  check((BITS == 4 ? g_entry.quantize : g_entry.quantize8)(x.t.data_ptr(), x.t.scalar_type() == ScalarType::Float, x.rows, x.cols, x.ld,
                         ptr<uint8_t>(q.codes), ptr<uint8_t>(q.scales), st.get()),
        BITS == 4 ? "mxfp4_quantize" : "mxfp8_quantize");
  return tuple_of({q.codes, q.scales});
}

// codes, scales, cols, dtype code, out, stream
template <int BITS>
PyObject* dequantize(PyObject* const* a) {
  const int64_t cols = integer(a[2]), rows = mx_input(a[0], a[1], cols, BITS), type = integer(a[3]);
  const OnStream st(a[5], tensor(a[0], "x_codes"));
  const Out y = output(a[4], "out", float_type(type), rows, cols);
  check((BITS == 4 ? g_entry.dequantize : g_entry.dequantize8)(ptr<uint8_t>(tensor(a[0], "")), ptr<uint8_t>(tensor(a[1], "")), rows, cols, (int32_t)type,
                           y.t.data_ptr(), y.ld, st.get()),
        BITS == 4 ? "mxfp4_dequantize" : "mxfp8_dequantize");
  return wrap(y.t);
}

// x_codes, x_scales, w_codes, w_scales, N, dtype code, y, workspace, stream
PyObject* linear(PyObject* const* a) {
  const Tensor& wc = tensor(a[2], "w_codes");
  if (wc.dim() != 5) raise(PyExc_ValueError, "w_codes must be [G, KK, 4, 64, 16]");
  const int64_t N = integer(a[4]), type = integer(a[5]), KK = wc.size(1), K = 256 * KK, G = (N + 31) / 32;
  const int64_t T = mx_input(a[0], a[1], K, 4);  // K is the padded width: the padding is zero on both sides
  need(a[2], "w_codes", ScalarType::Byte, {G, KK, 4, 64, 16});
  const Tensor& ws = need(a[3], "w_scales", ScalarType::Byte, {G, KK, 64, 4});
  const Tensor &xc = tensor(a[0], ""), &xs = tensor(a[1], "");
  const OnStream st(a[8], xc);
  const Out y = output(a[6], "y", float_type(type), T, N);
  if (given(a[7])) workspace(a[7], 0);  // of the right kind; the product uses none
  check(g_entry.linear(ptr<uint8_t>(xc), ptr<uint8_t>(xs), T, K, ptr<uint8_t>(wc), ptr<uint8_t>(ws), N, (int32_t)type,
                       y.t.data_ptr(), y.ld, nullptr, 0, st.get()),
        "mxfp4_linear");
  return wrap(y.t);
}

// x_codes, x_scales, w_codes, w_scales, N, dtype code, bias, activation code, residual, y, stream
PyObject* linear8(PyObject* const* a) {
  const Tensor& wc = tensor(a[2], "w_codes");
  if (wc.dim() != 5) raise(PyExc_ValueError, "w_codes must be [G, KK, 4, 64, 16]");
  const int64_t N = integer(a[4]), type = integer(a[5]), KK = wc.size(1), K = 256 * KK, G = (N + 31) / 32;
  const int64_t T = mx_input(a[0], a[1], K, 8);
  need(a[2], "w_codes", ScalarType::Byte, {G, KK, 4, 64, 16});
  const Tensor& ws = need(a[3], "w_scales", ScalarType::Byte, {G, KK, 64, 4});
  const Tensor &xc = tensor(a[0], ""), &xs = tensor(a[1], "");
  const Tensor bias = given(a[6]) ? need(a[6], "bias", ScalarType::BFloat16, {N}) : Tensor();
  Tensor r;
  int64_t ldr = N, rtype = 0;
  if (given(a[8])) {
    const Rows m = matrix(a[8], "residual", true);
    if (m.rows != T || m.cols != N)
      raise(PyExc_ValueError, "residual must have shape %s, got %s", shape_name({T, N}).c_str(),
                              shape_name(m.t.sizes()).c_str());
    r = m.t;
    ldr = m.ld;
    rtype = m.t.scalar_type() == ScalarType::Float;
  }
  const OnStream st(a[10], xc);
  const Out y = output(a[9], "y", float_type(type), T, N);
  check(g_entry.linear8(ptr<uint8_t>(xc), ptr<uint8_t>(xs), T, K, ptr<uint8_t>(wc), ptr<uint8_t>(ws), N,
                        ptr<uint16_t>(bias), (int32_t)integer(a[7]), r.defined() ? r.data_ptr() : nullptr,
                        (int32_t)rtype, ldr, (int32_t)type, y.t.data_ptr(), y.ld, st.get()),
        "mxfp8_linear");
  return wrap(y.t);
}

// x_codes, x_scales, w13_codes, w13_scales, w2_codes, w2_scales, w2_max_scale, H, I, k, expert_offsets,
// sorted_pair_ids, topk_w, pair_out, pair_scale, workspace, stream
template <int BITS>
PyObject* grouped_ffn(PyObject* const* a) {
  const int64_t H = integer(a[7]), I = integer(a[8]), k = integer(a[9]);
  const int64_t T = mx_input(a[0], a[1], H, BITS), E = tensor(a[2], "w13_codes").dim() ? tensor(a[2], "").size(0) : 0;
  const Tensor &xc = tensor(a[0], ""), &xs = tensor(a[1], "");
  const int64_t G13 = (2 * I + 31) / 32, K13 = padded(H) / 256, G2 = (H + 31) / 32, K2 = padded(I) / 256;
  const Tensor& c13 = need(a[2], "w13_codes", ScalarType::Byte, {E, G13, K13, 4, 64, 16});
  const Tensor& s13 = need(a[3], "w13_scales", ScalarType::Byte, {E, G13, K13, 64, 4});
  const Tensor& c2 = need(a[4], "w2_codes", ScalarType::Byte, {E, G2, K2, 4, 64, 16});
  const Tensor& s2 = need(a[5], "w2_scales", ScalarType::Byte, {E, G2, K2, 64, 4});
  const Tensor& m2 = need(a[6], "w2_max_scale", ScalarType::Int, {E});
  const Tensor& off = need(a[10], "expert_offsets", ScalarType::Int, {E + 1});
  const Tensor& srt = need(a[11], "sorted_pair_ids", ScalarType::Int, {T * k});
  const Tensor& tw = need(a[12], "topk_w", ScalarType::Float, {T, k});
  const OnStream st(a[16], xc);
  const Tensor po = buffer(a[13], "pair_out", ScalarType::Half, {T * k, H});
  const Tensor ps = buffer(a[14], "pair_scale", ScalarType::Float, {T * k});
  const Tensor ws = workspace(a[15], (BITS == 4 ? g_entry.ffn_ws : g_entry.ffn8_ws)(T, k, E, H, I));
  check((BITS == 4 ? g_entry.ffn : g_entry.ffn8)(ptr<uint8_t>(xc), ptr<uint8_t>(xs), T, H, ptr<uint8_t>(c13), ptr<uint8_t>(s13), ptr<uint8_t>(c2),
                    ptr<uint8_t>(s2), ptr<int32_t>(m2), E, I, k, ptr<int32_t>(off), ptr<int32_t>(srt), ptr<float>(tw),
                    ptr<uint16_t>(po), ptr<float>(ps), ptr<void>(ws), (size_t)ws.numel(), st.get()),
        BITS == 4 ? "mxfp4_grouped_ffn" : "mxfp8_grouped_ffn");
  return tuple_of({po, ps});
}

// x, w_router, bias, k, rsf, w13_codes, w13_scales, w2_codes, w2_scales, dtype code, y, topk_ids, topk_w, workspace,
// stream
PyObject* layer(PyObject* const* a) {
  const Rows x = matrix(a[0], "x_bf16");
  const int64_t T = x.rows, H = x.cols, k = integer(a[3]), type = integer(a[9]);
  const int64_t E = tensor(a[1], "w_router_bf16").dim() ? tensor(a[1], "").size(0) : 0;
  const Tensor& wr = need(a[1], "w_router_bf16", ScalarType::BFloat16, {E, H});
  const Tensor& bias = need(a[2], "bias", ScalarType::Float, {E});
  const Tensor& w13 = tensor(a[5], "w13_codes");
  const int64_t G13 = w13.dim() == 6 ? w13.size(1) : 0, I = 16 * G13;  // gate and up rows in groups of 32
  const int64_t K13 = padded(H) / 256, G2 = (H + 31) / 32, K2 = padded(I) / 256;
  const Tensor& c13 = need(a[5], "w13_codes", ScalarType::Byte, {E, G13, K13, 4, 64, 16});
  const Tensor& s13 = need(a[6], "w13_scales", ScalarType::Byte, {E, G13, K13, 64, 4});
  const Tensor& c2 = need(a[7], "w2_codes", ScalarType::Byte, {E, G2, K2, 4, 64, 16});
  const Tensor& s2 = need(a[8], "w2_scales", ScalarType::Byte, {E, G2, K2, 64, 4});
  if (k < 1 || k > E) raise(PyExc_ValueError, "need 1 <= k <= E, got k = %lld, E = %lld", (long long)k, (long long)E);
  const OnStream st(a[14], x.t);
  const Tensor y = buffer(a[10], "y", float_type(type), {T, H});
  const Tensor ids = buffer(a[11], "topk_ids", ScalarType::Int, {T, k});
  const Tensor tw = buffer(a[12], "topk_w", ScalarType::Float, {T, k});
  const Tensor ws = workspace(a[13], g_entry.layer_ws(T, H, E, k, I));
  check(g_entry.layer(ptr<uint16_t>(x.t), T, H, x.ld, ptr<uint16_t>(wr), ptr<float>(bias), E, k, (float)real(a[4]),
                      ptr<uint8_t>(c13), ptr<uint8_t>(s13), ptr<uint8_t>(c2), ptr<uint8_t>(s2), I, (int32_t)type,
                      y.data_ptr(), ptr<int32_t>(ids), ptr<float>(tw), ptr<void>(ws), (size_t)ws.numel(), st.get()),
        "mxfp8_moe_layer");
  return tuple_of({y, ids, tw});
}

// n of [T, H] (False: none) and, if asked for, its codes and scales
struct Normed {
  Out n;
  Codes q;
};
Normed norm_output(PyObject* n, bool quantize, PyObject* codes, PyObject* scales, int64_t T, int64_t H,
                   int bits) {
  Normed r{{Tensor(), H}, {}};
  if (n != Py_False) r.n = output(n, "n", ScalarType::BFloat16, T, H);
  if (quantize || given(codes) || given(scales)) r.q = mx_output(codes, scales, T, H, bits);
  return r;
}

// x, w, eps, n, quantize, codes, scales, stream (quantize: of the MXFP8 form always true)
template <int BITS>
PyObject* norm_in(PyObject* const* a) {
  const Rows x = matrix(a[0], "x");
  const Tensor& w = need(a[1], "w", ScalarType::BFloat16, {x.cols});
  const OnStream st(a[7], x.t);
  const Normed r = norm_output(a[3], truth(a[4]), a[5], a[6], x.rows, x.cols, BITS);
  check((BITS == 4 ? g_entry.norm_in : g_entry.norm_in8)(ptr<uint16_t>(x.t), x.rows, x.cols, x.ld, ptr<uint16_t>(w), (float)real(a[2]), ptr<uint16_t>(r.n.t),
                        r.n.ld, ptr<uint8_t>(r.q.codes), ptr<uint8_t>(r.q.scales), st.get()),
        BITS == 4 ? "moe_norm_in" : "moe_norm_in_mxfp8");
  return r.q.codes.defined() ? tuple_of({r.n.t, r.q.codes, r.q.scales}) : wrap(r.n.t);
}

// y, residual, w_post, w_next, gate, residual_scale, eps, out, n, quantize, codes, scales, stream
template <int BITS>
PyObject* norm_out(PyObject* const* a) {
  const Rows y = matrix(a[0], "y", true), r = matrix(a[1], "residual");
  const int64_t T = y.rows, H = y.cols;
  if (r.rows != T || r.cols != H)
    raise(PyExc_ValueError, "residual must have shape %s, got %s", shape_name({T, H}).c_str(),
                            shape_name(r.t.sizes()).c_str());
  const Tensor wp = given(a[2]) ? need(a[2], "w_post", ScalarType::BFloat16, {H}) : Tensor();
  const Tensor wn = given(a[3]) ? need(a[3], "w_next", ScalarType::BFloat16, {H}) : Tensor();
  Tensor g;
  int64_t grs = 0, gcs = 0;
  if (given(a[4])) {
    g = typed(a[4], "gate", ScalarType::BFloat16);
    if (g.dim() != 2 || (g.size(0) != 1 && g.size(0) != T) || (g.size(1) != 1 && g.size(1) != H))
      raise(PyExc_ValueError, "gate must be [T, 1], [1, H] or [T, H], got %s", shape_name(g.sizes()).c_str());
    grs = g.size(0) == 1 ? 0 : g.stride(0);
    gcs = g.size(1) == 1 ? 0 : g.stride(1);
  }
  const OnStream st(a[12], y.t);
  const Out ro = output(a[7], "out", ScalarType::BFloat16, T, H);
  Normed q{{Tensor(), H}, {}};
  if (wn.defined())
    q = norm_output(a[8], truth(a[9]), a[10], a[11], T, H, BITS);
  else if (given(a[8]) || truth(a[9]) || given(a[10]) || given(a[11]))
    raise(PyExc_ValueError, "n and its quantization need w_next");
  check((BITS == 4 ? g_entry.norm_out : g_entry.norm_out8)(y.t.data_ptr(), y.t.scalar_type() == ScalarType::Float, T, H, y.ld, ptr<uint16_t>(r.t), r.ld,
                         ptr<uint16_t>(wp), ptr<uint16_t>(g), grs, gcs, (float)real(a[5]), ptr<uint16_t>(wn),
                         (float)real(a[6]), ptr<uint16_t>(ro.t), ro.ld, ptr<uint16_t>(q.n.t), q.n.ld,
                         ptr<uint8_t>(q.q.codes), ptr<uint8_t>(q.q.scales), st.get()),
        BITS == 4 ? "moe_norm_out" : "moe_norm_out_mxfp8");
  if (!wn.defined()) return wrap(ro.t);
  if (!q.q.codes.defined()) return tuple_of({ro.t, q.n.t});
  return tuple_of({ro.t, q.n.t, q.q.codes, q.q.scales});
}

// pair_out, pair_scale, T, k, dtype code, y, stream
PyObject* combine(PyObject* const* a) {
  const Tensor &po = typed(a[0], "pair_out", ScalarType::Half), &ps = typed(a[1], "pair_scale", ScalarType::Float);
  const int64_t T = integer(a[2]), k = integer(a[3]), type = integer(a[4]);
  const __int128 pairs = (__int128)T * k;  // of the caller's numbers: in 64 bits they may wrap
  if (po.dim() != 2 || po.size(0) < pairs)
    raise(PyExc_ValueError, "pair_out must be [>= T*k, H], got %s", shape_name(po.sizes()).c_str());
  if (ps.numel() < pairs)
    raise(PyExc_ValueError, "pair_scale must hold T*k = %lld scales, got %lld", (long long)pairs, (long long)ps.numel());
  if (!po.is_contiguous() || !ps.is_contiguous()) raise(PyExc_ValueError, "pair_out and pair_scale must be contiguous");
  const OnStream st(a[6], po);
  Tensor y;
  if (given(a[5])) {  // any shape: the result is the first T * H elements
    y = typed(a[5], "y", float_type(type));
    if (!y.is_contiguous()) raise(PyExc_ValueError, "y must be contiguous");
    if (y.numel() < (__int128)T * po.size(1))
      raise(PyExc_ValueError, "y must hold T*H = %lld * %lld elements, got %lld", (long long)T, (long long)po.size(1),
            (long long)y.numel());
  } else {
    y = fresh(float_type(type), {T, po.size(1)});
  }
  check(g_entry.combine(ptr<uint16_t>(po), ptr<float>(ps), T, k, po.size(1), (int32_t)type, y.data_ptr(), st.get()),
        "moe_combine");
  return wrap(y);
}

// check, then the addresses in Entry's order
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 1 + (Py_ssize_t)(sizeof(Entry) / sizeof(void*))) raise(PyExc_TypeError, "bind: wrong number of entry points");
  void** to = reinterpret_cast<void**>(&g_entry);
  for (Py_ssize_t i = 1; i < n; ++i) to[i - 1] = address(a[i]);
  Py_INCREF(a[0]);
  Py_XDECREF(g_check);
  g_check = a[0];
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

template <int N, PyObject* (*F)(PyObject* const*)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<N, F>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&bind)), METH_FASTCALL, nullptr},
    method<4, quantize<4>>("mxfp4_quantize"),
    method<6, dequantize<4>>("mxfp4_dequantize"),
    method<9, linear>("mxfp4_linear"),
    method<17, grouped_ffn<4>>("mxfp4_grouped_ffn"),
    method<8, norm_in<4>>("moe_norm_in"),
    method<13, norm_out<4>>("moe_norm_out"),
    method<7, combine>("moe_combine"),
    method<4, quantize<8>>("mxfp8_quantize"),
    method<6, dequantize<8>>("mxfp8_dequantize"),
    method<11, linear8>("mxfp8_linear"),
    method<17, grouped_ffn<8>>("mxfp8_grouped_ffn"),
    method<8, norm_in<8>>("moe_norm_in_mxfp8"),
    method<13, norm_out<8>>("moe_norm_out_mxfp8"),
    method<15, layer>("mxfp8_moe_layer"),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&g_module); }
