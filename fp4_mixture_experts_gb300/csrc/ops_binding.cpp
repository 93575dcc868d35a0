// The operators' Python binding: argument checks, results and workspaces, and
// the call of the C entry points (include/moe_fp4.h), in one native call each.
//
// A single-token operator runs for a few microseconds; marshalling its
// arguments in Python takes longer than that on the host (one-token block end:
// 13 us a call through ctypes, 3.7 us so).  The module holds no state but
// the entry points' addresses and the exception to raise, both set by bind().
#include <Python.h>

#include <ATen/EmptyTensor.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string.h>

#include <optional>
#include <stdexcept>
#include <string>

#include "../../include/moe_fp4.h"

namespace {

struct Entry {
  decltype(&moe_fp4_mxfp4_quantize) quantize;
  decltype(&moe_fp4_mxfp4_dequantize) dequantize;
  decltype(&moe_fp4_mxfp4_tile_scales) tile_scales;
  decltype(&moe_fp4_mxfp4_matmul) matmul;
  decltype(&moe_fp4_mxfp4_linear) linear;
  decltype(&moe_fp4_mxfp4_linear_workspace_bytes) linear_workspace_bytes;
  decltype(&moe_fp4_mxfp4_gathered_workspace_bytes) gathered_workspace_bytes;
  decltype(&moe_fp4_block_norm) block_norm;
} g_entry;
PyObject* g_raise = nullptr;  // called with (status, entry point); raises

struct BadArgument : std::runtime_error {
  using std::runtime_error::runtime_error;
};

[[noreturn]] void bad(const std::string& what) { throw BadArgument(what); }

bool none(PyObject* o) { return o == nullptr || o == Py_None; }

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) bad(std::string(what) + " must be a tensor");
  return THPVariable_Unpack(o);
}

at::ScalarType dtype_of(PyObject* o) {
  if (!THPDtype_Check(o)) bad("dtype must be a torch.dtype");
  const at::ScalarType t = reinterpret_cast<THPDtype*>(o)->scalar_type;
  if (t != at::kBFloat16 && t != at::kFloat) bad("dtype must be bf16 or fp32");
  return t;
}

int type_of(const at::Tensor& t, const char* what) {
  if (t.scalar_type() == at::kBFloat16) return MOE_FP4_TYPE_BF16;
  if (t.scalar_type() == at::kFloat) return MOE_FP4_TYPE_F32;
  bad(std::string(what) + " must be bf16 or fp32");
}

int64_t whole(PyObject* o, const char* what) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    bad(std::string(what) + " must be an integer");
  }
  return v;
}

double real(PyObject* o, const char* what) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    bad(std::string(what) + " must be a number");
  }
  return v;
}

bool truth(PyObject* o, const char* what) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    bad(std::string(what) + " must be true or false");
  }
  return v == 1;
}

// rows: 2-D on the GPU, contiguous along a row; rows may be strided
struct Rows {
  int64_t rows, width, stride;
  int type;
  void* p;
};

Rows rows_of(const at::Tensor& t, const char* what) {
  if (!t.is_cuda() || t.dim() != 2) bad(std::string(what) + " must be a 2-D GPU tensor");
  const int64_t R = t.size(0), K = t.size(1);
  if ((t.stride(1) != 1 && K > 1) || (t.stride(0) < K && R > 1))
    bad(std::string(what) + " must have contiguous, separate rows");
  return {R, K, R > 1 ? t.stride(0) : K, type_of(t, what), t.data_ptr()};
}

uint8_t* bytes_of(const at::Tensor& t, const char* what, int64_t numel) {
  if (t.scalar_type() != at::kByte || !t.is_cuda() || !t.is_contiguous() || t.numel() < numel)
    bad(std::string(what) + " must be a contiguous uint8 GPU tensor of at least " + std::to_string(numel) + " elements");
  return static_cast<uint8_t*>(t.data_ptr());
}

const int32_t* indices(PyObject* o, const char* what, int64_t* numel) {
  if (none(o)) return nullptr;
  const at::Tensor& t = tensor(o, what);
  if (t.scalar_type() != at::kInt || !t.is_cuda() || t.dim() != 1 || !t.is_contiguous())
    bad(std::string(what) + " must be a contiguous 1-D int32 GPU tensor");
  *numel = t.numel();
  return static_cast<const int32_t*>(t.data_ptr());
}

// A new tensor on the current device, straight from PyTorch's allocator (without
// the dispatcher: 1.4 -> 1.0 us each).
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType t) {
  return at::detail::empty_generic(shape, c10::GetAllocator(c10::kCUDA), c10::DispatchKeySet(c10::DispatchKey::CUDA), t,
                                   std::nullopt);
}

at::Tensor result(PyObject* out, int64_t rows, int64_t width, at::ScalarType t, const char* what) {
  if (none(out)) return fresh({rows, width}, t);
  const at::Tensor& o = tensor(out, what);
  if (!o.is_cuda() || o.scalar_type() != t || !o.is_contiguous() || o.dim() != 2 || o.size(0) != rows ||
      o.size(1) != width)
    bad(std::string(what) + " must be a contiguous GPU tensor [" + std::to_string(rows) + ", " + std::to_string(width) +
        "] of the result's type");
  return o;
}

// The GPU that all tensors among a call's arguments are on.
c10::DeviceIndex gpu_of(PyObject* const* a, Py_ssize_t n) {
  c10::DeviceIndex gpu = -1;
  for (Py_ssize_t i = 0; i < n; ++i) {
    PyObject* const o = a[i];  // (the check for a tensor takes ~0.1 us on anything else)
    if (none(o) || PyBool_Check(o) || PyFloat_Check(o) || PyLong_Check(o) || THPDtype_Check(o)) continue;
    if (!THPVariable_Check(o)) continue;
    const c10::Device d = THPVariable_Unpack(o).device();
    if (!d.is_cuda()) bad("GPU tensors are needed");
    if (gpu >= 0 && d.index() != gpu) bad("all tensors must be on the same GPU");
    gpu = d.index();
  }
  if (gpu < 0) bad("GPU tensors are needed");
  return gpu;
}

// Where a call runs: on the GPU of its tensors, which is the current device
// meanwhile (results are allocated, sizes looked up and kernels launched there),
// and on that GPU's current stream or the one given, which is then the current
// one while results and workspaces are allocated, so that their memory is reused
// in that stream's order (a workspace is given back before its kernel has run).
struct Stream {
  std::optional<c10::cuda::CUDAGuard> device;
  std::optional<c10::cuda::CUDAStreamGuard> guard;
  void* handle;
  Stream(PyObject* s, c10::DeviceIndex gpu) {
    if (gpu != c10::cuda::current_device()) device.emplace(gpu);
    if (none(s)) {
      handle = c10::cuda::getCurrentCUDAStream(gpu).stream();
      return;
    }
    handle = reinterpret_cast<void*>(whole(s, "stream"));
    guard.emplace(c10::cuda::getStreamFromExternal(static_cast<cudaStream_t>(handle), gpu));
  }
};

// nullptr with the exception set, for a nonzero status
bool ok(int status, const char* entry) {
  if (status == 0) return true;
  PyObject* r = PyObject_CallFunction(g_raise, "is", status, entry);
  Py_XDECREF(r);
  if (r != nullptr) PyErr_SetString(PyExc_RuntimeError, entry);
  return false;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Weights {
  moe_fp4_mm_dims dims;
  uint8_t *w, *scales;
  int64_t n_out, a_scale_bytes;
};

Weights weights_of(int64_t M, int64_t K, PyObject* w_, PyObject* scales_, bool grouped, int64_t n_offsets, bool swiglu,
                   at::ScalarType t) {
  const at::Tensor& w = tensor(w_, "w");
  if ((w.dim() != 2 && w.dim() != 3) || w.size(-1) * 2 != K)
    bad("w must be uint8 [E, N, K/2] or [N, K/2] with K = " + std::to_string(K));
  const int64_t E = w.dim() == 3 ? w.size(0) : 1, N = w.size(-2);
  if (grouped ? n_offsets != E + 1 : E != 1) bad("several matrices need offsets, of E + 1 elements");
  if (swiglu && N % 2) bad("swiglu needs an even number of features");
  if (M > INT32_MAX || N > INT32_MAX || E > INT32_MAX || K > INT32_MAX) bad("sizes beyond 2^31");
  const int64_t kt = ceil_div(K, 128);
  return {{(int32_t)M, (int32_t)N, (int32_t)K, (int32_t)E, swiglu, t == at::kFloat ? MOE_FP4_TYPE_F32 : MOE_FP4_TYPE_BF16},
          bytes_of(w, "w", 0),
          bytes_of(tensor(scales_, "w_scale"), "w_scale (tiled, by mxfp4_tile_scales)", E * ceil_div(N, 128) * kt * 512),
          swiglu ? N / 2 : N, (M / 128 + E) * kt * 512};
}

#define NATIVE_BEGIN(name, n)                                       \
  PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t nargs) { \
    HANDLE_TH_ERRORS                                                \
    if (nargs != (n)) {                                             \
      PyErr_SetString(PyExc_TypeError, #name ": argument count");   \
      return nullptr;                                               \
    }                                                               \
    try {
#define NATIVE_END                                 \
    } catch (const BadArgument& e) {               \
      PyErr_SetString(PyExc_ValueError, e.what()); \
      return nullptr;                              \
    }                                              \
    END_HANDLE_TH_ERRORS                           \
  }

// x, row_index, index_div, offsets, tiled, codes, scales, stream
NATIVE_BEGIN(quantize, 8)
  const at::Tensor& x = tensor(a[0], "x");
  const Stream st(a[7], gpu_of(a, nargs));
  const Rows r = rows_of(x, "x");
  if (r.width % 32 || r.width == 0) bad("K must be a multiple of 32");
  const bool tiled = truth(a[4], "tiled");
  int64_t S = r.rows, n_off = 2;
  const int32_t* index = indices(a[1], "row_index", &S);
  const int32_t* off = indices(a[3], "offsets", &n_off);
  if (off != nullptr && (!tiled || n_off < 2)) bad("offsets need tiled scales, and E + 1 elements");
  const int64_t E = n_off - 1, K = r.width, kt = ceil_div(K, 128);
  at::Tensor codes, scales;
  if (none(a[5]))
    codes = fresh({S, K / 2}, at::kByte);
  else
    codes = tensor(a[5], "codes"), bytes_of(codes, "codes", S * (K / 2));
  if (none(a[6]))
    scales = tiled ? fresh({S / 128 + E, kt, 512}, at::kByte) : fresh({S, K / 32}, at::kByte);
  else
    scales = tensor(a[6], "scales"), bytes_of(scales, "scales", tiled ? (S / 128 + E) * kt * 512 : S * (K / 32));
  if (K > INT32_MAX) bad("sizes beyond 2^31");
  const int64_t div = whole(a[2], "index_div");
  if (div < 1 || div > INT32_MAX) bad("index_div must be at least 1");
  if (!ok(g_entry.quantize(r.p, r.type, r.rows, r.stride, (int32_t)K, index, (int32_t)div, S, off, (int32_t)E,
                           static_cast<uint8_t*>(codes.data_ptr()), static_cast<uint8_t*>(scales.data_ptr()), tiled,
                           st.handle),
          "moe_fp4_mxfp4_quantize"))
    return nullptr;
  PyObject* res = PyTuple_New(2);
  PyTuple_SET_ITEM(res, 0, THPVariable_Wrap(codes));
  PyTuple_SET_ITEM(res, 1, THPVariable_Wrap(scales));
  return res;
NATIVE_END

// codes, scales, dtype, out, stream
NATIVE_BEGIN(dequantize, 5)
  const at::Tensor& codes = tensor(a[0], "codes");
  const Stream st(a[4], gpu_of(a, nargs));
  const at::ScalarType t = dtype_of(a[2]);
  if (codes.dim() < 1) bad("codes must be uint8 [.., K/2]");
  const int64_t half = codes.size(-1), n = codes.numel();
  if (half % 16 || half == 0 || half > INT32_MAX / 2) bad("K must be a multiple of 32");
  const int64_t rows = n / half;
  uint8_t* c = bytes_of(codes, "codes", 0);
  uint8_t* s = bytes_of(tensor(a[1], "scales"), "scales", rows * (half / 16));
  at::Tensor out;
  if (none(a[3])) {
    at::SmallVector<int64_t, 6> shape(codes.sizes().begin(), codes.sizes().end());
    shape.back() = 2 * half;
    out = fresh(shape, t);
  } else {
    out = tensor(a[3], "out");
    if (!out.is_cuda() || out.scalar_type() != t || !out.is_contiguous() || out.numel() != 2 * n)
      bad("out must be a contiguous GPU tensor of dtype with a value for each code");
  }
  if (!ok(g_entry.dequantize(c, s, rows, (int32_t)(2 * half), t == at::kFloat, out.data_ptr(), st.handle),
          "moe_fp4_mxfp4_dequantize"))
    return nullptr;
  return THPVariable_Wrap(out);
NATIVE_END

// scales, swiglu, out, stream
NATIVE_BEGIN(tile_scales, 4)
  const at::Tensor& s = tensor(a[0], "scales");
  const Stream st(a[3], gpu_of(a, nargs));
  if (s.dim() != 2 && s.dim() != 3) bad("scales must be [E, N, K/32] or [N, K/32]");
  const int64_t E = s.dim() == 3 ? s.size(0) : 1, N = s.size(-2), nb = s.size(-1);
  if (E > INT32_MAX || N > INT32_MAX || nb > INT32_MAX / 32) bad("sizes beyond 2^31");
  const uint8_t* p = bytes_of(s, "scales", 0);
  at::Tensor out;
  if (none(a[2]))
    out = fresh({E, ceil_div(N, 128), ceil_div(nb, 4), 512}, at::kByte);
  else
    out = tensor(a[2], "out"), bytes_of(out, "out", E * ceil_div(N, 128) * ceil_div(nb, 4) * 512);
  if (!ok(g_entry.tile_scales(p, (int32_t)E, (int32_t)N, (int32_t)(32 * nb), truth(a[1], "swiglu"),
                              static_cast<uint8_t*>(out.data_ptr()), st.handle),
          "moe_fp4_mxfp4_tile_scales"))
    return nullptr;
  return THPVariable_Wrap(out);
NATIVE_END

// a, a_scale, w, w_scale, offsets, swiglu, dtype, out, stream
NATIVE_BEGIN(matmul, 9)
  const at::Tensor& x = tensor(a[0], "a");
  const Stream st(a[8], gpu_of(a, nargs));
  if (x.dim() != 2) bad("a must be uint8 [M, K/2]");
  const int64_t M = x.size(0), K = 2 * x.size(1);
  int64_t n_off = 0;
  const int32_t* off = indices(a[4], "offsets", &n_off);
  const at::ScalarType t = dtype_of(a[6]);
  const Weights W = weights_of(M, K, a[2], a[3], off != nullptr, n_off, truth(a[5], "swiglu"), t);
  const uint8_t* codes = bytes_of(x, "a", 0);
  const uint8_t* scales = bytes_of(tensor(a[1], "a_scale"), "a_scale (tiled)", W.a_scale_bytes);
  const at::Tensor out = result(a[7], M, W.n_out, t, "out");
  if (!ok(g_entry.matmul(&W.dims, codes, scales, off, W.w, W.scales, out.data_ptr(), st.handle),
          "moe_fp4_mxfp4_matmul"))
    return nullptr;
  return THPVariable_Wrap(out);
NATIVE_END

// x, w, w_scale, offsets, row_index, index_div, swiglu, dtype, out, workspace, stream
NATIVE_BEGIN(linear, 11)
  const at::Tensor& x = tensor(a[0], "x");
  const Stream st(a[10], gpu_of(a, nargs));
  const Rows r = rows_of(x, "x");
  int64_t M = r.rows, n_off = 0;
  const int32_t* off = indices(a[3], "offsets", &n_off);
  const int32_t* index = indices(a[4], "row_index", &M);
  const int64_t div = whole(a[5], "index_div");
  if (div < 1 || div > INT32_MAX) bad("index_div must be at least 1");
  const at::ScalarType t = dtype_of(a[7]);
  const Weights W = weights_of(M, r.width, a[1], a[2], off != nullptr, n_off, truth(a[6], "swiglu"), t);
  const size_t need = g_entry.linear_workspace_bytes(&W.dims);
  if (need == 0) return ok(MOE_FP4_ERR_UNSUPPORTED, "moe_fp4_mxfp4_linear"), nullptr;
  // the workspace: none for few rows, the one given, or scratch memory for this call
  void* ws = nullptr;
  size_t ws_bytes = 0;
  c10::DataPtr scratch;
  if (!none(a[9])) {
    const at::Tensor& given = tensor(a[9], "workspace");
    ws = bytes_of(given, "workspace", (int64_t)need);
    ws_bytes = (size_t)given.numel();
  } else if (off != nullptr || M > MOE_FP4_MXFP4_FEW_ROWS) {
    ws_bytes = index ? g_entry.gathered_workspace_bytes(&W.dims, r.rows) : need;
    scratch = c10::GetAllocator(c10::kCUDA)->allocate(ws_bytes);
    ws = scratch.get();
  }
  const at::Tensor out = result(a[8], M, W.n_out, t, "out");
  if (!ok(g_entry.linear(&W.dims, r.p, r.type, r.rows, r.stride, index, (int32_t)div, off, W.w, W.scales,
                         out.data_ptr(), ws, ws_bytes, st.handle),
          "moe_fp4_mxfp4_linear"))
    return nullptr;
  return THPVariable_Wrap(out);
NATIVE_END

void weight_of(PyObject* o, const char* what, int64_t d, const void** p, int32_t* type) {
  if (none(o)) return;
  const at::Tensor& w = tensor(o, what);
  if (!w.is_cuda() || !w.is_contiguous() || w.dim() != 1 || w.size(0) != d)
    bad(std::string(what) + " must be a contiguous GPU tensor [" + std::to_string(d) + "]");
  *p = w.data_ptr();
  *type = type_of(w, what);
}

// x, weight, eps, out, stream
NATIVE_BEGIN(rms_norm, 5)
  const at::Tensor& x = tensor(a[0], "x");
  const Stream st(a[4], gpu_of(a, nargs));
  const Rows r = rows_of(x, "x");
  moe_fp4_block_norm_args n{};
  if (r.width > INT32_MAX) bad("sizes beyond 2^31");
  n.T = r.rows, n.d = (int32_t)r.width;
  n.residual = r.p, n.residual_type = r.type, n.residual_stride = r.stride;
  n.scale = 1.f, n.eps = (float)real(a[2], "eps");
  weight_of(a[1], "weight", r.width, &n.next_weight, &n.next_weight_type);
  const at::Tensor out = result(a[3], r.rows, r.width, at::kBFloat16, "out");
  n.normed = out.data_ptr();
  if (!ok(g_entry.block_norm(&n, st.handle), "moe_fp4_block_norm")) return nullptr;
  return THPVariable_Wrap(out);
NATIVE_END

// residual, y, y2, post_norm, post_weight, gate, gate_sigmoid, scale, next_norm, next_weight, eps, out, normed, stream
NATIVE_BEGIN(block_residual, 14)
  const at::Tensor& res = tensor(a[0], "residual");
  const Stream st(a[13], gpu_of(a, nargs));
  const Rows r = rows_of(res, "residual");
  const int64_t T = r.rows, d = r.width;
  if (d > INT32_MAX) bad("sizes beyond 2^31");
  moe_fp4_block_norm_args n{};
  n.T = T, n.d = (int32_t)d;
  n.residual = r.p, n.residual_type = r.type, n.residual_stride = r.stride;
  const Rows y = rows_of(tensor(a[1], "y"), "y");
  if (y.rows != T || y.width != d) bad("y must have residual's shape");
  n.y = y.p, n.y_type = y.type, n.y_stride = y.stride;
  if (!none(a[2])) {
    const Rows y2 = rows_of(tensor(a[2], "y2"), "y2");
    if (y2.rows != T || y2.width != d) bad("y2 must have residual's shape");
    n.y2 = y2.p, n.y2_type = y2.type, n.y2_stride = y2.stride;
  }
  n.post_norm = truth(a[3], "post_norm");
  weight_of(a[4], "post_weight", d, &n.post_weight, &n.post_weight_type);
  if (!none(a[5])) {
    const at::Tensor& g = tensor(a[5], "gate");
    const int64_t dim = g.dim(), s0 = dim > 0 ? g.size(0) : 0, s1 = dim == 2 ? g.size(1) : 1;
    n.gate_sigmoid = truth(a[6], "gate_sigmoid");
    n.gate_stride = d;
    if (dim == 2 && s0 == T && s1 == d && !(T > 1 && d == 1)) {
      const Rows e = rows_of(g, "gate");
      n.gate_shape = MOE_FP4_GATE_ELEMENT, n.gate_stride = e.stride;
    } else {
      if (dim == 1 && T == d) bad("gate is ambiguous for T = d: give [T, 1] or [1, d]");
      if ((dim == 1 || dim == 2) && s0 == T && s1 == 1)
        n.gate_shape = MOE_FP4_GATE_TOKEN;
      else if ((dim == 1 && s0 == d) || (dim == 2 && s0 == 1 && s1 == d))
        n.gate_shape = MOE_FP4_GATE_CHANNEL;
      if (n.gate_shape == MOE_FP4_GATE_NONE || !g.is_cuda() || !g.is_contiguous())
        bad("gate must be a GPU tensor [T], [d] or [T, d]");
    }
    n.gate = g.data_ptr(), n.gate_type = type_of(g, "gate");
  }
  n.scale = (float)real(a[7], "scale"), n.eps = (float)real(a[10], "eps");
  const bool in_place = a[11] == a[0];
  const at::Tensor out = in_place ? res : result(a[11], T, d, res.scalar_type(), "out");
  n.out = out.data_ptr(), n.out_stride = in_place ? r.stride : d;
  at::Tensor normed;
  if (truth(a[8], "next_norm")) {
    weight_of(a[9], "next_weight", d, &n.next_weight, &n.next_weight_type);
    normed = result(a[12], T, d, at::kBFloat16, "normed");
    n.normed = normed.data_ptr();
  } else if (!none(a[9]) || !none(a[12])) {
    bad("next_norm=False takes no next_weight and no normed");
  }
  if (!ok(g_entry.block_norm(&n, st.handle), "moe_fp4_block_norm")) return nullptr;
  PyObject* both = PyTuple_New(2);
  if (in_place) {
    Py_INCREF(a[0]);
    PyTuple_SET_ITEM(both, 0, a[0]);
  } else {
    PyTuple_SET_ITEM(both, 0, THPVariable_Wrap(out));
  }
  if (normed.defined()) {
    PyTuple_SET_ITEM(both, 1, THPVariable_Wrap(normed));
  } else {
    Py_INCREF(Py_None);
    PyTuple_SET_ITEM(both, 1, Py_None);
  }
  return both;
NATIVE_END

// addresses (in Entry's order), raise
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  constexpr Py_ssize_t n = sizeof(Entry) / sizeof(void*);
  if (nargs != 2 || !PyTuple_Check(a[0]) || PyTuple_GET_SIZE(a[0]) != n || !PyCallable_Check(a[1])) {
    PyErr_SetString(PyExc_TypeError, "bind: the entry points' addresses and a callable");
    return nullptr;
  }
  void* p[n];
  for (Py_ssize_t i = 0; i < n; ++i) {
    p[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(a[0], i));
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_TypeError, "bind: a null address");
      return nullptr;
    }
  }
  memcpy(&g_entry, p, sizeof(p));
  Py_INCREF(a[1]);
  Py_XDECREF(g_raise);
  g_raise = a[1];
  Py_RETURN_NONE;
}

#define METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind),   METHOD(quantize), METHOD(dequantize), METHOD(tile_scales),
                         METHOD(matmul), METHOD(linear),   METHOD(rms_norm),   METHOD(block_residual),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops_native() { return PyModule_Create(&module); }
