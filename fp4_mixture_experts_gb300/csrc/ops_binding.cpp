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
  decltype(&moe_fp4_fp8_tile_scales) fp8_tile_scales;
  decltype(&moe_fp4_fp8_linear_workspace_bytes) fp8_linear_workspace_bytes;
  decltype(&moe_fp4_fp8_linear) fp8_linear;
  decltype(&moe_fp4_latent_decode_workspace_bytes) latent_decode_workspace_bytes;
  decltype(&moe_fp4_latent_decode) latent_decode;
  decltype(&moe_fp4_latent_attention_workspace_bytes) latent_attention_workspace_bytes;
  decltype(&moe_fp4_latent_attention) latent_attention;
  decltype(&moe_fp4_page_slots) page_slots;
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
  if (R > 0 && ((t.stride(1) != 1 && K > 1) || (t.stride(0) < K && R > 1)))
    bad(std::string(what) + " must have contiguous, separate rows");
  return {R, K, R > 1 ? t.stride(0) : K, type_of(t, what), t.data_ptr()};
}

uint8_t* bytes_of(const at::Tensor& t, const char* what, int64_t numel) {
  if (t.scalar_type() != at::kByte || !t.is_cuda() || !t.is_contiguous() || t.numel() < numel)
    bad(std::string(what) + " must be a contiguous uint8 GPU tensor of at least " + std::to_string(numel) + " elements");
  return static_cast<uint8_t*>(t.data_ptr());
}

uint8_t* e4m3_of(const at::Tensor& t, const char* what) {
  if (t.scalar_type() != at::kFloat8_e4m3fn || !t.is_cuda() || !t.is_contiguous())
    bad(std::string(what) + " must be a contiguous float8_e4m3fn GPU tensor");
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
                   at::ScalarType t, bool fp8 = false) {
  const at::Tensor& w = tensor(w_, "w");
  if ((w.dim() != 2 && w.dim() != 3) || w.size(-1) * (fp8 ? 1 : 2) != K)
    bad(fp8 ? "w must be float8_e4m3fn [E, N, K] or [N, K] with K = " + std::to_string(K)
            : "w must be uint8 [E, N, K/2] or [N, K/2] with K = " + std::to_string(K));
  const int64_t E = w.dim() == 3 ? w.size(0) : 1, N = w.size(-2);
  if (grouped ? n_offsets != E + 1 : E != 1) bad("several matrices need offsets, of E + 1 elements");
  if (swiglu && N % 2) bad("swiglu needs an even number of features");
  if (M > INT32_MAX || N > INT32_MAX || E > INT32_MAX || K > INT32_MAX) bad("sizes beyond 2^31");
  const int64_t kt = ceil_div(K, 128);
  return {{(int32_t)M, (int32_t)N, (int32_t)K, (int32_t)E, swiglu, t == at::kFloat ? MOE_FP4_TYPE_F32 : MOE_FP4_TYPE_BF16},
          fp8 ? e4m3_of(w, "w") : bytes_of(w, "w", 0),
          bytes_of(tensor(scales_, "w_scale"),
                   fp8 ? "w_scale (tiled, by fp8_tile_scales)" : "w_scale (tiled, by mxfp4_tile_scales)",
                   E * ceil_div(N, 128) * kt * 512),
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

// scales, N, K, swiglu, out, stream
NATIVE_BEGIN(fp8_tile_scales, 6)
  const at::Tensor& s = tensor(a[0], "scales");
  const Stream st(a[5], gpu_of(a, nargs));
  const int64_t N = whole(a[1], "N"), K = whole(a[2], "K");
  if (N < 1 || N > INT32_MAX || K < 1 || K > INT32_MAX) bad("N and K must be a matrix's sizes");
  const int64_t rt = ceil_div(N, 128), kt = ceil_div(K, 128);
  if ((s.dim() != 2 && s.dim() != 3) || s.size(-2) != rt || s.size(-1) != kt)
    bad("scales must be uint8 [E, ceil(N/128), ceil(K/128)], or without E");
  const int64_t E = s.dim() == 3 ? s.size(0) : 1;
  if (E > INT32_MAX) bad("sizes beyond 2^31");
  const uint8_t* p = bytes_of(s, "scales", 0);
  at::Tensor out;
  if (none(a[4]))
    out = fresh({E, rt, kt, 512}, at::kByte);
  else
    out = tensor(a[4], "out"), bytes_of(out, "out", E * rt * kt * 512);
  if (!ok(g_entry.fp8_tile_scales(p, (int32_t)E, (int32_t)N, (int32_t)K, truth(a[3], "swiglu"),
                                  static_cast<uint8_t*>(out.data_ptr()), st.handle),
          "moe_fp4_fp8_tile_scales"))
    return nullptr;
  return THPVariable_Wrap(out);
NATIVE_END

// x, w, w_scale, offsets, swiglu, dtype, out, workspace, stream
NATIVE_BEGIN(fp8_linear, 9)
  const at::Tensor& x = tensor(a[0], "x");
  const Stream st(a[8], gpu_of(a, nargs));
  const Rows r = rows_of(x, "x");
  int64_t n_off = 0;
  const int32_t* off = indices(a[3], "offsets", &n_off);
  const at::ScalarType t = dtype_of(a[5]);
  const Weights W = weights_of(r.rows, r.width, a[1], a[2], off != nullptr, n_off, truth(a[4], "swiglu"), t, true);
  const size_t need = g_entry.fp8_linear_workspace_bytes(&W.dims);
  if (need == 0) return ok(MOE_FP4_ERR_UNSUPPORTED, "moe_fp4_fp8_linear"), nullptr;
  void* ws = nullptr;
  c10::DataPtr scratch;
  if (!none(a[7])) {
    ws = bytes_of(tensor(a[7], "workspace"), "workspace", (int64_t)need);
  } else if (off != nullptr || r.rows > MOE_FP4_MXFP4_FEW_ROWS) {
    scratch = c10::GetAllocator(c10::kCUDA)->allocate(need);
    ws = scratch.get();
  }
  const at::Tensor out = result(a[6], r.rows, W.n_out, t, "out");
  if (!ok(g_entry.fp8_linear(&W.dims, r.p, r.type, r.rows, r.stride, off, W.w, W.scales, out.data_ptr(), ws, need,
                             st.handle),
          "moe_fp4_fp8_linear"))
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

const at::Tensor& bf16_of(PyObject* o, const char* what, int64_t dim) {
  const at::Tensor& t = tensor(o, what);
  if (t.scalar_type() != at::kBFloat16 || !t.is_cuda() || t.dim() != dim)
    bad(std::string(what) + " must be a bf16 GPU tensor of " + std::to_string(dim) + " dimensions");
  return t;
}

// [T, H, W]: the last dimension contiguous, rows that start on 16 bytes; the strides of a dimension of one element do
// not matter
struct Heads {
  int64_t rows, heads, width, stride, head_stride;
  void* p;
};

Heads heads_of(PyObject* o, const char* what, int64_t width) {
  const at::Tensor& t = bf16_of(o, what, 3);
  if (t.size(2) != width) bad(std::string(what) + " must have " + std::to_string(width) + " elements a head");
  const int64_t T = t.size(0), H = t.size(1);
  Heads h{T, H, width, T > 1 ? t.stride(0) : H * width, H > 1 ? t.stride(1) : width, t.data_ptr()};
  if (T == 0 || H == 0) return h;
  if (t.stride(2) != 1 || h.stride < width || h.head_stride < width || h.stride % 8 || h.head_stride % 8 ||
      reinterpret_cast<uintptr_t>(h.p) % 16)
    bad(std::string(what) + " must have contiguous heads, apart, that start on 16 bytes");
  return h;
}

const int32_t* table_of(PyObject* o, const char* what, int64_t rows, int64_t* width, int64_t* stride) {
  const at::Tensor& t = tensor(o, what);
  if (t.scalar_type() != at::kInt || !t.is_cuda() || t.dim() != 2 || t.size(0) != rows ||
      (rows > 0 && ((t.stride(1) != 1 && t.size(1) > 1) || (t.stride(0) < t.size(1) && rows > 1))))
    bad(std::string(what) + " must be an int32 GPU tensor of " + std::to_string(rows) + " separate, contiguous rows");
  *width = t.size(1);
  *stride = rows > 1 ? t.stride(0) : t.size(1);
  return static_cast<const int32_t*>(t.data_ptr());
}

// q, cache, block_table, lengths, scale, out, workspace, stream
NATIVE_BEGIN(latent_decode, 8)
  const Stream st(a[7], gpu_of(a, nargs));
  const Heads q = heads_of(a[0], "q", 576);
  const at::Tensor& c = bf16_of(a[1], "cache", 3);
  if (c.size(2) != 576 || !c.is_contiguous()) bad("cache must be contiguous [pages, page, 576]");
  int64_t width, n = 0;
  moe_fp4_latent_decode_args d{};
  d.table = table_of(a[2], "block_table", q.rows, &width, &d.table_stride);
  if (none(a[3])) bad("lengths must be a contiguous 1-D int32 GPU tensor");
  d.lengths = indices(a[3], "lengths", &n);
  if (n != q.rows) bad("lengths must have an element for each sequence");
  if (q.rows > INT32_MAX || q.heads > INT32_MAX || c.size(0) > INT32_MAX || c.size(1) > INT32_MAX || width > INT32_MAX)
    bad("sizes beyond 2^31");
  d.B = (int32_t)q.rows, d.H = (int32_t)q.heads, d.width = (int32_t)width;
  d.pages = (int32_t)c.size(0), d.page = (int32_t)c.size(1);
  d.scale = (float)real(a[4], "scale");
  d.q = q.p, d.q_stride = q.stride, d.q_head_stride = q.head_stride, d.cache = c.data_ptr();
  const size_t need = g_entry.latent_decode_workspace_bytes(d.H);
  if (need == 0) bad("q must have 1 to " + std::to_string(MOE_FP4_LATENT_MAX_HEADS) + " heads");
  void* ws;
  c10::DataPtr scratch;
  if (!none(a[6])) {
    ws = bytes_of(tensor(a[6], "workspace"), "workspace", (int64_t)need);
  } else {
    scratch = c10::GetAllocator(c10::kCUDA)->allocate(need);
    ws = scratch.get();
  }
  at::Tensor out;
  if (none(a[5])) {
    out = fresh({q.rows, q.heads, 512}, at::kBFloat16);
  } else {
    out = bf16_of(a[5], "out", 3);
    if (!out.is_contiguous() || out.size(0) != q.rows || out.size(1) != q.heads || out.size(2) != 512)
      bad("out must be contiguous [B, H, 512]");
  }
  d.out = out.data_ptr();
  if (!ok(g_entry.latent_decode(&d, ws, need, st.handle), "moe_fp4_latent_decode")) return nullptr;
  return THPVariable_Wrap(out);
NATIVE_END

// q, kv, k_rope, q_offsets, k_offsets, scale, causal, out, workspace, stream
NATIVE_BEGIN(latent_attention, 10)
  const Stream st(a[9], gpu_of(a, nargs));
  const Heads q = heads_of(a[0], "q", 192), kv = heads_of(a[1], "kv", 256);
  const at::Tensor& rope = bf16_of(a[2], "k_rope", 2);
  if (kv.heads != q.heads) bad("kv must have q's heads");
  if (rope.size(0) != kv.rows || rope.size(1) != 64) bad("k_rope must be [Tk, 64]");
  moe_fp4_latent_attention_args d{};
  d.rope_stride = kv.rows > 1 ? rope.stride(0) : 64;
  if (kv.rows > 0 && (rope.stride(1) != 1 || d.rope_stride < 64 || d.rope_stride % 8 ||
                      reinterpret_cast<uintptr_t>(rope.data_ptr()) % 16))
    bad("k_rope must have contiguous rows, apart, that start on 16 bytes");
  int64_t nq = 0, nk = 0;
  if (none(a[3]) || none(a[4])) bad("q_offsets and k_offsets must be contiguous 1-D int32 GPU tensors");
  d.q_offsets = indices(a[3], "q_offsets", &nq), d.k_offsets = indices(a[4], "k_offsets", &nk);
  if (nq < 1 || nq != nk) bad("q_offsets and k_offsets must have B + 1 elements each");
  if (q.heads < 1 || q.heads > MOE_FP4_LATENT_MAX_HEADS)
    bad("q must have 1 to " + std::to_string(MOE_FP4_LATENT_MAX_HEADS) + " heads");
  if (nq > INT32_MAX) bad("sizes beyond 2^31");
  d.B = (int32_t)(nq - 1), d.H = (int32_t)q.heads, d.Tq = q.rows, d.Tk = kv.rows;
  d.scale = (float)real(a[5], "scale"), d.causal = truth(a[6], "causal");
  d.q = q.p, d.q_stride = q.stride, d.q_head_stride = q.head_stride;
  d.kv = kv.p, d.kv_stride = kv.stride, d.kv_head_stride = kv.head_stride, d.k_rope = rope.data_ptr();
  at::Tensor out;
  if (none(a[7])) {
    out = fresh({q.rows, q.heads, 128}, at::kBFloat16);
  } else {
    out = bf16_of(a[7], "out", 3);
    if (!out.is_contiguous() || out.size(0) != q.rows || out.size(1) != q.heads || out.size(2) != 128)
      bad("out must be contiguous [Tq, H, 128]");
  }
  d.out = out.data_ptr();
  const size_t need = g_entry.latent_attention_workspace_bytes();
  void* ws;
  c10::DataPtr scratch;
  if (!none(a[8])) {
    ws = bytes_of(tensor(a[8], "workspace"), "workspace", (int64_t)need);
  } else {
    scratch = c10::GetAllocator(c10::kCUDA)->allocate(need);
    ws = scratch.get();
  }
  if (!ok(g_entry.latent_attention(&d, ws, need, st.handle), "moe_fp4_latent_attention")) return nullptr;
  return THPVariable_Wrap(out);
NATIVE_END

// lengths, new_tokens, block_table, free_pages, page_size, tokens, then the results or None: slots, positions, lengths,
// q_offsets, k_offsets, taken; stream
NATIVE_BEGIN(page_slots, 13)
  const Stream st(a[12], gpu_of(a, nargs));
  moe_fp4_page_slots_args d{};
  int64_t B = 0, n = 0, width;
  for (int i : {0, 1, 3})
    if (none(a[i])) bad("lengths, new_tokens and free_pages must be contiguous 1-D int32 GPU tensors");
  d.lengths = indices(a[0], "lengths", &B), d.new_tokens = indices(a[1], "new_tokens", &n);
  if (n != B) bad("new_tokens must have an element for each of lengths");
  d.table = const_cast<int32_t*>(table_of(a[2], "block_table", B, &width, &d.table_stride));
  d.free_pages = indices(a[3], "free_pages", &d.free_count);
  const int64_t page = whole(a[4], "page_size");
  d.tokens = whole(a[5], "tokens");
  if (d.tokens < 0 || d.tokens > INT32_MAX) bad("tokens must be 0 to 2^31 - 1");
  if (B > INT32_MAX || width > INT32_MAX || page > INT32_MAX) bad("sizes beyond 2^31");
  if (page < 1) bad("page_size must be at least 1");
  d.B = (int32_t)B, d.page = (int32_t)page, d.width = (int32_t)width;
  const struct {
    const char* what;
    int64_t size;  // -1: no dimension
    at::ScalarType type;
  } results[6] = {{"slots", d.tokens, at::kLong}, {"positions", d.tokens, at::kInt}, {"lengths", B, at::kInt},
                  {"q_offsets", B + 1, at::kInt}, {"k_offsets", B + 1, at::kInt},    {"taken", -1, at::kInt}};
  // Without given results: one block of memory, the slots' 64 bits first (a view of it takes 0.2 us, a tensor of its own 1 us)
  at::Tensor out[6], block;
  int64_t at_element = 0;
  for (int i = 0; i < 6; ++i) {
    const int64_t size = results[i].size;
    const at::IntArrayRef shape(&size, size < 0 ? 0 : 1);
    if (none(a[6 + i])) {
      if (!block.defined()) block = fresh({3 * d.tokens + 3 * B + 3}, at::kInt);
      out[i] = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(block.storage()), block.key_set(),
                                                        c10::scalarTypeToTypeMeta(results[i].type));
      out[i].unsafeGetTensorImpl()->set_storage_offset(at_element);
      out[i].unsafeGetTensorImpl()->set_sizes_contiguous(shape);
      at_element += i == 0 ? 2 * size : size < 0 ? 1 : size;  // (of 32 bits; the slots are at 0)
    } else {
      out[i] = tensor(a[6 + i], results[i].what);
      if (out[i].scalar_type() != results[i].type || !out[i].is_cuda() || !out[i].is_contiguous() || out[i].sizes() != shape)
        bad(std::string("out's ") + results[i].what + " must be as of a call of these sizes");
    }
  }
  d.slots = static_cast<int64_t*>(out[0].data_ptr());
  int32_t** const to[5] = {&d.positions, &d.out_lengths, &d.q_offsets, &d.k_offsets, &d.taken};
  for (int i = 0; i < 5; ++i) *to[i] = static_cast<int32_t*>(out[i + 1].data_ptr());
  if (!ok(g_entry.page_slots(&d, st.handle), "moe_fp4_page_slots")) return nullptr;
  PyObject* res = PyTuple_New(6);
  for (int i = 0; i < 6; ++i) PyTuple_SET_ITEM(res, i, THPVariable_Wrap(out[i]));
  return res;
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
                         METHOD(fp8_tile_scales), METHOD(fp8_linear), METHOD(latent_decode), METHOD(latent_attention), METHOD(page_slots),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_ops_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops_native() { return PyModule_Create(&module); }
