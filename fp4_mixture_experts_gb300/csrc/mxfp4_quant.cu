// MXFP4 quantisation of rows, the way back, and the products' scale layout.
//
// Per block of 32 elements the scale is 2^e, e = max(floor(log2 amax) - 2,
// -127) (2 is the exponent of the largest E2M1 value, 6), and an element's
// code the E2M1 value nearest to x 2^-e.  floor(log2 amax) is the exponent
// field of amax in fp32, so the scale byte is that field minus 2, at least 0
// (every subnormal ends there); x 2^-e is exact, and the hardware conversion
// (round to nearest even, saturating) gives the code.  Two lanes share a
// block, 16 elements each: loads of 16 bytes, one shuffle for amax, one
// 8-byte store of codes.
#include "moe_fp4_internal.cuh"
#include "mxfp4_ops.cuh"

namespace moe_fp4 {
namespace {

__device__ int32_t g_quant_err[4];

constexpr int kPer = 16;  // elements per thread
constexpr int kThreads = 256;

struct QuantParams {
  const void* x;
  int64_t x_rows, x_stride;
  const int32_t* row_index;
  const int32_t* offsets;
  uint8_t* codes;
  uint8_t* scales;
  int64_t rows;
  int K, div, groups;
};

template <bool F32, bool VEC, bool TILED>
__global__ void __launch_bounds__(kThreads) mxfp4_quantize_kernel(const QuantParams P) {
  griddep_launch_dependents();  // a product that waits for these rows may be set up meanwhile
  const int per_row = P.K / kPer, nb = P.K / 32, kt = (P.K + 127) / 128;
  const int64_t total = P.rows * per_row;
  // whole warps leave the loop together (the shuffle below needs both lanes of a block)
  for (int64_t i0 = (int64_t)blockIdx.x * kThreads + (threadIdx.x & ~31); i0 < total;
       i0 += (int64_t)gridDim.x * kThreads) {
    const int64_t i = i0 + (threadIdx.x & 31);
    const bool in = i < total;
    const int64_t r = in ? i / per_row : 0;
    const int c = in ? (int)(i - r * per_row) : 0;
    uint32_t w[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) w[j] = 0;
    int64_t src = r;
    if (P.row_index) {
      src = P.row_index[r];
      src = src < 0 ? -1 : src / P.div;
    }
    if (src >= 0 && src < P.x_rows) {
      if (in) load16_raw<F32, VEC>(P.x, src * P.x_stride + (int64_t)c * kPer, w);
    } else if (c == 0) {
      atomicOr(&g_quant_err[0], kErrBadExpertId);
    }
    float v[kPer];
    unpack16<F32>(w, v);
    uint32_t sb;
    const uint2 q = quantize16(v, sb);
    if (!in) continue;
    *reinterpret_cast<uint2*>(P.codes + r * (P.K / 2) + (int64_t)c * (kPer / 2)) = q;
    if (c & 1) continue;
    const int b = c >> 1;
    if (!TILED) {
      P.scales[r * nb + b] = (uint8_t)sb;
    } else {
      int64_t tile = r >> 7, row = r & 127;
      if (P.offsets) {
        const int e = find_group(P.offsets, P.groups, r, P.rows);
        if (e < 0) continue;
        const int64_t first = P.offsets[e];
        tile = (first >> 7) + e + ((r - first) >> 7);
        row = (r - first) & 127;
      }
      uint8_t* t = P.scales + (tile * kt + (b >> 2)) * 512 + 16 * (row & 31) + 4 * (row >> 5);
      t[b & 3] = (uint8_t)sb;
      if (b == nb - 1)
        for (int p = (b & 3) + 1; p < 4; ++p) t[p] = 0;
    }
  }
}

template <bool F32>
__global__ void __launch_bounds__(kThreads)
mxfp4_dequantize_kernel(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t total,
                        void* __restrict__ out) {
  // one thread: 8 elements, 4 bytes of codes
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
    const uint32_t c = __ldg(reinterpret_cast<const uint32_t*>(codes) + i);
    const float s = e8m0_to_f32(__ldg(scales + (i >> 2)));
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t h = e2m1x2_to_f16x2((c >> (8 * j)) & 0xFFu);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      v[2 * j] = f.x * s;
      v[2 * j + 1] = f.y * s;
    }
    if (F32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + 8 * i);
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = (uint32_t)f32_to_bf16_rn(v[2 * j]) | ((uint32_t)f32_to_bf16_rn(v[2 * j + 1]) << 16);
      reinterpret_cast<uint4*>(out)[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// one thread: the four scales of one row and tile, one word
__global__ void __launch_bounds__(kThreads)
tile_scales_kernel(const uint8_t* __restrict__ scales, int N, int nb, int rt, int kt, int swiglu, int64_t words,
                   uint32_t* __restrict__ tiled) {
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < words; i += (int64_t)gridDim.x * kThreads) {
    const int w = (int)(i & 127);                  // word of the tile: row (w % 4) * 32 + w / 4
    const int64_t t = i >> 7;
    const int k = (int)(t % kt);
    const int64_t er = t / kt;
    const int row = (int)(er % rt) * 128 + (w & 3) * 32 + (w >> 2);
    const int64_t e = er / rt;
    uint32_t v = 0;
    if (row < N) {
      const int src = swiglu ? (row & 1) * (N / 2) + (row >> 1) : row;
      const uint8_t* p = scales + (e * N + src) * nb + 4 * k;
      for (int j = 0; j < 4 && 4 * k + j < nb; ++j) v |= (uint32_t)p[j] << (8 * j);
    }
    tiled[i] = v;
  }
}

template <bool F32, bool VEC>
cudaError_t launch_quant(const QuantParams& P, bool tiled, int grid, cudaStream_t st) {
  if (tiled)
    mxfp4_quantize_kernel<F32, VEC, true><<<grid, kThreads, 0, st>>>(P);
  else
    mxfp4_quantize_kernel<F32, VEC, false><<<grid, kThreads, 0, st>>>(P);
  return cudaGetLastError();
}

int grid_for(int64_t threads, int per_sm) {
  const int64_t blocks = (threads + kThreads - 1) / kThreads, cap = (int64_t)num_sms() * per_sm;
  return (int)(blocks < cap ? blocks : cap);
}

}  // namespace

cudaError_t launch_mxfp4_quantize(const MxRows& R, uint8_t* codes, uint8_t* scales, bool tiled, cudaStream_t st) {
  QuantParams P{R.x, R.x_rows, R.x_stride, R.row_index, R.offsets, codes, scales, R.rows, R.K, R.div, R.groups};
  const int64_t size = R.f32 ? 4 : 2;
  const bool vec = ((uintptr_t)R.x & 15) == 0 && (R.x_stride * size) % 16 == 0;
  const int grid = grid_for(R.rows * (R.K / kPer), 16);
  if (R.f32) return vec ? launch_quant<true, true>(P, tiled, grid, st) : launch_quant<true, false>(P, tiled, grid, st);
  return vec ? launch_quant<false, true>(P, tiled, grid, st) : launch_quant<false, false>(P, tiled, grid, st);
}

cudaError_t ops_quant_error(int32_t* word, bool clear, cudaStream_t st) {
  if (clear) {
    const int32_t zero = 0;
    return cudaMemcpyToSymbolAsync(g_quant_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, st);
  }
  return cudaMemcpyFromSymbolAsync(word, g_quant_err, sizeof(*word), 0, cudaMemcpyDeviceToHost, st);
}

int check_mx_rows(const MxRows& R) {
  if (R.K <= 0 || R.K % 32 != 0 || R.K > 32768 || R.rows < 0 || R.x_rows < 0 || R.div < 1) return MOE_FP4_ERR_INVALID_ARG;
  if (R.rows >= (1LL << 31) || R.rows * R.K >= (1LL << 36)) return MOE_FP4_ERR_INVALID_ARG;
  if (R.rows == 0) return MOE_FP4_OK;
  if (!R.x || R.x_stride < R.K || R.x_stride >= (1LL << 32) || R.x_rows >= (1LL << 31)) return MOE_FP4_ERR_INVALID_ARG;
  if (((uintptr_t)R.x & (R.f32 ? 3 : 1)) || ((uintptr_t)R.row_index & 3) || ((uintptr_t)R.offsets & 3))
    return MOE_FP4_ERR_INVALID_ARG;
  if (!R.row_index && R.rows > R.x_rows) return MOE_FP4_ERR_INVALID_ARG;
  if (R.offsets && (R.groups < 1 || R.groups > kMaxGroups)) return MOE_FP4_ERR_INVALID_ARG;
  return MOE_FP4_OK;
}

}  // namespace moe_fp4

using namespace moe_fp4;

extern "C" {

size_t moe_fp4_mxfp4_tiled_scale_bytes(int64_t rows, int32_t groups, int32_t K) {
  if (rows < 0 || rows >= (1LL << 31) || groups < 1 || groups > kMaxGroups || K <= 0 || K % 32 != 0 || K > 32768)
    return 0;
  return (size_t)(rows / 128 + groups) * ((K + 127) / 128) * 512;
}

int moe_fp4_mxfp4_quantize(const void* x, int x_type, int64_t x_rows, int64_t x_stride, int32_t K,
                           const int32_t* row_index, int32_t index_div, int64_t rows, const int32_t* group_offsets,
                           int32_t groups, uint8_t* codes, uint8_t* scales, int tiled, void* cuda_stream) {
  if (x_type != MOE_FP4_TYPE_BF16 && x_type != MOE_FP4_TYPE_F32) return MOE_FP4_ERR_INVALID_ARG;
  const MxRows R{x, x_rows, x_stride, row_index, group_offsets, rows, K, row_index ? index_div : 1, groups,
                 x_type == MOE_FP4_TYPE_F32};
  const int rc = check_mx_rows(R);
  if (rc != MOE_FP4_OK || rows == 0) return rc;
  if (!codes || !scales || ((uintptr_t)codes & 15) || (tiled && ((uintptr_t)scales & 15)))
    return MOE_FP4_ERR_INVALID_ARG;
  if (group_offsets && !tiled) return MOE_FP4_ERR_INVALID_ARG;
  return launch_mxfp4_quantize(R, codes, scales, tiled != 0, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess
             ? MOE_FP4_OK
             : MOE_FP4_ERR_CUDA;
}

int moe_fp4_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t K, int out_type,
                             void* out, void* cuda_stream) {
  if (rows < 0 || K <= 0 || K % 32 != 0 || K > 32768 || rows >= (1LL << 31) || rows * K >= (1LL << 36))
    return MOE_FP4_ERR_INVALID_ARG;
  if (out_type != MOE_FP4_TYPE_BF16 && out_type != MOE_FP4_TYPE_F32) return MOE_FP4_ERR_INVALID_ARG;
  if (rows == 0) return MOE_FP4_OK;
  if (!codes || !scales || !out || ((uintptr_t)codes & 15) || ((uintptr_t)out & 15)) return MOE_FP4_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const int64_t total = rows * (K / 8);
  const int grid = grid_for(total, 16);
  if (out_type == MOE_FP4_TYPE_F32)
    mxfp4_dequantize_kernel<true><<<grid, kThreads, 0, st>>>(codes, scales, total, out);
  else
    mxfp4_dequantize_kernel<false><<<grid, kThreads, 0, st>>>(codes, scales, total, out);
  return cudaGetLastError() == cudaSuccess ? MOE_FP4_OK : MOE_FP4_ERR_CUDA;
}

int moe_fp4_mxfp4_tile_scales(const uint8_t* scales, int32_t E, int32_t N, int32_t K, int swiglu, uint8_t* tiled,
                              void* cuda_stream) {
  if (!scales || !tiled || ((uintptr_t)tiled & 15) || E < 1 || E > kMaxGroups || N < 1 || K <= 0 || K % 32 != 0 ||
      K > 32768 || (swiglu && N % 2 != 0))
    return MOE_FP4_ERR_INVALID_ARG;
  const int rt = (N + 127) / 128, kt = (K + 127) / 128;
  const int64_t words = (int64_t)E * rt * kt * 128;
  tile_scales_kernel<<<grid_for(words, 16), kThreads, 0, static_cast<cudaStream_t>(cuda_stream)>>>(
      scales, N, K / 32, rt, kt, swiglu, words, reinterpret_cast<uint32_t*>(tiled));
  return cudaGetLastError() == cudaSuccess ? MOE_FP4_OK : MOE_FP4_ERR_CUDA;
}

int moe_fp4_ops_check(void* cuda_stream) {
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  cudaError_t (*const words[])(int32_t*, bool, cudaStream_t) = {ops_quant_error, ops_mm_error, ops_mm1_error,
                                                              ops_mm2_error};
  int32_t bits = 0;
  for (auto word : words) {
    int32_t w = 0;
    if (word(&w, false, st) != cudaSuccess || cudaStreamSynchronize(st) != cudaSuccess) return MOE_FP4_ERR_CUDA;
    bits |= w;
  }
  if (bits == 0) return MOE_FP4_OK;
  for (auto word : words)
    if (word(nullptr, true, st) != cudaSuccess) return MOE_FP4_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return MOE_FP4_ERR_CUDA;
  return MOE_FP4_ERR_DEVICE;
}

}  // extern "C"
