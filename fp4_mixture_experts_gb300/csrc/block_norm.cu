// The end of a block in one pass over its rows:
//
//   b = y + y2;  b *= rsqrt(mean b^2 + eps);  b *= post_weight;  b *= gate | sigmoid(gate)
//   out = residual + scale b;  normed = out rsqrt(mean out^2 + eps) next_weight
//
// One CTA per row.  The row stays in registers between its two sums of
// squares, so that every operand is read once; residual and gate are loaded
// before the first sum is ready, so that the wait for it hides their latency.
// Sums are fp32: a thread's elements in order, then a tree over the CTA (a
// fixed order: the same bits on every call).  HBM-bound for many rows.
#include "moe_fp4_internal.cuh"

namespace moe_fp4 {
namespace {

struct NormParams {
  moe_fp4_block_norm_args a;
  float k;  // d^-1/2: the squares of k v sum to the mean, which overflows only if the mean itself does
};

// where element j of a thread's chunk c is: chunks of 8 adjacent elements
// (VEC: rows start on 16 bytes and d is a multiple of 8), else interleaved
template <bool VEC>
__device__ __forceinline__ int elem(int c, int j) {
  return VEC ? (c * (int)blockDim.x + (int)threadIdx.x) * 8 + j
             : (c * 8 + j) * (int)blockDim.x + (int)threadIdx.x;
}

template <bool VEC>
__device__ __forceinline__ void load8(const void* base, int type, int64_t row_at, int c, int d, float (&v)[8]) {
  if (VEC) {
    const int e = elem<true>(c, 0);
    if (e >= d) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
      return;
    }
    if (type == MOE_FP4_TYPE_F32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + row_at + e);
      const float4 x = p[0], y = p[1];
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
    } else {
      const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + row_at + e);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = elem<false>(c, j);
      v[j] = e >= d ? 0.f
             : type == MOE_FP4_TYPE_F32 ? static_cast<const float*>(base)[row_at + e]
                                        : bf16_to_f32(static_cast<const uint16_t*>(base)[row_at + e]);
    }
  }
}

template <bool VEC>
__device__ __forceinline__ void store8(void* base, int type, int64_t row_at, int c, int d, const float (&v)[8]) {
  if (VEC) {
    const int e = elem<true>(c, 0);
    if (e >= d) return;
    if (type == MOE_FP4_TYPE_F32) {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + row_at + e);
      p[0] = make_float4(v[0], v[1], v[2], v[3]);
      p[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&p);
      }
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + row_at + e) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int e = elem<false>(c, j);
      if (e >= d) continue;
      if (type == MOE_FP4_TYPE_F32)
        static_cast<float*>(base)[row_at + e] = v[j];
      else
        static_cast<uint16_t*>(base)[row_at + e] = f32_to_bf16_rn(v[j]);
    }
  }
}

// sum over the CTA, the same in every thread; `part` holds 32 floats
__device__ __forceinline__ float cta_sum(float s, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (warps == 1) return s;
  if (lane == 0) part[warp] = s;
  __syncthreads();
  float t = lane < warps ? part[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
  return t;
}

template <int NC, bool VEC>
__global__ void __launch_bounds__(512) block_norm_kernel(const NormParams P) {
  __shared__ float part[2][32];
  const moe_fp4_block_norm_args& a = P.a;
  const int64_t t = blockIdx.x;
  const int d = a.d;
  float r[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c) load8<VEC>(a.residual, a.residual_type, t * a.residual_stride, c, d, r[c]);
  if (a.y) {
    float b[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c) load8<VEC>(a.y, a.y_type, t * a.y_stride, c, d, b[c]);
    if (a.y2) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float v[8];
        load8<VEC>(a.y2, a.y2_type, t * a.y2_stride, c, d, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) b[c][j] += v[j];
      }
    }
    float m = a.scale;
    if (a.gate_shape == MOE_FP4_GATE_TOKEN) {
      const float g = a.gate_type == MOE_FP4_TYPE_F32 ? static_cast<const float*>(a.gate)[t]
                                                      : bf16_to_f32(static_cast<const uint16_t*>(a.gate)[t]);
      m *= a.gate_sigmoid ? 1.f / (1.f + __expf(-g)) : g;
    }
    if (a.post_norm) {
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) s += (P.k * b[c][j]) * (P.k * b[c][j]);
      m *= rsqrtf(cta_sum(s, part[0]) + a.eps);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) b[c][j] *= m;
      if (a.post_weight) {
        load8<VEC>(a.post_weight, a.post_weight_type, 0, c, d, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) b[c][j] *= v[j];
      }
      if (a.gate_shape >= MOE_FP4_GATE_CHANNEL) {
        load8<VEC>(a.gate, a.gate_type, a.gate_shape == MOE_FP4_GATE_ELEMENT ? t * a.gate_stride : 0, c, d, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) b[c][j] *= a.gate_sigmoid ? 1.f / (1.f + __expf(-v[j])) : v[j];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) r[c][j] += b[c][j];
    }
  }
  if (a.out) {
#pragma unroll
    for (int c = 0; c < NC; ++c) store8<VEC>(a.out, a.residual_type, t * a.out_stride, c, d, r[c]);
  }
  if (!a.normed) return;
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) s += (P.k * r[c][j]) * (P.k * r[c][j]);
  const float n = rsqrtf(cta_sum(s, part[1]) + a.eps);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[c][j] *= n;
    if (a.next_weight) {
      load8<VEC>(a.next_weight, a.next_weight_type, 0, c, d, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) r[c][j] *= v[j];
    }
    store8<VEC>(a.normed, MOE_FP4_TYPE_BF16, t * d, c, d, r[c]);
  }
}

template <bool VEC>
cudaError_t launch_norm(const NormParams& P, cudaStream_t st) {
  const int chunks = (P.a.d + 7) / 8;
  // chunks of 8 elements per thread: 1 up to 512 threads, then 2, 4
  const int nc = chunks <= 512 ? 1 : chunks <= 1024 ? 2 : 4;
  const int threads = ((chunks + nc - 1) / nc + 31) / 32 * 32;
  const unsigned grid = (unsigned)P.a.T;
  if (nc == 1)
    block_norm_kernel<1, VEC><<<grid, threads, 0, st>>>(P);
  else if (nc == 2)
    block_norm_kernel<2, VEC><<<grid, threads, 0, st>>>(P);
  else
    block_norm_kernel<4, VEC><<<grid, threads, 0, st>>>(P);
  return cudaGetLastError();
}

bool is_type(int t) { return t == MOE_FP4_TYPE_BF16 || t == MOE_FP4_TYPE_F32; }
int64_t type_size(int t) { return t == MOE_FP4_TYPE_F32 ? 4 : 2; }
// an operand of whole elements; *vec stays set if its rows start on 16 bytes
bool operand_ok(const void* p, int type, int64_t stride, int64_t rows, int d, bool* vec) {
  if (!is_type(type) || ((uintptr_t)p & (uintptr_t)(type_size(type) - 1))) return false;
  if (rows > 1 && (stride < d || stride >= (1LL << 32))) return false;
  if (((uintptr_t)p & 15) || (rows > 1 && (stride * type_size(type)) % 16)) *vec = false;
  return true;
}

}  // namespace
}  // namespace moe_fp4

extern "C" int moe_fp4_block_norm(const moe_fp4_block_norm_args* args, void* cuda_stream) {
  using namespace moe_fp4;
  if (!args) return MOE_FP4_ERR_INVALID_ARG;
  const moe_fp4_block_norm_args& a = *args;
  if (a.T < 0 || a.T >= (1LL << 31) || a.d < 1 || a.d > 16384) return MOE_FP4_ERR_INVALID_ARG;
  if (!(a.eps >= 0.f) || a.gate_shape < MOE_FP4_GATE_NONE || a.gate_shape > MOE_FP4_GATE_ELEMENT)
    return MOE_FP4_ERR_INVALID_ARG;
  if (a.T == 0) return MOE_FP4_OK;
  if (!a.residual || (!a.out && !a.normed) || (a.y && !a.out)) return MOE_FP4_ERR_INVALID_ARG;
  if (!a.y && (a.y2 || a.post_norm || a.post_weight || a.gate_shape != MOE_FP4_GATE_NONE))
    return MOE_FP4_ERR_INVALID_ARG;
  if ((a.gate_shape != MOE_FP4_GATE_NONE) != (a.gate != nullptr) || (!a.normed && a.next_weight))
    return MOE_FP4_ERR_INVALID_ARG;
  bool vec = a.d % 8 == 0;
  if (!operand_ok(a.residual, a.residual_type, a.residual_stride, a.T, a.d, &vec)) return MOE_FP4_ERR_INVALID_ARG;
  if (a.y && !operand_ok(a.y, a.y_type, a.y_stride, a.T, a.d, &vec)) return MOE_FP4_ERR_INVALID_ARG;
  if (a.y2 && !operand_ok(a.y2, a.y2_type, a.y2_stride, a.T, a.d, &vec)) return MOE_FP4_ERR_INVALID_ARG;
  if (a.post_weight && !operand_ok(a.post_weight, a.post_weight_type, a.d, 1, a.d, &vec))
    return MOE_FP4_ERR_INVALID_ARG;
  if (a.next_weight && !operand_ok(a.next_weight, a.next_weight_type, a.d, 1, a.d, &vec))
    return MOE_FP4_ERR_INVALID_ARG;
  bool any = true;  // a [T] gate is read one element a row
  if (a.gate && !operand_ok(a.gate, a.gate_type, a.gate_stride, a.gate_shape == MOE_FP4_GATE_ELEMENT ? a.T : 1, a.d,
                            a.gate_shape == MOE_FP4_GATE_TOKEN ? &any : &vec))
    return MOE_FP4_ERR_INVALID_ARG;
  if (a.out && !operand_ok(a.out, a.residual_type, a.out_stride, a.T, a.d, &vec)) return MOE_FP4_ERR_INVALID_ARG;
  if (a.normed && !operand_ok(a.normed, MOE_FP4_TYPE_BF16, a.d, a.T, a.d, &vec)) return MOE_FP4_ERR_INVALID_ARG;
  const NormParams P{a, 1.0f / sqrtf((float)a.d)};
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  return (vec ? launch_norm<true>(P, st) : launch_norm<false>(P, st)) == cudaSuccess ? MOE_FP4_OK : MOE_FP4_ERR_CUDA;
}
