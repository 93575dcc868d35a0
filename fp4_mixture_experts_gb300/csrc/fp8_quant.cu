// E4M3 form of rows with one power-of-two scale for 128 elements, and the scale
// layout of weights that have one for 128 x 128.
//
// Per 128 elements of a row e is the least integer with amax <= 448 2^e (at least
// -127), the scale byte e + 127 and an element's code the E4M3 value nearest to x
// 2^-e (ties to even).  Eight lanes share a block, 16 elements each: loads of 32 or
// 16 bytes, three shuffles for amax, one 16-byte store of codes.  The products'
// scale tiles hold a byte for 32 elements: the same one four times, one word.
// Its instructions and HBM bound it side by side: 8192 x 8192 bf16 27 us in one launch
// with cold caches, 134 MB read at 5.0 TB/s (69% of DRAM's peak) and 0.72 instructions a
// cycle of a scheduler; 8192 x 4096 16 us, 55% and 0.68.  The codes stay in L2 for the
// product (12 of 67 MB are written meanwhile).
#include <algorithm>

#include "moe_fp4_internal.cuh"
#include "mxfp4_ops.cuh"

namespace moe_fp4 {
namespace {

constexpr int kPer = 16;  // elements of a thread
constexpr int kThreads = 256;

struct Fp8QuantParams {
  const void* x;
  int64_t x_stride;
  const int32_t* offsets;
  uint8_t* codes;
  uint8_t* scales;
  int64_t rows;
  int K, groups;
  int lanes_log;  // log2 of the lanes a row's segment has: 3 .. 5
  int segments;   // segments a row
};

// 8, 16 or 32 lanes a segment of a row, two chunks of 16 elements each, so that
// short rows share a warp and long ones have several.
template <bool F32, int ALIGN>
__global__ void __launch_bounds__(kThreads) fp8_quantize_kernel(const Fp8QuantParams P) {
  griddep_begin();
  const int per_row = P.K / kPer, kt = (P.K + 127) / 128;
  const int lanes = 1 << P.lanes_log;
  const int64_t seg = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> P.lanes_log;
  const int64_t r0 = seg / P.segments;
  const bool in = r0 < P.rows;  // lanes past the end stay for the shuffles
  const int r = in ? (int)r0 : 0;
  const int c0 = (int)(seg - r0 * P.segments) * 2 * lanes + (threadIdx.x & (lanes - 1));
  uint32_t w[2][kPer];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) w[u][j] = 0;
    if (in && c0 + u * lanes < per_row)
      load16_raw<F32, ALIGN>(P.x, r * P.x_stride + (int64_t)(c0 + u * lanes) * kPer, w[u]);
  }
  // the row's place in the tiles, while the loads are on their way
  int tile = r >> 7, row = r & 127;
  bool grouped = true;
  if (P.offsets) {
    const int e = find_group(P.offsets, P.groups, r, P.rows);
    grouped = e >= 0;
    if (grouped) {
      const int first = P.offsets[e];
      tile = (first >> 7) + e + ((r - first) >> 7);
      row = (r - first) & 127;
    }
  }
  uint8_t* const t = P.scales + (size_t)tile * kt * 512 + 16 * (row & 31) + 4 * (row >> 5);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int c = c0 + u * lanes;
    uint32_t sb;
    const uint4 q = quantize16_fp8<F32>(w[u], sb);
    if (!in || c >= per_row) continue;
    *reinterpret_cast<uint4*>(P.codes + (size_t)r * P.K + c * kPer) = q;
    if ((c & 7) == 0 && grouped) *reinterpret_cast<uint32_t*>(t + (c >> 3) * 512) = sb * 0x01010101u;
  }
}

// (every row is read once, and a product reads the codes next)
template <bool F32>
cudaError_t launch_quant(const Fp8QuantParams& P, int align, cudaStream_t st) {
  const int64_t threads = (P.rows * P.segments) << P.lanes_log;
  auto* k = align == 32   ? fp8_quantize_kernel<F32, kLeaving>
            : align == 16 ? fp8_quantize_kernel<F32, 16>
                          : fp8_quantize_kernel<F32, 0>;
  return launch_spread(k, (unsigned)((threads + kThreads - 1) / kThreads), kThreads, st, P);
}

// one thread: a row's scale of one tile, one word
__global__ void __launch_bounds__(kThreads)
fp8_tile_scales_kernel(const uint8_t* scales, int N, int rt, int kt, int swiglu, int64_t words, uint32_t* tiled) {
  griddep_begin();
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < words; i += (int64_t)gridDim.x * kThreads) {
    const int w = (int)(i & 127);  // word of the tile: row (w % 4) * 32 + w / 4
    const int64_t t = i >> 7;
    const int k = (int)(t % kt);
    const int64_t er = t / kt, e = er / rt;
    const int row = (int)(er % rt) * 128 + (w & 3) * 32 + (w >> 2);
    uint32_t v = 0;
    if (row < N) {
      const int src = swiglu ? (row & 1) * (N / 2) + (row >> 1) : row;
      v = scales[(e * rt + (src >> 7)) * kt + k] * 0x01010101u;
    }
    tiled[i] = v;
  }
}

}  // namespace

cudaError_t launch_fp8_quantize(const MxRows& R, uint8_t* codes, uint8_t* scales, cudaStream_t st) {
  Fp8QuantParams P{R.x, R.x_stride, R.offsets, codes, scales, R.rows, R.K, R.groups, 5, 1};
  const int chunks = R.K / kPer;
  while (P.lanes_log > 3 && (1 << P.lanes_log) >= chunks) --P.lanes_log;  // half the lanes, two chunks each, do
  P.segments = (chunks + (2 << P.lanes_log) - 1) >> (P.lanes_log + 1);
  return R.f32 ? launch_quant<true>(P, R.align(), st) : launch_quant<false>(P, R.align(), st);
}

}  // namespace moe_fp4

using namespace moe_fp4;

extern "C" int moe_fp4_fp8_tile_scales(const uint8_t* scales, int32_t E, int32_t N, int32_t K, int swiglu, uint8_t* tiled,
                                       void* cuda_stream) {
  if (!scales || !tiled || ((uintptr_t)tiled & 15) || E < 1 || E > kMaxGroups || N < 1 || N > kMaxFeatures || K <= 0 ||
      K % 32 != 0 || K > 32768 || (swiglu && N % 2 != 0))
    return MOE_FP4_ERR_INVALID_ARG;
  const int rt = (N + 127) / 128, kt = (K + 127) / 128;
  const int64_t words = (int64_t)E * rt * kt * 128;
  const int64_t blocks = std::min<int64_t>((words + kThreads - 1) / kThreads, 16LL * num_sms());
  return launch_spread(fp8_tile_scales_kernel, (unsigned)blocks, kThreads, static_cast<cudaStream_t>(cuda_stream), scales,
                       N, rt, kt, swiglu, words, reinterpret_cast<uint32_t*>(tiled)) == cudaSuccess
             ? MOE_FP4_OK
             : MOE_FP4_ERR_CUDA;
}
