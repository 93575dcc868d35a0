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
#include <algorithm>
#include <mutex>

#include "moe_fp4_internal.cuh"
#include "mxfp4_ops.cuh"

namespace moe_fp4 {
namespace {

__device__ int32_t g_quant_err[4];

constexpr int kPer = 16;  // elements per thread
constexpr int kThreads = 256;
constexpr int kDequantRuns = 4;

struct QuantParams {
  const void* x;
  int64_t x_rows, x_stride;
  const int32_t* row_index;
  const int32_t* offsets;
  uint8_t* codes;
  uint8_t* scales;
  int64_t rows;
  int K, div, groups;
  int segments;  // warps a row (mxfp4_quantize_rows_kernel)
};

// The first byte of the tile word of (row, block 0) for a row r of the output,
// null if the row is in no group; whole warp.
__device__ __forceinline__ uint8_t* tile_row(const QuantParams& P, int r, int kt) {
  int tile = r >> 7, row = r & 127;
  if (P.offsets) {
    int first;
    const int e = find_group_warp(P.offsets, P.groups, r, (int)P.rows, &first);
    if (e < 0) return nullptr;
    tile = (first >> 7) + e + ((r - first) >> 7);
    row = (r - first) & 127;
  }
  return P.scales + (size_t)tile * kt * 512 + 16 * (row & 31) + 4 * (row >> 5);
}

// The source row of output row r, -1 for an index out of range.
__device__ __forceinline__ int source_row(const QuantParams& P, int r) {
  if (!P.row_index) return r;
  int s = P.row_index[r];
  s = s < 0 ? -1 : s / P.div;
  return s < P.x_rows ? s : -1;
}

// Many rows: a warp a row, or every segments-th 1024 elements of one, with what
// belongs to the row (its source, its place in the tiles) looked up once.  Flat
// over the elements instead, with a division and a group search in every thread,
// gathering 36,864 rows of 2048 took 63 us (25 so).  65536 x 4096: 96 us, the rate
// of a copy; tiled on a grid that fills the SMs and strides, 109.
template <bool F32, int ALIGN, bool TILED>
__global__ void __launch_bounds__(kThreads) mxfp4_quantize_rows_kernel(const QuantParams P) {
  griddep_begin();
  const int per_row = P.K / kPer, nb = P.K / 32, kt = (P.K + 127) / 128;
  const int lane = threadIdx.x & 31;
  int r = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), c1 = 0;  // this warp's row, and its first chunk
  if (P.segments > 1) {
    const uint32_t id = r;
    r = id / P.segments;
    c1 = 64 * (id - r * P.segments);
  }
  if (r >= (int)P.rows) return;
  const int src = source_row(P, r);
  if (src < 0 && lane == 0) atomicOr(&g_quant_err[0], kErrBadExpertId);
  const int64_t at = src * P.x_stride;
  uint32_t w[2][kPer];
  auto load = [&](int c0) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int j = 0; j < kPer; ++j) w[u][j] = 0;
      if (src >= 0 && c0 + 32 * u < per_row) load16_raw<F32, ALIGN>(P.x, at + (c0 + 32 * u) * kPer, w[u]);
    }
  };
  load(c1 + lane);
  uint8_t* const tile = TILED ? tile_row(P, r, kt) : nullptr;  // while the loads are on their way
  uint8_t* const codes = P.codes + (size_t)r * (P.K / 2);
  for (int c0 = c1 + lane;;) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int c = c0 + 32 * u, b = c >> 1;
      uint32_t sb;
      const uint2 q = quantize16<F32>(w[u], sb);
      if (TILED) {  // a word of four scales in every eighth lane, 0 past the end of K
        sb <<= 8 * (b & 3);
        sb |= __shfl_xor_sync(0xFFFFFFFFu, sb, 2);
        sb |= __shfl_xor_sync(0xFFFFFFFFu, sb, 4);
      }
      if (c >= per_row) continue;
      *reinterpret_cast<uint2*>(codes + c * (kPer / 2)) = q;
      if (!TILED) {
        if ((c & 1) == 0) P.scales[(size_t)r * nb + b] = (uint8_t)sb;
      } else if ((c & 7) == 0 && tile != nullptr) {
        *reinterpret_cast<uint32_t*>(tile + (b >> 2) * 512) = sb;
      }
    }
    c0 += 64 * P.segments;
    if (c0 - lane >= per_row) break;
    load(c0);
  }
}

// Few or short rows: flat over the chunks of 16 elements
template <bool F32, int ALIGN, bool TILED>
__global__ void __launch_bounds__(kThreads) mxfp4_quantize_flat_kernel(const QuantParams P) {
  griddep_begin();
  const int per_row = P.K / kPer, nb = P.K / 32, kt = (P.K + 127) / 128;
  const uint32_t total = (uint32_t)P.rows * per_row;  // rows K < 2^35
  // whole warps leave the loop together (the shuffle needs both lanes of a block)
  for (uint32_t i0 = blockIdx.x * kThreads + (threadIdx.x & ~31); i0 < total; i0 += gridDim.x * kThreads) {
    const uint32_t i = i0 + (threadIdx.x & 31);
    const bool in = i < total;
    const int r = in ? i / per_row : 0, c = in ? i - r * per_row : 0;
    uint32_t w[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) w[j] = 0;
    const int src = source_row(P, r);
    if (src < 0)
      atomicOr(&g_quant_err[0], kErrBadExpertId);
    else if (in)
      load16_raw<F32, ALIGN>(P.x, src * P.x_stride + (int64_t)c * kPer, w);
    uint32_t sb;
    const uint2 q = quantize16<F32>(w, sb);
    if (!in) continue;
    *reinterpret_cast<uint2*>(P.codes + (size_t)r * (P.K / 2) + c * (kPer / 2)) = q;
    if (c & 1) continue;
    const int b = c >> 1;
    if (!TILED) {
      P.scales[(size_t)r * nb + b] = (uint8_t)sb;
    } else {
      int tile = r >> 7, row = r & 127;
      if (P.offsets) {
        const int e = find_group(P.offsets, P.groups, r, P.rows);
        if (e < 0) continue;
        const int first = P.offsets[e];
        tile = (first >> 7) + e + ((r - first) >> 7);
        row = (r - first) & 127;
      }
      uint8_t* t = P.scales + ((size_t)tile * kt + (b >> 2)) * 512 + 16 * (row & 31) + 4 * (row >> 5);
      t[b & 3] = (uint8_t)sb;
      if (b == nb - 1)
        for (int p = (b & 3) + 1; p < 4; ++p) t[p] = 0;
    }
  }
}

// ---- rows used several times ----
// The expert sort uses every token k times.  Quantising each output row does
// the arithmetic k times, and that bounds it; so the places of a source row are
// gathered first, and a warp a source row quantises it once and writes it to all
// of them (36,864 rows of 2048 from 4608, with a product of 64 features behind:
// 32.1 -> 23.5 us).
// A source row's table has room for twice the mean number of uses (up to 32, a
// lane each); places beyond it, and those whose index is out of range, which get
// zeros, go to one list that all warps share out, a row each: however uneven the
// uses are, no warp writes more than a few rows.  (Half of the 36,864 places
// naming one row: 35 us, and 7,160 where a row's own warp writes all of its
// places, one after the other.  Rows drawn at random: 25.0 us.)
// counts[s], s < x_rows: the uses of row s; counts[x_rows]: places on the shared
// list.  Which places are on it depends on the atomics' order, what is written
// does not.
struct Places {
  int32_t* counts;  // [x_rows + 1]
  int32_t* table;   // [x_rows][cap]
  int32_t* shared;  // [rows]
  int cap;
};

__global__ void __launch_bounds__(kThreads) places_init_kernel(int32_t* counts, int n) {
  griddep_begin();
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i < n) counts[i] = 0;
}

__global__ void __launch_bounds__(kThreads) places_gather_kernel(const QuantParams P, const Places L) {
  griddep_begin();
  const int r = blockIdx.x * kThreads + threadIdx.x, lane = threadIdx.x & 31;
  const uint32_t in = __ballot_sync(0xFFFFFFFFu, r < (int)P.rows);
  if (r >= (int)P.rows) return;
  const int s = source_row(P, r);
  if (s < 0) atomicOr(&g_quant_err[0], kErrBadExpertId);
  // one addition for the lanes that name the same row: many uses of one row are one address
  const uint32_t below = (1u << lane) - 1, same = __match_any_sync(in, s);
  const int first = __ffs(same) - 1;
  int at = 0;
  if (s >= 0 && lane == first) at = atomicAdd(&L.counts[s], __popc(same));
  at = __shfl_sync(in, at, first) + __popc(same & below);
  const bool over = s < 0 || at >= L.cap;
  if (!over) L.table[(int64_t)s * L.cap + at] = r;
  const uint32_t rest = __ballot_sync(in, over);
  if (!over) return;
  const int leader = __ffs(rest) - 1;
  if (lane == leader) at = atomicAdd(&L.counts[P.x_rows], __popc(rest));
  L.shared[__shfl_sync(rest, at, leader) + __popc(rest & below)] = r;
}

template <bool F32, int ALIGN>
__global__ void __launch_bounds__(kThreads) mxfp4_quantize_places_kernel(const QuantParams P, const Places L) {
  griddep_begin();
  const int per_row = P.K / kPer, kt = (P.K + 127) / 128;
  const int lane = threadIdx.x & 31, warp = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
  const int listed = L.counts[P.x_rows];
  // the warp's source row, then its share of the list
  for (int64_t i = warp - warps; i < listed; i += warps) {
    int s, n = 1, mine = 0;  // source row, its places here, this lane's place
    if (i < 0) {
      if (warp >= (int)P.x_rows) continue;
      s = warp;
      n = min(L.counts[s], L.cap);
      if (lane < n) mine = L.table[(int64_t)s * L.cap + lane];
      if (n == 0) continue;
    } else {
      mine = L.shared[i];
      s = source_row(P, mine);
    }
    int tile = mine >> 7, row = mine & 127;
    bool in_group = true;
    if (P.offsets) {
      const int e = find_group(P.offsets, P.groups, mine, P.rows);
      in_group = e >= 0;
      const int first = in_group ? P.offsets[e] : 0;
      tile = (first >> 7) + e + ((mine - first) >> 7);
      row = (mine - first) & 127;
    }
    const int64_t at = in_group ? (int64_t)tile * kt * 512 + 16 * (row & 31) + 4 * (row >> 5) : -1;
    for (int c0 = lane; c0 - lane < per_row; c0 += 64) {
      uint32_t w[2][kPer];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) w[u][j] = 0;
        if (s >= 0 && c0 + 32 * u < per_row)
          load16_raw<F32, ALIGN>(P.x, s * P.x_stride + (c0 + 32 * u) * kPer, w[u]);
      }
      uint2 q[2];
      uint32_t sw[2];  // in every eighth lane, the word of four scales
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        q[u] = quantize16<F32>(w[u], sw[u]);
        sw[u] <<= 8 * ((lane >> 1) & 3);
        sw[u] |= __shfl_xor_sync(0xFFFFFFFFu, sw[u], 2);
        sw[u] |= __shfl_xor_sync(0xFFFFFFFFu, sw[u], 4);
      }
      for (int i = 0; i < n; ++i) {
        uint8_t* const codes = P.codes + (size_t)__shfl_sync(0xFFFFFFFFu, mine, i) * (P.K / 2);
        const int64_t t = __shfl_sync(0xFFFFFFFFu, at, i);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int c = c0 + 32 * u;
          if (c >= per_row) continue;
          *reinterpret_cast<uint2*>(codes + c * (kPer / 2)) = q[u];
          if (t >= 0 && (lane & 7) == 0) *reinterpret_cast<uint32_t*>(P.scales + t + (c >> 3) * 512) = sw[u];
        }
      }
    }
  }
}

template <bool F32>
__global__ void __launch_bounds__(kThreads)
mxfp4_dequantize_kernel(const uint8_t* codes, const uint8_t* scales, int64_t total, void* out) {
  griddep_begin();
  // One thread: 8 elements, 4 bytes of codes, at kDequantRuns places loaded
  // together, in adjacent runs of the CTA; a CTA for each 8192 elements.  (65536
  // x 4096: 99 us, the rate of a copy; 111 with one place a thread on a grid that
  // fills the SMs, 119 with these four on that grid.)
  constexpr int kU = kDequantRuns;
  const int64_t i0 = (int64_t)blockIdx.x * kU * kThreads + threadIdx.x;
  uint32_t c[kU];
  float s[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t i = min(i0 + u * kThreads, total - 1);
    c[u] = reinterpret_cast<const uint32_t*>(codes)[i];
    s[u] = e8m0_to_f32(scales[i >> 2]);
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t i = i0 + u * kThreads;
    if (i >= total) break;
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t h = e2m1x2_to_f16x2((c[u] >> (8 * j)) & 0xFFu);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      v[2 * j] = f.x * s[u];
      v[2 * j + 1] = f.y * s[u];
    }
    if (F32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + 8 * i);
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t*>(&p);
      }
      reinterpret_cast<uint4*>(out)[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// one thread: the four scales of one row and tile, one word
__global__ void __launch_bounds__(kThreads)
tile_scales_kernel(const uint8_t* scales, int N, int nb, int rt, int kt, int swiglu, int64_t words, uint32_t* tiled) {
  griddep_begin();
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

// The error words of all the operators, taken: each read and cleared in one
// step, so that an error which another stream raises meanwhile is in this check or
// in the next.
constexpr int kErrorWords = 5;
struct ErrorWords {
  int32_t* word[kErrorWords];
};
__device__ int32_t g_taken_err;
__global__ void take_errors_kernel(const ErrorWords w) {
  int32_t bits = 0;
  for (int i = 0; i < kErrorWords; ++i) bits |= atomicExch(w.word[i], 0);
  g_taken_err = bits;
}

int grid_for(int64_t threads, int per_sm) {
  const int64_t blocks = (threads + kThreads - 1) / kThreads, cap = (int64_t)num_sms() * per_sm;
  return (int)(blocks < cap ? blocks : cap);
}

}  // namespace

namespace {

template <bool F32, int ALIGN, bool TILED>
cudaError_t launch_quant(const QuantParams& P, cudaStream_t st) {
  // a warp a row where that fills the SMs (8 rows each at least) and most lanes
  if (P.K >= 512 && P.rows >= 8 * num_sms()) {
    // Rows as they lie: a warp every 1024 elements (2000 x 16384, fp32: 23 us, 34 with a warp a row; 8192 x 4096,
    // bf16: 13.2 and 15.2).  Gathered or grouped ones: up to 64 warps an SM, as each looks its row up (36864 rows of
    // 2048: 26 us with a warp a row, 33 with two; 4000 of 7168: 11.0 with three, 12.1 and 12.8 with one and seven).
    QuantParams Q = P;
    const int64_t steps = (P.K + 64 * kPer - 1) / (64 * kPer);
    Q.segments = (int)(P.row_index || P.offsets ? std::min(steps, (64 * num_sms() + P.rows - 1) / P.rows) : steps);
    return launch_spread(mxfp4_quantize_rows_kernel<F32, ALIGN, TILED>, (unsigned)((P.rows * Q.segments + 7) / 8), kThreads, st, Q);
  }
  return launch_spread(mxfp4_quantize_flat_kernel<F32, ALIGN, TILED>, (unsigned)grid_for(P.rows * (P.K / kPer), 8),
                       kThreads, st, P);
}

template <bool F32, int ALIGN>
cudaError_t launch_quant(const QuantParams& P, bool tiled, cudaStream_t st) {
  return tiled ? launch_quant<F32, ALIGN, true>(P, st) : launch_quant<F32, ALIGN, false>(P, st);
}

template <bool F32>
cudaError_t launch_quant(const QuantParams& P, int align, bool tiled, cudaStream_t st) {
  return align == 32   ? launch_quant<F32, 32>(P, tiled, st)
         : align == 16 ? launch_quant<F32, 16>(P, tiled, st)
                       : launch_quant<F32, 0>(P, tiled, st);
}

}  // namespace

cudaError_t launch_mxfp4_quantize(const MxRows& R, uint8_t* codes, uint8_t* scales, bool tiled, cudaStream_t st) {
  const QuantParams P{R.x, R.x_rows, R.x_stride, R.row_index, R.offsets, codes, scales, R.rows, R.K, R.div, R.groups};
  return R.f32 ? launch_quant<true>(P, R.align(), tiled, st) : launch_quant<false>(P, R.align(), tiled, st);
}

cudaError_t launch_mxfp4_quantize_once(const MxRows& R, int32_t* lists, uint8_t* codes, uint8_t* scales,
                                       cudaStream_t st) {
  const QuantParams P{R.x, R.x_rows, R.x_stride, R.row_index, R.offsets, codes, scales, R.rows, R.K, R.div, R.groups};
  Places L;
  L.cap = once_cap(R);
  L.counts = lists;
  L.table = L.counts + R.x_rows + 1;
  L.shared = L.table + R.x_rows * L.cap;
  const auto blocks = [](int64_t threads) { return (unsigned)((threads + kThreads - 1) / kThreads); };
  cudaError_t e = launch_spread(places_init_kernel, blocks(R.x_rows + 1), kThreads, st, L.counts, (int)R.x_rows + 1);
  if (e == cudaSuccess) e = launch_spread(places_gather_kernel, blocks(R.rows), kThreads, st, P, L);
  if (e != cudaSuccess) return e;
  const int al = R.align();
  auto* k = R.f32 ? (al == 32   ? mxfp4_quantize_places_kernel<true, 32>
                     : al == 16 ? mxfp4_quantize_places_kernel<true, 16>
                                : mxfp4_quantize_places_kernel<true, 0>)
                  : (al == 32   ? mxfp4_quantize_places_kernel<false, 32>
                     : al == 16 ? mxfp4_quantize_places_kernel<false, 16>
                                : mxfp4_quantize_places_kernel<false, 0>);
  // a warp a source row, and enough of them to share the list out
  const int64_t warps = std::max(R.x_rows, std::min<int64_t>(R.rows, 16 * num_sms()));
  return launch_spread(k, blocks(warps * 32), kThreads, st, P, L);
}

cudaError_t ops_quant_error(int32_t** word) { return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_quant_err); }

int check_mx_rows(const MxRows& R) {
  if (R.K <= 0 || R.K % 32 != 0 || R.K > 32768 || R.rows < 0 || R.x_rows < 0 || R.div < 1) return MOE_FP4_ERR_INVALID_ARG;
  if (R.rows >= (1LL << 31) || R.rows * R.K >= (1LL << 35)) return MOE_FP4_ERR_INVALID_ARG;
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
  if (rows < 0 || K <= 0 || K % 32 != 0 || K > 32768 || rows >= (1LL << 31) || rows * K >= (1LL << 35))
    return MOE_FP4_ERR_INVALID_ARG;
  if (out_type != MOE_FP4_TYPE_BF16 && out_type != MOE_FP4_TYPE_F32) return MOE_FP4_ERR_INVALID_ARG;
  if (rows == 0) return MOE_FP4_OK;
  if (!codes || !scales || !out || ((uintptr_t)codes & 15) || ((uintptr_t)out & 15)) return MOE_FP4_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const int64_t total = rows * (K / 8);
  const unsigned grid = (unsigned)((total + kDequantRuns * kThreads - 1) / (kDequantRuns * kThreads));
  return launch_spread(out_type == MOE_FP4_TYPE_F32 ? mxfp4_dequantize_kernel<true> : mxfp4_dequantize_kernel<false>,
                       grid, kThreads, st, codes, scales, total, out) == cudaSuccess
             ? MOE_FP4_OK
             : MOE_FP4_ERR_CUDA;
}

int moe_fp4_mxfp4_tile_scales(const uint8_t* scales, int32_t E, int32_t N, int32_t K, int swiglu, uint8_t* tiled,
                              void* cuda_stream) {
  if (!scales || !tiled || ((uintptr_t)tiled & 15) || E < 1 || E > kMaxGroups || N < 1 || N > kMaxFeatures || K <= 0 || K % 32 != 0 ||
      K > 32768 || (swiglu && N % 2 != 0))
    return MOE_FP4_ERR_INVALID_ARG;
  const int rt = (N + 127) / 128, kt = (K + 127) / 128;
  const int64_t words = (int64_t)E * rt * kt * 128;
  return launch_spread(tile_scales_kernel, (unsigned)grid_for(words, 16), kThreads,
                       static_cast<cudaStream_t>(cuda_stream), scales, N, K / 32, rt, kt, swiglu, words,
                       reinterpret_cast<uint32_t*>(tiled)) == cudaSuccess
             ? MOE_FP4_OK
             : MOE_FP4_ERR_CUDA;
}

int moe_fp4_ops_check(void* cuda_stream) {
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  ErrorWords words;
  cudaError_t (*const address[])(int32_t**) = {ops_quant_error, ops_mm_error, ops_mm1_error, ops_mm2_error, ops_norm_error};
  for (int i = 0; i < kErrorWords; ++i)
    if (address[i](&words.word[i]) != cudaSuccess) return MOE_FP4_ERR_CUDA;
  static std::mutex one_check;  // g_taken_err is one word
  const std::lock_guard<std::mutex> lock(one_check);
  take_errors_kernel<<<1, 1, 0, st>>>(words);
  int32_t bits = 0;
  if (cudaGetLastError() != cudaSuccess ||
      cudaMemcpyFromSymbolAsync(&bits, g_taken_err, sizeof(bits), 0, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return MOE_FP4_ERR_CUDA;
  return bits == 0 ? MOE_FP4_OK : MOE_FP4_ERR_DEVICE;
}

}  // extern "C"
