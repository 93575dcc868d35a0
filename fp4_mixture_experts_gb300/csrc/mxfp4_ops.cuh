// Declarations shared by the MXFP4 operators' translation units.
#pragma once

#include <cuda_fp16.h>

#include <algorithm>

#include "moe_fp4_internal.cuh"

namespace moe_fp4 {

constexpr int kMaxGroups = 1024;
constexpr int kMaxFeatures = INT32_MAX - 255;  // a tile past them is still counted in 32 bits

// rows to quantise: row r is row (row_index ? row_index[r] / div : r) of x
struct MxRows {
  const void* x;
  int64_t x_rows, x_stride;
  const int32_t* row_index;
  const int32_t* offsets;  // groups (tiled scales): [groups + 1], or null
  int64_t rows;
  int K, div, groups;
  bool f32;
  // what every row of x starts on: 32 or 16 bytes, or 0: on an element
  int align() const {
    const uintptr_t starts = (uintptr_t)x | (uintptr_t)(x_stride * (f32 ? 4 : 2));
    return starts % 32 == 0 ? 32 : starts % 16 == 0 ? 16 : 0;
  }
};

int check_mx_rows(const MxRows& R);  // a moe_fp4_status
// for_product: a product reads the codes next (tiled ones)
cudaError_t launch_mxfp4_quantize(const MxRows& R, uint8_t* codes, uint8_t* scales, bool tiled, bool for_product,
                                  cudaStream_t st);
// The same result (tiled) for rows that are used several times: every row of x
// is quantised once, with up to once_cap of its uses, twice the mean; the others
// one by one.  lists: once_lists integers.
inline int once_cap(const MxRows& R) { return (int)std::min<int64_t>(32, 2 * ((R.rows + R.x_rows - 1) / R.x_rows)); }
inline int64_t once_lists(const MxRows& R) { return R.x_rows + 1 + R.x_rows * once_cap(R) + R.rows; }
cudaError_t launch_mxfp4_quantize_once(const MxRows& R, int32_t* lists, uint8_t* codes, uint8_t* scales,
                                       cudaStream_t st);
// E4M3 form of rows (no row_index) with a scale for 128 elements, tiled; by groups with offsets
cudaError_t launch_fp8_quantize(const MxRows& R, uint8_t* codes, uint8_t* scales, cudaStream_t st);
// the error words of the operators' kernels on the current device (one in each translation unit)
cudaError_t ops_quant_error(int32_t** word);
cudaError_t ops_mm_error(int32_t** word);
cudaError_t ops_mm1_error(int32_t** word);
cudaError_t ops_mm2_error(int32_t** word);
cudaError_t ops_norm_error(int32_t** word);
cudaError_t latent_decode_error(int32_t** word);
cudaError_t latent_attention_error(int32_t** word);
cudaError_t page_slots_error(int32_t** word);

#ifdef __CUDACC__

// launch_early with the CTAs spread evenly.  CTAs that start early all go to the
// SMs that the kernel before leaves free, and stay there (a product on 96 SMs,
// then a quantiser of 247 CTAs: 16.0 us, 12.0 launched in the ordinary way).  So
// a CTA of a grid that fills the SMs less than once asks for shared memory that
// it does not use, as much as lets only its even share of them onto an SM.
template <typename... KArgs, typename... Args>
cudaError_t launch_spread(void (*kernel)(KArgs...), unsigned grid, unsigned threads, cudaStream_t st, Args&&... args) {
  constexpr int kSmSmem = 228 * 1024, kMost = 227 * 1024, kReserved = 2048;  // of an SM, of a CTA, beside a CTA's own
  const unsigned sms = (unsigned)num_sms(), per_sm = (grid + sms - 1) / sms;
  size_t smem = 0;
  if (per_sm * threads < 2048) {
    const cudaError_t e = ensure_smem_optin(reinterpret_cast<const void*>(kernel), kMost - kReserved);
    if (e != cudaSuccess) return e;
    smem = (size_t)(per_sm == 1 ? kMost : kSmSmem / per_sm) - kReserved;
  }
  return launch_early(kernel, dim3(grid), dim3(threads), smem, st, static_cast<Args&&>(args)...);
}

// The operators' kernels are launched early, so that a chain of them pays for a
// launch while the kernel before still runs, and begin with this (every
// thread): wait until all work before has ended and is visible, then let the
// next kernel be set up.  In this order: a kernel that starts early knows that
// everything before the kernel ahead of it has ended.  What the kernel ahead
// writes is read by plain loads: the read-only ones (__ldg, ld.global.nc, what
// the compiler makes of const __restrict__) are for memory that nobody writes
// while the kernel runs, and may be moved ahead of the wait.
__device__ __forceinline__ void griddep_begin() {
  griddep_wait();
  griddep_launch_dependents();
}

// 1 / (1 + e^-g) to a few 2^-24 of the value for every g.  With t = e^-|g|, at
// most 1, it is r = 1 / (1 + t), or t r for negative g: nothing overflows.  t is 2^h (1 + l ln 2), where
// h + l is -|g| log2 e as a rounded product and what it leaves (a rounded
// argument alone makes an error that grows with |g|, 2^-18 at 80); r is the
// approximate reciprocal after one Newton step.
__device__ __forceinline__ float sigmoid(float g) {
  constexpr float kLog2e = 1.4426950408889634f, kRest = (float)(1.4426950408889634 - (double)kLog2e);
  float a, t, r;
  asm("max.NaN.f32 %0, %1, 0fC3480000;" : "=f"(a) : "f"(-fabsf(g)));  // -200: t is 0 there, and l not inf - inf
  const float h = a * kLog2e, l = fmaf(a, kRest, fmaf(a, kLog2e, -h));
  asm("ex2.approx.f32 %0, %1;" : "=f"(t) : "f"(h));
  t = fmaf(t, l * 0.6931471805599453f, t);
  const float y = 1.f + t;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
  r = fmaf(r, fmaf(-y, r, 1.f), r);
  return g < 0.f ? t * r : r;
}

// eight fp32 values -> eight E2M1 codes, element 0 in the low nibble
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// 16 consecutive elements as they are: 16 words of fp32, or 8 words of bf16
// pairs.  They start on ALIGN bytes: 32 or 16, or 0 (on an element).  With loads
// of 32 bytes a warp's requests for fp32 touch a line half as often (6667 x 2528,
// fp32: 10.0 us, 11.9 with loads of 16 bytes).
//
// kLeaving is an ALIGN of 32 bytes whose elements leave the caches first: for rows that
// are read once and whose codes a product reads next, which are then still in L2 (bf16
// rows and their product of 4096 columns, in a graph of calls: FP8 4608 x 4096 59.6 -> 57.3
// us, 2048 x 7168 49.8 -> 48.1, no slower for fewer; MXFP4 from 32 MB of rows on, 4608 x
// 7168 60 -> 57, 2600 x 7168 38.5 -> 38.2, but 2048 x 7168 27.5 -> 27.9).  What is read
// again must not: rows quantised by themselves in a loop (4608 x 4096 6.8 -> 8.2 us),
// gathered ones, which are read once for each use (2048 rows, 8 uses, cold caches 25 ->
// 29), and the few rows that all CTAs of their kernel read (16 x 16384 by 2048, cold
// caches 25 -> 27).
constexpr int kLeaving = 33;
template <bool F32, int ALIGN>
__device__ __forceinline__ void load16_raw(const void* x, int64_t at, uint32_t (&w)[16]) {
#define MOE_LOAD32(form)                                                                                        \
  asm volatile("ld.global" form ".v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"                               \
               : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3]), "=r"(w[i + 4]), "=r"(w[i + 5]),    \
                 "=r"(w[i + 6]), "=r"(w[i + 7])                                                                 \
               : "l"(p + 4 * i))
  if (ALIGN == 32 || ALIGN == kLeaving) {
    const char* p = static_cast<const char*>(x) + at * (F32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < (F32 ? 16 : 8); i += 8)
      if (ALIGN == kLeaving)
        MOE_LOAD32(".L1::no_allocate.L2::evict_first");
      else
        MOE_LOAD32("");
#undef MOE_LOAD32
  } else if (ALIGN == 16) {
    const uint4* p = F32 ? reinterpret_cast<const uint4*>(static_cast<const float*>(x) + at)
                         : reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at);
#pragma unroll
    for (int i = 0; i < (F32 ? 4 : 2); ++i) {
      const uint4 q = p[i];
      w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
    }
  } else if (F32) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = static_cast<const uint32_t*>(x)[at + i];
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(x) + at;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = (uint32_t)p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
  }
}

// The codes of half a block, 16 elements as load16_raw leaves them, by a pair of
// lanes (l, l ^ 1) that hold a block together (whole warp; every lane takes
// part), and the block's scale byte.  bf16 elements stay in pairs up to the
// conversion: magnitudes compare as their bit patterns do, and x 2^-e is exact
// in bf16 too (an underflow ends at the code 0 with its sign all the same).
template <bool F32>
__device__ __forceinline__ uint2 quantize16(const uint32_t (&w)[16], uint32_t& scale) {
  uint32_t amax;  // bits of the largest magnitude as fp32
  if (F32) {
    amax = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) amax = max(amax, w[j] & 0x7FFFFFFFu);
    amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = __vmaxu2(m, w[j] & 0x7FFF7FFFu);
    m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    amax = max(m << 16, m & 0xFFFF0000u);
  }
  const uint32_t ef = amax >> 23;
  scale = ef == 255u ? 255u : (ef > 2u ? ef - 2u : 0u);
  if (scale == 255u) return make_uint2(0x77777777u, 0x77777777u);
  float v[16];
  if (F32) {
    const float inv = __uint_as_float((254u - scale) << 23);  // 2^(127 - scale), normal for scale in [0, 253]
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(w[j]) * inv;
  } else {
    const uint32_t inv = ((254u - scale) << 7) * 0x10001u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t p;
      asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(p) : "r"(w[j]), "r"(inv));
      v[2 * j] = __uint_as_float(p << 16);
      v[2 * j + 1] = __uint_as_float(p & 0xFFFF0000u);
    }
  }
  return make_uint2(e2m1x8(v), e2m1x8(v + 8));
}

// four fp32 values, in [-448, 448], -> four E4M3 codes, to nearest even
__device__ __forceinline__ uint32_t e4m3x4(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]));
  return r;
}

// The E4M3 codes of 16 elements as load16_raw leaves them, by eight lanes (8 i ..
// 8 i + 7) that hold a block of 128 together (whole warp; every lane takes part),
// and the block's scale byte: e + 127 with the least e >= -127 for which amax <= 448
// 2^e.  448 is 1.75 2^8, so e is the exponent of amax minus 8, and one more for
// mantissas above 1.75.  x 2^-e is exact but where it underflows to the code 0.
template <bool F32>
__device__ __forceinline__ uint4 quantize16_fp8(const uint32_t (&w)[16], uint32_t& scale) {
  uint32_t amax = 0;  // bits of the largest magnitude as fp32
  if (F32) {
#pragma unroll
    for (int j = 0; j < 16; ++j) amax = max(amax, w[j] & 0x7FFFFFFFu);
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = __vmaxu2(m, w[j] & 0x7FFF7FFFu);
    amax = max(m << 16, m & 0xFFFF0000u);
  }
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, d));
  const uint32_t ef = (amax >> 23) + ((amax & 0x7FFFFFu) > 0x600000u ? 1u : 0u);
  scale = amax >= 0x7F800000u ? 255u : (ef > 8u ? ef - 8u : 0u);
  if (scale == 255u) return make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
  const float inv = __uint_as_float((254u - scale) << 23);  // 2^(127 - scale), normal for scale in [0, 247]
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = (F32 ? __uint_as_float(w[4 * i + j])
                  : __uint_as_float(j & 1 ? w[2 * i + j / 2] & 0xFFFF0000u : w[2 * i + j / 2] << 16)) * inv;
    q[i] = e4m3x4(v);
  }
  return make_uint4(q[0], q[1], q[2], q[3]);
}

// The group that holds row r: the last e with off[e] <= r, if r < off[e + 1];
// -1 if none does.  Offsets are taken as they are; a row is given a group only
// if the group lies in [0, rows], so that tile indices stay in their range.
__device__ __forceinline__ int find_group(const int32_t* off, int groups, int64_t r, int64_t rows) {
  int lo = 0, hi = groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= r)
      lo = mid;
    else
      hi = mid;
  }
  const int64_t first = off[lo], end = off[lo + 1];
  return first >= 0 && first <= r && r < end && end <= rows ? lo : -1;
}

// The same by a whole warp, in one round of loads for each 32 groups; *first is
// the group's first row.
__device__ __forceinline__ int find_group_warp(const int32_t* off, int groups, int r, int rows, int* first) {
  const int lane = threadIdx.x & 31;
  int below = 0;  // groups that begin at or before r
  for (int e0 = 0; e0 < groups; e0 += 32) {
    const int e = e0 + lane;
    below += __popc(__ballot_sync(0xFFFFFFFFu, e < groups && off[min(e, groups)] <= r));
  }
  if (below == 0) return -1;
  const int b = off[below - 1], end = off[below];
  *first = b;
  return b >= 0 && b <= r && r < end && end <= rows ? below - 1 : -1;
}

#endif

}  // namespace moe_fp4
