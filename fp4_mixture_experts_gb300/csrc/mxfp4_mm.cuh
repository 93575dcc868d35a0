// Pieces shared by the MXFP4 product kernels (one CTA per tile, and CTA
// pairs): parameters, group tables, the block-scaled MMA's wrappers and the
// epilogue.
#pragma once

#include <cuda.h>

#include "moe_fp4_internal.cuh"
#include "mxfp4_ops.cuh"
#include "ptx_sm103.cuh"
#include "tc_helpers.cuh"

namespace moe_fp4 {
namespace mm {

constexpr int kBM = 128;        // weight rows of a CTA's tile
constexpr int kStageK = 256;    // K elements per stage: 128 bytes of codes a row
constexpr int kSfTile = 512;    // bytes of one scale tile: 128 rows x 4 scales (K = 128)
constexpr uint32_t kTmemCols = 512;
constexpr int kSmemMax = 227 * 1024;

struct MmParams {
  const uint8_t* a_scales;   // tiled, grouped
  const uint8_t* w_scales;   // [E][mblocks][kt][512]
  const int32_t* offsets;    // [E + 1] or null
  void* y;
  int32_t* err;
  int M, N, K, E;
  int n_out;                 // features of y
  int mblocks;               // ceil(N / 128)
  int kt;                    // scale tiles along K
  int f32, swiglu;
  int vec;                   // rows of y start on 16 bytes
  int split;                 // CTAs of a cluster that share an item's K (1: none)
  int early;                 // launched before the kernel that writes the rows has ended
  uint64_t wait_ns;
};

// Values that are the same in all lanes, in a form that lets the compiler know
// it: a role's loops then run in uniform control flow and its tensor-core and
// TMA operands in uniform registers.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }
__device__ __forceinline__ int warp_index() { return uniform((int)(threadIdx.x >> 5)); }

// true in one lane of the (converged) warp.  The tensor-core and TMA
// instructions take their operands from uniform registers: issued under this
// predicate they need no loop over possibly active lanes, which a branch on
// the lane index costs (one-token product, K = 4096: 12.4 us with the branch,
// 8.6 us so).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// bytes (a multiple of 16) from global to shared memory, both 16-byte aligned
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

template <int CTAS>
__device__ __forceinline__ void umma_mxf4(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                          uint32_t sfb, uint32_t acc) {
  if (CTAS == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(
            d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(
            d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}

// Instruction descriptor of kind::mxf4: A and B E2M1 (1), E8M0 scales; `half`:
// which two bytes of the scale words the K = 64 of this instruction uses.
__device__ __forceinline__ uint32_t idesc_mxf4(int M, int N, uint32_t half) {
  return ((2 * half) << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
         ((uint32_t)(M >> 4) << 24) | ((2 * half) << 29);
}

// Shared-memory descriptors as two words: the high one is fixed by the layout,
// the low one holds the address in units of 16 bytes, so that a step of 32
// bytes is one addition of 2.  (Built whole for every instruction, they cost
// the issuing warp more than the tensor core needs for the MMAs.)
constexpr uint32_t kDescHiSw128 = (1024u >> 4) | (1u << 14) | (2u << 29);  // 8-row groups 1 KB apart, version, 128-byte swizzle
constexpr uint32_t kDescLoSw128 = (16u >> 4) << 16;
constexpr uint32_t kDescHiScales = (128u >> 4) | (1u << 14);               // groups of 8 rows of 16 bytes, no swizzle
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr) { return (saddr & 0x3FFFFu) >> 4; }
__device__ __forceinline__ uint64_t desc(uint32_t lo, uint32_t hi) { return ((uint64_t)hi << 32) | lo; }

// one scale tile (512 bytes) from shared memory to four columns of tensor
// memory, of every lane quarter (CTAS = 2: in both CTAs of the pair, each from
// its own shared memory at the same offset)
template <int CTAS>
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint32_t lo) {
  const uint64_t d = desc(lo, kDescHiScales);
  if (CTAS == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

// this thread's TMEM lane, 32 columns
__device__ __forceinline__ void tmem_ld32(uint32_t ta, uint32_t (&a)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]),
        "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15]),
        "=r"(a[16]), "=r"(a[17]), "=r"(a[18]), "=r"(a[19]), "=r"(a[20]), "=r"(a[21]), "=r"(a[22]), "=r"(a[23]),
        "=r"(a[24]), "=r"(a[25]), "=r"(a[26]), "=r"(a[27]), "=r"(a[28]), "=r"(a[29]), "=r"(a[30]), "=r"(a[31])
      : "r"(ta)
      : "memory");
}

// four 8 x 8 matrices of 16-bit elements, transposed: lane l gives the address
// of row l % 8 of matrix l / 8
__device__ __forceinline__ void stmatrix4_trans(uint32_t saddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(saddr), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(uint32_t lo, uint32_t hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
  return *reinterpret_cast<const uint32_t*>(&p);
}

// One work item; every role walks the same sequence with its own cursor.
struct Item {
  int g;        // group
  int row0;     // first token row
  int n;        // token rows, 1 .. NT
  int local;    // row0 within its group
  int mb;       // block of weight rows
};

template <int NT>
__device__ __forceinline__ void item_at(Item& t, int item, int mblocks, const int* off, const int* pre) {
  const int tile = item / mblocks;
  t.mb = item - tile * mblocks;
  while (tile >= uniform(pre[t.g + 1])) ++t.g;
  t.local = (tile - uniform(pre[t.g])) * NT;
  t.row0 = uniform(off[t.g]) + t.local;
  t.n = min(NT, uniform(off[t.g + 1]) - t.row0);
}

// Group tables, by one warp: off[e], e in [0, E], the offsets clamped to [0, M]
// and made non-decreasing (offsets that decrease make empty groups); pre[e],
// the token tiles before group e.
template <int NT>
__device__ void group_tables(const MmParams& P, int* off, int* pre, int lane) {
  int tiles = 0, last = 0;
  for (int e0 = 0; e0 <= P.E; e0 += 32) {
    const int e = e0 + lane;
    int o = 0;
    if (e <= P.E) o = P.offsets ? min(max(P.offsets[e], 0), P.M) : (e == 0 ? 0 : P.M);
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, o, s);
      if (lane >= s) o = max(o, v);
    }
    o = max(o, last);
    int before = __shfl_up_sync(0xFFFFFFFFu, o, 1);
    if (lane == 0) before = last;
    // tiles of group e - 1 = [off[e - 1], off[e]), counted at lane e
    int c = e >= 1 && e <= P.E ? (o - before + NT - 1) / NT : 0;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, c, s);
      if (lane >= s) c += v;
    }
    if (e <= P.E) {
      off[e] = o;
      pre[e] = tiles + c;
    }
    tiles += __shfl_sync(0xFFFFFFFFu, c, 31);
    last = __shfl_sync(0xFFFFFFFFu, o, 31);
  }
}

// a bounded wait of the whole (converged) warp
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, const MmParams& P) {
  if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
  const bool ok = mbar_wait(bar, parity, abort_flag, P.err, kErrWaitTimeout, P.wait_ns);
  return __all_sync(0xFFFFFFFFu, ok);
}

// position in a ring of S stages
template <int S>
struct Ring {
  int s = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++s == S) {
      s = 0;
      phase ^= 1;
    }
  }
};

// ---- epilogue -----------------------------------------------------------------
// The accumulator has features in lanes and tokens in columns; y wants a
// token's features side by side.  A chunk of 32 tokens (16 of a plain fp32
// product) goes to shared memory, [token][feature], and leaves from there 16
// bytes a thread (or, where rows of y do not start on 16 bytes, by single
// elements).  bf16: TMEM is read as 16 x 8 fragments, which stmatrix stores
// transposed: 16 conversions and 4 stores for 32 x 32 values.  (One bulk copy a
// row instead costs its issuing thread ~70 cycles each, 2,300 a chunk:
// measured.)
//
// Eight warps, in two groups of four (a lane quarter each): group h takes every
// other chunk, in two buffers of its own, one barrier a chunk.  Chunks are
// read in rounds of 64 columns a group, so that the accumulator is given back
// after the reads alone.
constexpr int kEpiWarps = 8;
constexpr int kEpiBuf = 32 * (kBM * 2 + 16);
constexpr int kEpiBytes = 4 * kEpiBuf;

// whether `ok` holds in all epilogue warps: they go on, or leave, together
__device__ __forceinline__ bool all_of_epilogue(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred pin, pout;\n\tsetp.ne.u32 pin, %1, 0;\n\tbar.red.and.pred pout, 3, %2, pin;\n\t"
      "selp.u32 %0, 1, 0, pout;\n}"
      : "=r"(all)
      : "r"(ok ? 1u : 0u), "r"(kEpiWarps * 32)
      : "memory");
  return all != 0;
}

template <bool F32, bool SW>
struct Epilogue {
  static constexpr int kTokens = F32 && !SW ? 16 : 32;         // tokens of a chunk = its columns
  static constexpr int kLoads = 64 / kTokens;                  // chunks of a round
  static constexpr int kFeatures = SW ? kBM / 2 : kBM;         // features of a tile
  static constexpr int kRowBytes = kFeatures * (F32 ? 4 : 2);
  static constexpr int kPitch = kRowBytes + 16;
  static constexpr int kPerRow = kRowBytes / 16;               // threads of a row
  static constexpr int kRowStep = kEpiWarps * 16 / kPerRow;    // rows of a step of the group
  static constexpr int kEs = F32 ? 4 : 2;
  static_assert(kTokens * kPitch <= kEpiBuf, "buffer");

  uint8_t* buf;      // the group's two buffers
  int q, h, lane;    // lane quarter, group
  int tid;           // thread of the group
  int vec, n_out;
  uint32_t count;    // chunks of this group so far

  __device__ __forceinline__ Epilogue(const MmParams& P, uint8_t* epi, int warp, int lane_)
      : buf(epi + ((warp >> 2) & 1) * 2 * kEpiBuf), q(warp & 3), h((warp >> 2) & 1), lane(lane_),
        tid((warp & 3) * 32 + lane_), vec(P.vec), n_out(P.n_out), count(0) {}

  __device__ __forceinline__ void sync() { asm volatile("bar.sync %0, 128;" ::"r"(1 + h) : "memory"); }

  // kTokens columns from taddr (with the warp's lane base)
  __device__ __forceinline__ void load(uint32_t ta, uint32_t* a) {
    if (F32 && !SW)
      asm volatile(
          "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
          : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]),
            "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15])
          : "r"(ta)
          : "memory");
    else
      // 16 x 8 fragments: a[16 k + 4 j + i] of thread t is lane 16 k + t / 4 + 8 (i / 2), column
      // 8 j + 2 (t % 4) + i % 2
      asm volatile(
          "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n\t"
          "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, "
          "[%33];"
          : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]),
            "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15]),
            "=r"(a[16]), "=r"(a[17]), "=r"(a[18]), "=r"(a[19]), "=r"(a[20]), "=r"(a[21]), "=r"(a[22]), "=r"(a[23]),
            "=r"(a[24]), "=r"(a[25]), "=r"(a[26]), "=r"(a[27]), "=r"(a[28]), "=r"(a[29]), "=r"(a[30]), "=r"(a[31])
          : "r"(ta), "r"(ta + (16u << 16))
          : "memory");
  }

  // a chunk's values to shared memory
  __device__ __forceinline__ void stage(uint32_t* v, uint8_t* b) {
    if (F32 && !SW) {
      float* o = reinterpret_cast<float*>(b) + q * 32 + lane;
#pragma unroll
      for (int j = 0; j < kTokens; ++j) o[j * (kPitch / 4)] = __uint_as_float(v[j]);
      return;
    }
    if (!SW) {
      const uint32_t s = smem_u32(b) + (lane & 7) * kPitch + (q * 32 + (lane >> 3) * 8) * 2;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        stmatrix4_trans(s + 8 * j * kPitch, pack_bf16(v[4 * j], v[4 * j + 1]), pack_bf16(v[4 * j + 2], v[4 * j + 3]),
                        pack_bf16(v[16 + 4 * j], v[16 + 4 * j + 1]), pack_bf16(v[16 + 4 * j + 2], v[16 + 4 * j + 3]));
      return;
    }
    // Gate and up rows alternate: of a fragment's rows r = t / 4 and r + 8,
    // threads of even r compute feature r / 2 (rows r, r + 1), threads of odd r
    // feature 4 + (r - 1) / 2 (rows r + 7, r + 8).
    const bool odd = (lane >> 2) & 1;
    const int r = lane >> 2;
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
      const uint32_t x0 = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[i] : v[i + 2], 4);
      const uint32_t x1 = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[i + 1] : v[i + 3], 4);
      const float g0 = __uint_as_float(odd ? x0 : v[i]), u0 = __uint_as_float(odd ? v[i + 2] : x0);
      const float g1 = __uint_as_float(odd ? x1 : v[i + 1]), u1 = __uint_as_float(odd ? v[i + 3] : x1);
      v[i] = __float_as_uint(swiglu(g0, u0));
      v[i + 1] = __float_as_uint(swiglu(g1, u1));
    }
    if (F32) {
      float* o = reinterpret_cast<float*>(b) + q * 16 + (odd ? 4 + (r >> 1) : r >> 1) + 2 * (lane & 3) * (kPitch / 4);
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        float* p = o + 8 * ((i & 15) >> 2) * (kPitch / 4) + 8 * (i >> 4);
        p[0] = __uint_as_float(v[i]);
        p[kPitch / 4] = __uint_as_float(v[i + 1]);
      }
    } else {
      // feature f back to the threads of matrix row f; h[j], h[4 + j]: lanes 0..15 and 16..31 of columns 8 j on
      const int src = (r < 4 ? 2 * r : 2 * r - 7) * 4 + (lane & 3);
      uint32_t hv[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) hv[i] = __shfl_sync(0xFFFFFFFFu, pack_bf16(v[4 * i], v[4 * i + 1]), src);
      const int m = lane >> 3;
      const uint32_t s = smem_u32(b) + (8 * (m >> 1) + (lane & 7)) * kPitch + (q * 16 + (m & 1) * 8) * 2;
      stmatrix4_trans(s, hv[0], hv[4], hv[1], hv[5]);
      stmatrix4_trans(s + 16 * kPitch, hv[2], hv[6], hv[3], hv[7]);
    }
  }

  // a staged chunk to y (at its first token and feature): `rows` tokens, nf features
  __device__ __forceinline__ void write(const uint8_t* b, uint8_t* y, int rows, int nf) {
    const size_t ldy = (size_t)n_out * kEs;
    if (vec) {
      const int r = tid / kPerRow, c = (tid % kPerRow) * 16;
      const uint8_t* src = b + r * kPitch + c;
      uint8_t* dst = y + r * ldy + c;
      const bool in = c < nf * kEs;
      uint4 v[kTokens / kRowStep];
#pragma unroll
      for (int k = 0; k < kTokens / kRowStep; ++k) v[k] = *reinterpret_cast<const uint4*>(src + k * kRowStep * kPitch);
#pragma unroll
      for (int k = 0; k < kTokens / kRowStep; ++k)
        if (in && r + k * kRowStep < rows) *reinterpret_cast<uint4*>(dst + k * kRowStep * ldy) = v[k];
    } else if (F32) {
      write_elements(reinterpret_cast<const float*>(b), reinterpret_cast<float*>(y), rows, nf);
    } else {
      write_elements(reinterpret_cast<const uint16_t*>(b), reinterpret_cast<uint16_t*>(y), rows, nf);
    }
  }

  // rows by warps, a row's features by lanes
  template <typename T>
  __device__ __forceinline__ void write_elements(const T* b, T* y, int rows, int nf) {
    constexpr int kR = 4;  // rows in flight
#pragma unroll
    for (int i0 = 0; i0 < kTokens; i0 += 4 * kR) {
      T v[kR][kFeatures / 32];
#pragma unroll
      for (int k = 0; k < kR; ++k)
#pragma unroll
        for (int u = 0; u < kFeatures / 32; ++u) v[k][u] = b[(i0 + 4 * k + q) * (kPitch / kEs) + 32 * u + lane];
#pragma unroll
      for (int k = 0; k < kR; ++k) {
        const int i = i0 + 4 * k + q;
        T* row = y + (size_t)i * n_out + lane;
        if (i < rows)
#pragma unroll
          for (int u = 0; u < kFeatures / 32; ++u)
            if (32 * u + lane < nf) row[32 * u] = v[k][u];
      }
    }
  }

  // One item: n tokens from row0, its accumulator at taddr, features from f0
  // (nf of them in y).  Chunks are taken from `first` on, cyclically.
  // after_reads(last): this group has read its chunks of the first round
  // (chunks first .. first + 127 / kTokens of the item), or, last, all of them.
  // False, with nothing written, if some epilogue warp's wait for the
  // accumulator ran out (not ok).
  template <typename F>
  __device__ __forceinline__ bool item(void* y, uint32_t taddr, int row0, int n, int f0, int nf, int first, bool ok,
                                       F&& after_reads) {
    const int chunks = (n + kTokens - 1) / kTokens;
    uint8_t* const y0 = static_cast<uint8_t*>(y) + ((size_t)row0 * n_out + f0) * kEs;
    taddr += (uint32_t)(q * 32) << 16;
    int i = h;
    do {
      uint32_t v[kLoads][kTokens];
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int at = first + i + 2 * k;
        if (i + 2 * k < chunks) load(taddr + (at < chunks ? at : at - chunks) * kTokens, v[k]);
      }
      asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      after_reads(i == h, i + 2 * kLoads >= chunks);
      if (i == h && !all_of_epilogue(ok)) return false;
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        if (i + 2 * k >= chunks) break;
        const int at = first + i + 2 * k, t0 = (at < chunks ? at : at - chunks) * kTokens;
        // (a warp here has passed the barrier of the last chunk, and with it every warp of the group has read
        // what the chunk before that left in this buffer)
        uint8_t* b = buf + (count++ & 1) * kEpiBuf;
        stage(v[k], b);
        sync();
        write(b, y0 + (size_t)t0 * n_out * kEs, min(kTokens, n - t0), nf);
      }
      i += 2 * kLoads;
    } while (i < chunks);
    return true;
  }
};

}  // namespace mm

// the kernel for few rows of one matrix, M <= kFewRows (mxfp4_mm1.cu): rows x
// to quantise, or (x null) their codes with P.a_scales
constexpr int kFewRows = 16;
cudaError_t launch_mm_few(const CUtensorMap& map_w, const mm::MmParams& P, const MxRows* x, const uint8_t* codes,
                          cudaStream_t st);
// the pair kernel (mxfp4_mm2.cu); the boxes of map_a have 32 rows, those of
// map_a128 128; map_ws and map_as: scale tiles as rows of 512 bytes, boxes of 2
cudaError_t launch_mm_pairs(const CUtensorMap& map_w, const CUtensorMap& map_a, const CUtensorMap& map_a128,
                            const CUtensorMap& map_ws, const CUtensorMap& map_as, const mm::MmParams& P,
                            cudaStream_t st);

}  // namespace moe_fp4
