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
  int vec;                   // rows of y start on 4 bytes and have an even number of features
  int split;                 // CTAs of a cluster that share an item's K (1: none)
  int rows_ahead;            // the kernel ahead writes the rows (a and a_scales); all before it has ended
  int fault;                 // nonzero: the first CTA withholds its first stage (fault-injection test)
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

// this thread's TMEM lane, 32 columns; valid after tcgen05.wait::ld
__device__ __forceinline__ void tmem_ld32_async(uint32_t ta, uint32_t (&a)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]),
        "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15]),
        "=r"(a[16]), "=r"(a[17]), "=r"(a[18]), "=r"(a[19]), "=r"(a[20]), "=r"(a[21]), "=r"(a[22]), "=r"(a[23]),
        "=r"(a[24]), "=r"(a[25]), "=r"(a[26]), "=r"(a[27]), "=r"(a[28]), "=r"(a[29]), "=r"(a[30]), "=r"(a[31])
      : "r"(ta)
      : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(uint32_t lo, uint32_t hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(__uint_as_float(lo), __uint_as_float(hi));
  return *reinterpret_cast<const uint32_t*>(&p);
}

// silu(g) u.  For results in fp32 with the sigmoid to a few 2^-24: the fast one's
// error grows with |g|, 2^-18 of the result at 50.  Results in bf16 lose nothing
// by it.  (In fp32, 4096 x 4096 x 4096: 34.7 us, 33.5 with the fast one, 42 with expf and
// a rounded quotient; 8192 x 8192 x 512: 62, 55 and 102.)
template <bool F32>
__device__ __forceinline__ float gated(float g, float u) {
  return F32 ? g * sigmoid(g) * u : swiglu(g, u);
}

// Lanes l and l ^ d hold two bf16 each, (a0, a1) and (b0, b1): the lower lane
// gets (a0, b0), the upper (a1, b1); sel is 0x5410 in the lower, 0x3276 in the upper.
__device__ __forceinline__ uint32_t swap_pair(uint32_t p, int d, uint32_t sel) {
  return __byte_perm(p, __shfl_xor_sync(0xFFFFFFFFu, p, d), sel);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// four floats of shared memory at this offset in CTA `rank` of the cluster
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [a];\n}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}
// a word of it
__device__ __forceinline__ uint32_t ld_cluster1(uint32_t addr, uint32_t rank) {
  uint32_t v;
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.b32 %0, [a];\n}"
      : "=r"(v)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

// K split over a cluster: the CTAs' partial sums [token][weight row] (floats,
// kPartPitch apart, at the same offset `part` in each) summed in rank order; a
// warp a token, four rows a lane, CTA `rank` the tokens rank, rank + split, ...
// Nothing is stored if a wait ran out in any of the CTAs (its abort flag, at
// `abort` in each, is up): its sums are then missing or incomplete.
constexpr int kPartPitch = kBM + 4;
template <bool F32, bool SW>
__device__ __forceinline__ void sum_parts(const MmParams& P, uint32_t part, uint32_t abort, int rank, int row0, int n,
                                          int mb, int warp, int lane) {
  constexpr int kF = SW ? kBM / 2 : kBM, kOwn = SW ? 2 : 4;  // features of a tile, of a lane
  const int f = mb * kF + lane * kOwn, warps = blockDim.x >> 5;
  const uint32_t failed = lane < P.split ? ld_cluster1(abort, lane) : 0;  // on its way with the first sums
  for (int t = rank + warp * P.split; t < n; t += warps * P.split) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int r = 0; r < P.split; ++r) {
      const float4 v = ld_cluster4(part + (t * kPartPitch + 4 * lane) * 4, r);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    if (__any_sync(0xFFFFFFFFu, failed)) return;
    float o[4] = {s.x, s.y, s.z, s.w};
    if (SW) o[0] = gated<F32>(s.x, s.y), o[1] = gated<F32>(s.z, s.w);
    const size_t at = (size_t)(row0 + t) * P.n_out + f;
    if (!F32 && P.vec) {
#pragma unroll
      for (int j = 0; j < kOwn; j += 2)
        if (f + j < P.n_out)
          *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(P.y) + at + j) =
              pack_bf16(__float_as_uint(o[j]), __float_as_uint(o[j + 1]));
    } else {
#pragma unroll
      for (int j = 0; j < kOwn; ++j)
        if (f + j < P.n_out) {
          if (F32)
            static_cast<float*>(P.y)[at + j] = o[j];
          else
            static_cast<uint16_t*>(P.y)[at + j] = f32_to_bf16_rn(o[j]);
        }
    }
  }
}

// One work item; every role walks the same sequence with its own cursor.
struct Item {
  int g;        // group
  int row0;     // first token row
  int n;        // token rows, 1 .. NT
  int local;    // row0 within its group
  int mb;       // block of weight rows
};

// The item of number `item` (of a tile below pre[E]) from a cursor that is not
// past it; whole warp: 32 groups a step.
template <int NT>
__device__ __forceinline__ void item_at(Item& t, int item, int mblocks, const int* off, const int* pre, int groups) {
  const int tile = item / mblocks, lane = threadIdx.x & 31;
  t.mb = item - tile * mblocks;
  int passed;
  do {
    const int e = t.g + 1 + lane;
    passed = __popc(__ballot_sync(0xFFFFFFFFu, e < groups && pre[min(e, groups)] <= tile));
    t.g += passed;
  } while (passed == 32);
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
// token's features side by side.  Values go from registers to y as they are, a
// token's 32 features of a warp a store: whole sectors.  (bf16, with lane pairs
// that swap values and store two features: 8192 x 2048 x 4096 28.5 us against
// 27.4.  With SwiGLU's 16 features a warp that swap pays: 13073 x 128 x 1522 19
// us against 20.)  Nothing passes through shared memory: the MMAs of 256 x 256
// tiles take all of its bandwidth, and an epilogue that turned its tile there
// took 7,000 cycles beside them, longer than the MMAs of K = 2048.
//
// Eight warps, in two groups of four (a lane quarter each): group h takes every
// other chunk of 32 tokens.  Chunks are read in rounds of two a group, so that
// the accumulator is given back after the reads alone.
constexpr int kEpiWarps = 8;
constexpr int kTokens = 32;  // tokens of a chunk = its columns

// Whether `ok` holds in all the `warps` epilogue warps that share barrier `id`.
// This barrier has no time limit, so every epilogue warp comes to every one of
// them: a warp whose wait ran out walks through all of its items still, without
// waits and without stores (see Epilogue::item).
__device__ __forceinline__ bool all_of_epilogue(bool ok, int id, int warps) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred pin, pout;\n\tsetp.ne.u32 pin, %1, 0;\n\tbar.red.and.pred pout, %3, %2, pin;\n\t"
      "selp.u32 %0, 1, 0, pout;\n}"
      : "=r"(all)
      : "r"(ok ? 1u : 0u), "r"(warps * 32), "r"(id)
      : "memory");
  return all != 0;
}

template <bool F32, bool SW>
struct Epilogue {
  static constexpr int kFeatures = SW ? kBM / 2 : kBM;  // features of a tile
  static constexpr int kEs = F32 ? 4 : 2;

  int q, h, lane;    // lane quarter, group
  int vec;           // rows of y start on 4 bytes, and n_out is even
  size_t ldy;        // bytes

  __device__ __forceinline__ Epilogue(const MmParams& P, int warp, int lane_)
      : q(warp & 3), h((warp >> 2) & 1), lane(lane_), vec(P.vec), ldy((size_t)P.n_out * kEs) {}

  // rows tokens of one chunk to y (at its first token, the tile's first
  // feature), nf features.  ALL: 32 tokens and a whole tile.
  template <bool ALL>
  __device__ __forceinline__ void put(const uint32_t (&v)[kTokens], uint8_t* y, int rows, int nf) {
    const bool odd = lane & 1;
    if (!SW && F32) {
      const int f = q * 32 + lane;
      y += f * 4;
#pragma unroll
      for (int j = 0; j < kTokens; ++j)
        if (ALL || (j < rows && f < nf)) *reinterpret_cast<uint32_t*>(y + j * ldy) = v[j];
    } else if (!SW) {
      const int f = q * 32 + lane;
      y += f * 2;
#pragma unroll
      for (int j = 0; j < kTokens; ++j)
        if (ALL || (j < rows && f < nf)) *reinterpret_cast<uint16_t*>(y + j * ldy) = f32_to_bf16_rn(__uint_as_float(v[j]));
    } else {
      // gate in even lanes, up in odd ones: of tokens j and j + 1 the even lane takes the first, the odd the second
      float s[kTokens / 2];
#pragma unroll
      for (int j = 0; j < kTokens; j += 2) {
        const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[j] : v[j + 1], 1);
        s[j / 2] = gated<F32>(__uint_as_float(odd ? other : v[j]), __uint_as_float(odd ? v[j + 1] : other));
      }
      if (F32 || !vec) {
        const int f = q * 16 + (lane >> 1);
        y += (odd ? ldy : 0) + f * kEs;
#pragma unroll
        for (int j = 0; j < kTokens; j += 2)
          if (ALL || (j + (odd ? 1 : 0) < rows && f < nf)) {
            if (F32)
              *reinterpret_cast<float*>(y + j * ldy) = s[j / 2];
            else
              *reinterpret_cast<uint16_t*>(y + j * ldy) = f32_to_bf16_rn(s[j / 2]);
          }
      } else {
        // the same swap between lanes 2 apart, which hold adjacent features: each stores two features of one token
        const bool second = lane & 2;
        const uint32_t sel = second ? 0x3276u : 0x5410u;
        const int f = q * 16 + (lane >> 2) * 2, jj = (odd ? 1 : 0) + (second ? 2 : 0);
        y += jj * ldy + f * 2;
#pragma unroll
        for (int j = 0; j < kTokens; j += 4) {
          const uint32_t p =
              swap_pair(pack_bf16(__float_as_uint(s[j / 2]), __float_as_uint(s[j / 2 + 1])), 2, sel);
          if (ALL || (j + jj < rows && f < nf)) *reinterpret_cast<uint32_t*>(y + j * ldy) = p;
        }
      }
    }
  }

  // An item of one chunk: the groups take such items in turn (32 tokens x 8 over
  // 128 experts, K = 512, N = 2048: 16.9 -> 15.2 us; 1024 x 8 over 256: 41.4 -> 39.2).
  template <typename F>
  __device__ __forceinline__ bool one_chunk(void* y, uint32_t taddr, int row0, int n, int f0, int nf, bool ok, int turn,
                                            F&& after_reads) {
    if ((turn & 1) != h) {
      __syncwarp();
      if (ok) after_reads(true, true);
      return ok;
    }
    uint32_t v[kTokens];
    tmem_ld32_async(taddr + ((uint32_t)(q * 32) << 16), v);
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncwarp();
    if (ok) after_reads(true, true);
    if (!all_of_epilogue(ok, 4 + h, kEpiWarps / 2)) return false;
    put<false>(v, static_cast<uint8_t*>(y) + (size_t)row0 * ldy + (size_t)f0 * kEs, n, nf);
    return true;
  }

  // One item: n tokens from row0, its accumulator at taddr, features from f0
  // (nf of them in y).  Chunks are taken from `first` on, cyclically.
  // after_reads(round0, last): this group has read its chunks of the first
  // round (the item's chunks first .. first + 3), or, last, all of them.
  // False, with nothing written, if the wait for the accumulator ran out in a
  // warp that takes chunks of the item (not ok).  The caller hands that result
  // on as the next item's `ok`: which barriers an item has depends on its rows
  // alone, so that no warp is left alone in one, and a warp that failed gives no
  // accumulator back that others may still read.
  template <typename F>
  __device__ __forceinline__ bool item(void* y, uint32_t taddr, int row0, int n, int f0, int nf, int first, bool ok,
                                       int turn, F&& after_reads) {
    const int chunks = (n + kTokens - 1) / kTokens;
    if (chunks == 1) return one_chunk(y, taddr, row0, n, f0, nf, ok, turn, after_reads);
    uint8_t* const y0 = static_cast<uint8_t*>(y) + (size_t)row0 * ldy + (size_t)f0 * kEs;
    taddr += (uint32_t)(q * 32) << 16;
    int i = h;
    do {
      uint32_t v[2][kTokens];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int at = first + i + 2 * k;
        if (i + 2 * k < chunks) tmem_ld32_async(taddr + (at < chunks ? at : at - chunks) * kTokens, v[k]);
      }
      asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (ok) after_reads(i == h, i + 4 >= chunks);
      if (i == h && !all_of_epilogue(ok, 3, kEpiWarps)) return false;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (i + 2 * k >= chunks) break;
        const int at = first + i + 2 * k, t0 = (at < chunks ? at : at - chunks) * kTokens;
        if (n - t0 >= kTokens && nf == kFeatures)
          put<true>(v[k], y0 + (size_t)t0 * ldy, kTokens, nf);
        else
          put<false>(v[k], y0 + (size_t)t0 * ldy, min(kTokens, n - t0), nf);
      }
      i += 4;
    } while (i < chunks);
    return true;
  }
};

}  // namespace mm

// launch_early with clusters of `cluster` CTAs
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster_early(void (*kernel)(KArgs...), int grid, int cluster, int threads, size_t smem,
                                 cudaStream_t st, Args&&... args) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = threads;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

// the kernel for few rows of one matrix, M <= kFewRows (mxfp4_mm1.cu): rows x
// to quantise, or (x null) their codes with P.a_scales
constexpr int kFewRows = MOE_FP4_MXFP4_FEW_ROWS;
cudaError_t launch_mm_few(const CUtensorMap& map_w, const mm::MmParams& P, const MxRows* x, const uint8_t* codes,
                          cudaStream_t st);
// the pair kernel (mxfp4_mm2.cu); the boxes of map_a have 32 rows, those of
// map_a128 128; map_ws and map_as: scale tiles as rows of 512 bytes, boxes of 2
cudaError_t launch_mm_pairs(const CUtensorMap& map_w, const CUtensorMap& map_a, const CUtensorMap& map_a128,
                            const CUtensorMap& map_ws, const CUtensorMap& map_as, const mm::MmParams& P,
                            cudaStream_t st);

}  // namespace moe_fp4
