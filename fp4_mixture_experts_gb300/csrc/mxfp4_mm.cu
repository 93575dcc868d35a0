// Products of MXFP4 matrices on block-scaled tensor cores, dense and grouped.
//
//   y[m, n] = sum_b 2^(sa[m, b] + sw[n, b]) sum_{j < 32} a[m, 32 b + j] w[n, 32 b + j]
//
// tcgen05.mma kind::mxf4 takes both operands as packed E2M1 codes (K = 64 an
// instruction) and one E8M0 scale for 32 elements of either (scale_vec::2X),
// so nothing is decoded in software: the products and their scales are exact,
// the sums fp32.
//
// A work item is 128 weight rows (the MMA's M) by up to NT token rows (its N)
// of one group.  Weights are M because a group may have few rows: N goes down
// to 16 in steps of 16.  A stage of the ring holds K = 256 of both operands
// (128 bytes a row, 128-byte swizzle, TMA) and their scale tiles, which a
// one-dimensional bulk copy brings as they lie in memory: a tile of 128 rows x
// 4 scales is the 512 bytes that one tcgen05.cp (32x128b, to all four lane
// quarters) takes to four columns of tensor memory.
//
// With SwiGLU the weight map has gate and up rows in turn (a dimension of
// extent 2 between K and the feature), so that a pair of lanes holds the gate
// and the up value of one feature.
//
// Warp roles: 0 the TMA producer, 1 the MMA issuer (and owner of tensor
// memory), 2..5 the epilogue.  All waits are bounded; on a timeout every role
// leaves its loop, and copies and MMAs in flight end before memory is given
// back.
#include <cuda.h>

#include <algorithm>

#include "moe_fp4_internal.cuh"
#include "mxfp4_ops.cuh"
#include "ptx_sm103.cuh"
#include "tc_helpers.cuh"

namespace moe_fp4 {
namespace {

using namespace tc;

__device__ int32_t g_mm_err[4];

constexpr int kBM = 128;        // weight rows per item
constexpr int kStageK = 256;    // K elements per stage: 128 bytes of codes a row
constexpr int kSfTile = 512;    // bytes of one scale tile: 128 rows x 4 scales (K = 128)
constexpr int kThreads = 192;
constexpr uint32_t kTmemCols = 512;
constexpr int kSmemMax = 227 * 1024;

template <int NT>
struct Cfg {
  static constexpr int kATile = kBM * 128;
  static constexpr int kBTile = NT * 128;
  static constexpr int kSfB = (NT + 127) / 128;              // scale tiles of the token rows, per K = 128
  static constexpr int kStage = kATile + kBTile + 2 * kSfTile * (1 + kSfB);
  static constexpr int kSfCols = 2 * 4 * (1 + kSfB);         // tensor-memory columns of a stage's scales
  static constexpr int kAccs = NT <= 128 ? 2 : 1;            // accumulators (double buffered where they fit)
  static constexpr int kGroupBytes = 2 * (kMaxGroups + 1) * 4;
  static constexpr int kFixed = 1024 + 512 + kGroupBytes;    // alignment, barriers, group tables
  static constexpr int kByMem = (kSmemMax - kFixed) / kStage;
  static constexpr int kByTmem = ((int)kTmemCols - kAccs * NT) / kSfCols;
  static constexpr int kStages = kByMem < kByTmem ? kByMem : kByTmem;
  static constexpr int kSmem = kStages * kStage + kFixed;
  static_assert(kStage % 1024 == 0, "stages stay 1 KB aligned for the 128-byte swizzle");
  static_assert(kStages >= 3, "ring too short");
};

struct MmParams {
  const uint8_t* a_scales;   // tiled, grouped
  const uint8_t* w_scales;   // [E][wrt][kt][512]
  const int32_t* offsets;    // [E + 1] or null
  void* y;
  int M, N, K, E;
  int n_out;                 // features of y
  int mblocks;               // ceil(N / 128)
  int kt;                    // scale tiles along K
  int f32, swiglu;
  int paired;                // bf16 rows of y are 4-byte aligned and even: two features a store
  uint64_t wait_ns;
};

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

__device__ __forceinline__ void umma_mxf4(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                          uint32_t sfb, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n}" ::"r"(
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

// one scale tile (512 bytes) from shared memory to four columns of tensor memory
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(128u >> 4) << 32;  // stride between groups of 8 rows of 16 bytes
  d |= (uint64_t)1 << 46;            // descriptor version; no swizzle
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(d) : "memory");
}

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

// One work item; every role walks the same sequence with its own cursor.
struct Item {
  int g;        // group
  int row0;     // first token row
  int n;        // token rows, 1 .. NT
  int n_mma;    // n rounded up to 16
  int local;    // row0 within its group
  int mb;       // block of 128 weight rows
};

// off[e], e in [0, E], clamped to [0, M] and made non-decreasing; pre[e]: token tiles before group e
template <int NT>
__device__ __forceinline__ void item_at(Item& t, int item, int mblocks, const int* off, const int* pre) {
  const int tile = item / mblocks;
  t.mb = item - tile * mblocks;
  while (tile >= pre[t.g + 1]) ++t.g;
  t.local = (tile - pre[t.g]) * NT;
  t.row0 = off[t.g] + t.local;
  t.n = min(NT, off[t.g + 1] - t.row0);
  t.n_mma = (t.n + 15) & ~15;
}

// Group tables, by one warp.
template <int NT>
__device__ void group_tables(const MmParams& P, int* off, int* pre, int lane) {
  int tiles = 0, last = 0;
  for (int e0 = 0; e0 <= P.E; e0 += 32) {
    const int e = e0 + lane;
    int o = 0;
    if (e <= P.E) o = P.offsets ? min(max(P.offsets[e], 0), P.M) : (e == 0 ? 0 : P.M);
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {  // running maximum: offsets that decrease make empty groups
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

template <int NT>
__global__ void __launch_bounds__(kThreads, 1)
mm_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a, const MmParams P) {
  using C = Cfg<NT>;
  constexpr int kStages = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* tail = smem + kStages * C::kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(tail);    // [stage]: bytes landed
  uint64_t* empty = full + kStages;                      // [stage]: its MMAs completed
  uint64_t* acc_full = empty + kStages;                  // [2]
  uint64_t* acc_empty = acc_full + 2;                    // [2]
  uint64_t* mma_done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* off = reinterpret_cast<int*>(tail + 512);
  int* pre = off + kMaxGroups + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t lim = P.wait_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (warp == 2) group_tables<NT>(P, off, pre, lane);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = *tmem_slot;
  const uint32_t sf_base = tmem + C::kAccs * NT;
  const int items = pre[P.E] * P.mblocks;
  const int nks = (P.K + kStageK - 1) / kStageK;

  if (warp == 0) {
    if (lane == 0) {
      Item t{};
      int g = 0;
      bool ok = true;
      for (int it = blockIdx.x; it < items && ok; it += gridDim.x) {
        item_at<NT>(t, it, P.mblocks, off, pre);
        const int sf_rows = t.n > 128 ? 2 : 1;
        const uint8_t* ws = P.w_scales + ((size_t)t.g * P.mblocks + t.mb) * P.kt * kSfTile;
        const uint8_t* as = P.a_scales + ((size_t)((off[t.g] >> 7) + t.g + (t.local >> 7))) * P.kt * kSfTile;
        for (int ks = 0; ks < nks; ++ks, ++g) {
          const int s = g % kStages;
          if (!mbar_wait(&empty[s], ((g / kStages) & 1) ^ 1, abort_flag, &g_mm_err[0], kErrWaitTimeout, lim)) {
            ok = false;
            break;
          }
          uint8_t* st = smem + s * C::kStage;
          const uint32_t sf_bytes = min(2, P.kt - 2 * ks) * kSfTile;
          mbar_expect_tx(&full[s], C::kATile + C::kBTile + sf_bytes * (1 + sf_rows));
          if (P.swiglu)
            tma_load_4d(st, &map_w, ks * 128, 0, t.mb * 64, t.g, &full[s]);
          else
            tma_load_4d(st, &map_w, ks * 128, 0, t.mb * 128, t.g, &full[s]);
          tma_load_2d(st + C::kATile, &map_a, ks * 128, t.row0, &full[s]);
          uint8_t* sf = st + C::kATile + C::kBTile;
          bulk_load(sf, ws + (size_t)ks * 2 * kSfTile, sf_bytes, &full[s]);
          for (int j = 0; j < sf_rows; ++j)
            bulk_load(sf + (1 + j) * 2 * kSfTile, as + ((size_t)j * P.kt + ks * 2) * kSfTile, sf_bytes, &full[s]);
        }
      }
      // every issued copy has landed before shared memory is given back
      for (int q = g > kStages ? g - kStages : 0; q < g; ++q)
        mbar_wait_drain(&full[q % kStages], (q / kStages) & 1, &g_mm_err[0], kErrWaitTimeout, lim);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      Item t{};
      int g = 0, li = 0;
      bool ok = true;
      for (int it = blockIdx.x; it < items && ok; it += gridDim.x, ++li) {
        item_at<NT>(t, it, P.mblocks, off, pre);
        const int b = li % C::kAccs, use = li / C::kAccs;
        if (!mbar_wait(&acc_empty[b], (use & 1) ^ 1, abort_flag, &g_mm_err[0], kErrWaitTimeout, lim)) break;
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        const uint32_t d_tmem = tmem + b * NT;
        const uint32_t id0 = idesc_mxf4(kBM, t.n_mma, 0), id1 = idesc_mxf4(kBM, t.n_mma, 1);
        const int sf_rows = t.n > 128 ? 2 : 1;
        const uint32_t shift = (t.local & 127) >> 5;  // a 64-row tile may start in the middle of a scale tile
        for (int ks = 0; ks < nks; ++ks, ++g) {
          const int s = g % kStages;
          if (!mbar_wait(&full[s], (g / kStages) & 1, abort_flag, &g_mm_err[0], kErrWaitTimeout, lim)) {
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          const uint32_t a_addr = smem_u32(smem + s * C::kStage), b_addr = a_addr + C::kATile;
          const uint32_t sf_s = b_addr + C::kBTile;
          const uint32_t sf_t = sf_base + s * C::kSfCols;
          const int chunks = min(2, P.kt - 2 * ks);  // scale tiles (K = 128) of this stage
          for (int c = 0; c < chunks; ++c) {
            // columns: [4 c, 4 c + 4) weights; 8 + 4 kSfB c on: the token rows' kSfB tiles
            tmem_cp_scales(sf_t + 4 * c, sf_s + c * kSfTile);
            for (int j = 0; j < sf_rows; ++j)
              tmem_cp_scales(sf_t + 8 + 4 * (C::kSfB * c + j), sf_s + ((1 + j) * 2 + c) * kSfTile);
          }
          const int steps = min(4, (P.K - ks * kStageK + 63) / 64);
          for (int kk = 0; kk < steps; ++kk) {
            const int c = kk >> 1;
            umma_mxf4(d_tmem, desc_sw128(a_addr + kk * 32), desc_sw128(b_addr + kk * 32), (kk & 1) ? id1 : id0,
                      sf_t + 4 * c, sf_t + 8 + 4 * C::kSfB * c + shift, (ks > 0 || kk > 0) ? 1u : 0u);
          }
          umma_commit(&empty[s]);
        }
        if (!ok) break;
        umma_commit(&acc_full[b]);
      }
      umma_commit(mma_done);
      mbar_wait_drain(mma_done, 0, &g_mm_err[0], kErrWaitTimeout, lim);
    }
  } else {
    const int q = warp & 3;  // the lane quarter this warp may read
    const uint32_t lane_base = tmem + ((uint32_t)(q * 32) << 16);
    const int r = q * 32 + lane;
    const bool odd = lane & 1;
    Item t{};
    int li = 0;
    for (int it = blockIdx.x; it < items; it += gridDim.x, ++li) {
      item_at<NT>(t, it, P.mblocks, off, pre);
      const int b = li % C::kAccs, use = li / C::kAccs;
      const bool ok = mbar_wait(&acc_full[b], use & 1, abort_flag, &g_mm_err[0], kErrWaitTimeout, lim);
      if (!__all_sync(0xFFFFFFFFu, ok)) break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      for (int c0 = 0; c0 < t.n; c0 += 32) {
        uint32_t v[32];
        tmem_ld32(lane_base + b * NT + c0, v);
        const int left = t.n - c0;
        if (P.swiglu) {
          // even lanes hold gate rows, odd lanes up rows: of tokens j and j + 1 the even lane
          // computes the first, the odd lane the second
          const int f = t.mb * 64 + (r >> 1);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[j] : v[j + 1], 1);
            const float gate = __uint_as_float(odd ? other : v[j]), up = __uint_as_float(odd ? v[j + 1] : other);
            const float h = swiglu(gate, up);
            const int jj = j + (odd ? 1 : 0);
            if (jj < left && f < P.n_out) {
              const size_t at = (size_t)(t.row0 + c0 + jj) * P.n_out + f;
              if (P.f32)
                static_cast<float*>(P.y)[at] = h;
              else
                static_cast<uint16_t*>(P.y)[at] = f32_to_bf16_rn(h);
            }
          }
        } else if (P.f32) {
          const int f = t.mb * kBM + r;
          float* y = static_cast<float*>(P.y) + (size_t)(t.row0 + c0) * P.n_out + f;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j < left && f < P.n_out) y[(size_t)j * P.n_out] = __uint_as_float(v[j]);
        } else if (P.paired) {
          // features r, r + 1 of one token in one 4-byte store: even lanes token j, odd lanes token j + 1
          const int f = t.mb * kBM + (r & ~1);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[j] : v[j + 1], 1);
            const float lo = __uint_as_float(odd ? other : v[j]), hi = __uint_as_float(odd ? v[j + 1] : other);
            const int jj = j + (odd ? 1 : 0);
            if (jj < left && f < P.n_out) {
              const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
              *reinterpret_cast<__nv_bfloat162*>(static_cast<uint16_t*>(P.y) +
                                                 (size_t)(t.row0 + c0 + jj) * P.n_out + f) = p;
            }
          }
        } else {
          const int f = t.mb * kBM + r;
          uint16_t* y = static_cast<uint16_t*>(P.y) + (size_t)(t.row0 + c0) * P.n_out + f;
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j < left && f < P.n_out) y[(size_t)j * P.n_out] = f32_to_bf16_rn(__uint_as_float(v[j]));
        }
      }
      asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[b]);
    }
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (warp == 1) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
}

template <int NT>
cudaError_t launch_nt(const moe_fp4_mm_dims& d, const uint8_t* a, const uint8_t* w, const MmParams& P,
                      cudaStream_t st) {
  CUtensorMap map_w, map_a;
  const uint32_t pair = P.swiglu ? 2 : 1;
  const uint64_t row = (uint64_t)d.K / 2;
  const uint64_t dims[4] = {row, pair, (uint64_t)d.N / pair, (uint64_t)d.E};
  const uint64_t strides[3] = {(d.N / pair) * row, row, (uint64_t)d.N * row};
  const uint32_t box[4] = {128, pair, 128 / pair, 1};
  if (!make_map_4d(&map_w, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !make_map_2d(&map_a, CU_TENSOR_MAP_DATA_TYPE_UINT8, a, row, d.M, row, 128, NT, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const void* k = reinterpret_cast<const void*>(mm_kernel<NT>);
  const cudaError_t oe = ensure_smem_optin(k, Cfg<NT>::kSmem);
  if (oe != cudaSuccess) return oe;
  const int64_t most = ((int64_t)d.M / NT + std::min(d.E, d.M)) * P.mblocks;
  const int grid = (int)std::min<int64_t>(most, num_sms());
  mm_kernel<NT><<<grid, kThreads, Cfg<NT>::kSmem, st>>>(map_w, map_a, P);
  return cudaGetLastError();
}

int check_mm(const moe_fp4_mm_dims& d) {
  if (d.M < 0 || d.N < 1 || d.K <= 0 || d.K % 32 != 0 || d.K > 32768 || d.E < 1 || d.E > kMaxGroups ||
      d.swiglu < 0 || d.swiglu > 1 || (d.swiglu && d.N % 2 != 0) ||
      (d.y_type != MOE_FP4_TYPE_BF16 && d.y_type != MOE_FP4_TYPE_F32))
    return MOE_FP4_ERR_INVALID_ARG;
  // item counts and tensor-map extents stay below 2^31
  const int64_t mb = (d.N + 127) / 128;
  if ((int64_t)d.M * d.K >= (1LL << 36) || ((int64_t)d.M / 64 + d.E) * mb >= (1LL << 30)) return MOE_FP4_ERR_UNSUPPORTED;
  return MOE_FP4_OK;
}

int check_mm_pointers(const moe_fp4_mm_dims& d, const void* w, const void* ws, const void* y, const void* offsets) {
  if (!w || !ws || !y || (!offsets && d.E != 1)) return MOE_FP4_ERR_INVALID_ARG;
  const uintptr_t ya = d.y_type == MOE_FP4_TYPE_F32 ? 3 : 1;
  if (((uintptr_t)w & 15) || ((uintptr_t)ws & 15) || ((uintptr_t)y & ya) || ((uintptr_t)offsets & 3))
    return MOE_FP4_ERR_INVALID_ARG;
  return MOE_FP4_OK;
}

cudaError_t launch_mm(const moe_fp4_mm_dims& d, const uint8_t* a, const uint8_t* as, const int32_t* offsets,
                      const uint8_t* w, const uint8_t* ws, void* y, cudaStream_t st) {
  MmParams P{};
  P.a_scales = as;
  P.w_scales = ws;
  P.offsets = offsets;
  P.y = y;
  P.M = d.M, P.N = d.N, P.K = d.K, P.E = d.E;
  P.n_out = d.swiglu ? d.N / 2 : d.N;
  P.mblocks = (d.N + kBM - 1) / kBM;
  P.kt = (d.K + 127) / 128;
  P.f32 = d.y_type == MOE_FP4_TYPE_F32;
  P.swiglu = d.swiglu;
  P.paired = P.n_out % 2 == 0 && ((uintptr_t)y & 3) == 0;
  P.wait_ns = wait_limit_ns();
  // token rows per tile by the rows that a group has on average
  const int64_t mean = (d.M + d.E - 1) / d.E;
  if (mean <= 64) return launch_nt<64>(d, a, w, P, st);
  if (mean <= 128) return launch_nt<128>(d, a, w, P, st);
  return launch_nt<256>(d, a, w, P, st);
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace

cudaError_t ops_mm_error(int32_t* word, bool clear, cudaStream_t st) {
  if (clear) {
    const int32_t zero = 0;
    return cudaMemcpyToSymbolAsync(g_mm_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, st);
  }
  return cudaMemcpyFromSymbolAsync(word, g_mm_err, sizeof(*word), 0, cudaMemcpyDeviceToHost, st);
}

}  // namespace moe_fp4

using namespace moe_fp4;

extern "C" {

int moe_fp4_mxfp4_matmul(const moe_fp4_mm_dims* dims, const uint8_t* a, const uint8_t* a_scales,
                         const int32_t* offsets, const uint8_t* w, const uint8_t* w_scales, void* y,
                         void* cuda_stream) {
  if (!dims) return MOE_FP4_ERR_INVALID_ARG;
  const moe_fp4_mm_dims d = *dims;
  int rc = check_mm(d);
  if (rc != MOE_FP4_OK || d.M == 0) return rc;
  rc = check_mm_pointers(d, w, w_scales, y, offsets);
  if (rc != MOE_FP4_OK) return rc;
  if (!a || !a_scales || ((uintptr_t)a & 15) || ((uintptr_t)a_scales & 15)) return MOE_FP4_ERR_INVALID_ARG;
  return launch_mm(d, a, a_scales, offsets, w, w_scales, y, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess
             ? MOE_FP4_OK
             : MOE_FP4_ERR_CUDA;
}

size_t moe_fp4_mxfp4_linear_workspace_bytes(const moe_fp4_mm_dims* dims) {
  if (!dims || check_mm(*dims) != MOE_FP4_OK) return 0;
  return align256((size_t)dims->M * (dims->K / 2)) + moe_fp4_mxfp4_tiled_scale_bytes(dims->M, dims->E, dims->K);
}

int moe_fp4_mxfp4_linear(const moe_fp4_mm_dims* dims, const void* x, int x_type, int64_t x_rows, int64_t x_stride,
                         const int32_t* row_index, int32_t index_div, const int32_t* offsets, const uint8_t* w,
                         const uint8_t* w_scales, void* y, void* workspace, size_t workspace_bytes,
                         void* cuda_stream) {
  if (!dims || (x_type != MOE_FP4_TYPE_BF16 && x_type != MOE_FP4_TYPE_F32)) return MOE_FP4_ERR_INVALID_ARG;
  const moe_fp4_mm_dims d = *dims;
  int rc = check_mm(d);
  if (rc != MOE_FP4_OK) return rc;
  const MxRows R{x, x_rows, x_stride, row_index, offsets, d.M, d.K, row_index ? index_div : 1, d.E,
                 x_type == MOE_FP4_TYPE_F32};
  rc = check_mx_rows(R);
  if (rc != MOE_FP4_OK || d.M == 0) return rc;
  rc = check_mm_pointers(d, w, w_scales, y, offsets);
  if (rc != MOE_FP4_OK) return rc;
  if (!workspace || ((uintptr_t)workspace & 255)) return MOE_FP4_ERR_INVALID_ARG;
  if (workspace_bytes < moe_fp4_mxfp4_linear_workspace_bytes(dims)) return MOE_FP4_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  uint8_t* codes = static_cast<uint8_t*>(workspace);
  uint8_t* scales = codes + align256((size_t)d.M * (d.K / 2));
  if (launch_mxfp4_quantize(R, codes, scales, true, st) != cudaSuccess) return MOE_FP4_ERR_CUDA;
  return launch_mm(d, codes, scales, offsets, w, w_scales, y, st) == cudaSuccess ? MOE_FP4_OK : MOE_FP4_ERR_CUDA;
}

}  // extern "C"
