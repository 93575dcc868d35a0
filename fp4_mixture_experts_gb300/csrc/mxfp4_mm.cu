// Products of MXFP4 matrices on block-scaled tensor cores, dense and grouped; and,
// with the format Fp8 (mxfp4_mm.cuh), of E4M3 ones with a scale for 128 elements: the
// same tiles, stages of half as many elements, at half the rate (8192 x 8192 x 4096 on SM
// pairs 165 us, 3.3 PFLOP/s; one row, 4096 x 2048, 5.8 us; 64 x 4096 x 4096 with its
// quantiser 9.2; the choice of the tile below is within 3% of the best for them too).
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
// This kernel, one SM a tile, serves groups of up to some 100 rows and dense
// products that cannot fill the SM pairs of mxfp4_mm2.cu.  There reading the
// weights bounds it: the experts' W13 of a 32-token batch (256 x 4096 x 4096, 1.5
// GB touched) takes 210 us, 6.9 TB/s.  What it took beyond a simple ring: uniform
// issue (elect_one), descriptors as sums, the epilogue in registers, and for few
// rounds the start: the first stages' weights are loaded while the kernel ahead
// still quantises the rows (333 x 1056 x 1000, fp32: 13.2 -> 5.9 us with the
// smaller tiles that choose_tile picks).
//
// Warp roles: 0 the TMA producer, 1 the MMA issuer (and owner of tensor
// memory), 4..11 the epilogue.  Two accumulators, so that the epilogue of one
// item runs beside the MMAs of the next.  All waits are bounded; on a timeout
// the producer and the issuer leave their loops, the epilogue goes through its
// items without waits and stores, and copies and MMAs in flight end before
// memory is given back.
#include <cuda.h>

#include <algorithm>
#include <cmath>

#include "mxfp4_mm.cuh"

namespace moe_fp4 {
namespace {

using namespace tc;
using namespace mm;

__device__ int32_t g_mm_err[4];

constexpr int kThreads = 384;

template <typename F, int NT>
struct Cfg {
  static constexpr int kATile = kBM * 128;
  static constexpr int kBTile = NT * 128;
  static constexpr int kSf = 2 * F::kSfTiles;                // scale tiles of a stage
  static constexpr int kStage = kATile + kBTile + kSf * kSfTile;
  static constexpr int kSfCols = 4 * kSf;                    // tensor-memory columns of them
  static constexpr int kGroupBytes = 2 * (kMaxGroups + 1) * 4;
  static constexpr int kFixed = 1024 + 512 + kGroupBytes;
  static constexpr int kByMem = (kSmemMax - kFixed) / kStage;
  static constexpr int kByTmem = ((int)kTmemCols - 2 * NT) / kSfCols;
  static constexpr int kStages = kByMem < kByTmem ? kByMem : kByTmem;
  static constexpr int kSmem = kStages * kStage + kFixed;
  static_assert(NT <= 128, "a token tile's rows lie in one scale tile");
  static_assert(kStage % 1024 == 0, "stages stay 1 KB aligned for the 128-byte swizzle");
  static_assert(kStages >= 3, "ring too short");
};

// SPLIT: a dense product with too few tiles for the SMs.  The CTAs of a cluster
// share one tile's K; their partial sums meet in rank order through distributed
// shared memory, each CTA summing every split-th token.
template <typename F, int NT, bool F32, bool SW, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
mm_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a, MmParams P) {
  P.err = &g_mm_err[0];
  using C = Cfg<F, NT>;
  constexpr int kStages = C::kStages, kStageK = F::kStageK, kSf = F::kSfTiles;
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
  const int warp = warp_index(), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kEpiWarps);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  __syncwarp();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  // behind the quantiser of its rows (rows_ahead) only the rows are waited for, by their producer
  if (!P.rows_ahead) griddep_wait();
  if (warp == 2) group_tables<NT>(P, off, pre, lane);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
  const uint32_t sf_base = tmem + 2 * NT;
  const int items = uniform(pre[P.E]) * P.mblocks;
  // this CTA's items, and its stages of K
  const int rank = SPLIT ? uniform((int)cluster_rank()) : 0;
  const int first = SPLIT ? blockIdx.x / P.split : blockIdx.x, step = SPLIT ? items : gridDim.x;
  const int all_ks = (P.K + kStageK - 1) / kStageK;
  const int k0 = SPLIT ? all_ks * rank / P.split : 0, k1 = SPLIT ? all_ks * (rank + 1) / P.split : all_ks;

  if (warp == 0) {
    Item t{};
    Ring<kStages> ring;
    int g = 0;
    bool ok = true, waited = false;
    for (int it = first; it < items && ok; it += step) {
      item_at<NT>(t, it, P.mblocks, off, pre, P.E);
      const uint8_t* ws = P.w_scales + ((size_t)t.g * P.mblocks + t.mb) * P.kt * kSfTile;
      const uint8_t* as = P.a_scales + ((size_t)((uniform(off[t.g]) >> 7) + t.g + (t.local >> 7))) * P.kt * kSfTile;
      const int wrow = t.mb * (SW ? 64 : 128);
      auto load_w = [&](int ks, int s) {  // and announce the stage's bytes
        if (elect_one()) {
          uint8_t* st = smem + s * C::kStage;
          const uint32_t sf_bytes = min(kSf, P.kt - kSf * ks) * kSfTile;
          mbar_expect_tx(&full[s], C::kATile + C::kBTile + 2 * sf_bytes);
          tma_load_4d(st, &map_w, ks * 128, 0, wrow, t.g, &full[s]);
          bulk_load(st + C::kATile + C::kBTile, ws + ks * kSf * kSfTile, sf_bytes, &full[s]);
        }
        __syncwarp();
      };
      auto load_a = [&](int ks, int s) {
        if (elect_one()) {
          uint8_t* st = smem + s * C::kStage;
          const uint32_t sf_bytes = min(kSf, P.kt - kSf * ks) * kSfTile;
          tma_load_2d(st + C::kATile, &map_a, ks * 128, t.row0, &full[s]);
          bulk_load(st + C::kATile + C::kBTile + kSf * kSfTile, as + ks * kSf * kSfTile, sf_bytes, &full[s]);
        }
        __syncwarp();
      };
      int ks = k0;
      if (!waited) {
        // the first stages' weights do not depend on the kernel that quantises the rows
        const int early = min(kStages, k1 - k0);
        for (int i = 0; i < early; ++i) load_w(k0 + i, i);
        griddep_wait();
        griddep_launch_dependents();
        waited = true;
        for (; g < early; ++ks, ++g, ring.next())
          if (!(P.fault && blockIdx.x == 0 && g == 0)) load_a(ks, g);
      }
      for (; ks < k1; ++ks, ++g, ring.next()) {
        if (!warp_wait(&empty[ring.s], ring.phase ^ 1, abort_flag, P)) {
          ok = false;
          break;
        }
        load_w(ks, ring.s);
        load_a(ks, ring.s);
      }
    }
    if (!waited) griddep_wait();  // no CTA ends before the kernel ahead: what follows this launch may rely on both
    // every issued copy has landed before shared memory is given back
    __syncwarp();
    for (int q = g > kStages ? g - kStages : 0; q < g; ++q)
      mbar_wait_drain(&full[q % kStages], (q / kStages) & 1, P.err, kErrWaitTimeout, P.wait_ns);
  } else if (warp == 1) {
    Item t{};
    Ring<kStages> ring;
    int li = 0;
    bool ok = true;
    const uint32_t lo0 = desc_lo(smem_u32(smem));
    for (int it = first; it < items && ok; it += step, ++li) {
      item_at<NT>(t, it, P.mblocks, off, pre, P.E);
      const int b = li & 1, use = li >> 1;
      if (!warp_wait(&acc_empty[b], (use & 1) ^ 1, abort_flag, P)) break;
      const uint32_t d_tmem = tmem + b * NT;
      const int n_mma = (t.n + 15) & ~15;
      uint32_t id[4];
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) id[kk] = idesc_mx<F>(kBM, n_mma, kk);
      const uint32_t shift = (t.local & 127) >> 5;  // a 64-row tile may start in the middle of a scale tile
      for (int ks = k0; ks < k1; ++ks, ring.next()) {
        if (!warp_wait(&full[ring.s], ring.phase, abort_flag, P)) {
          ok = false;
          break;
        }
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        if (elect_one()) {
          const uint32_t lo = lo0 + ring.s * (C::kStage >> 4);
          const uint32_t a_lo = lo | kDescLoSw128, b_lo = (lo + (C::kATile >> 4)) | kDescLoSw128;
          const uint32_t sf_lo = lo + ((C::kATile + C::kBTile) >> 4);
          const uint32_t sf_t = sf_base + ring.s * C::kSfCols;
          // the weights' K chunks (128 elements each), then the token rows'; a chunk past the end of K copies
          // what the stage holds, and no MMA uses it
#pragma unroll
          for (int i = 0; i < 2 * kSf; ++i) tmem_cp_scales<1>(sf_t + 4 * i, sf_lo + i * (kSfTile >> 4));
          const int steps = (P.K - ks * kStageK + F::kMmaK - 1) / F::kMmaK;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const int sf = 4 * (kk * F::kMmaK / 128);  // columns of this MMA's scale tile
            if (kk < steps)
              umma_mx<F, 1>(d_tmem, desc(a_lo + 2 * kk, kDescHiSw128), desc(b_lo + 2 * kk, kDescHiSw128), id[kk],
                            sf_t + sf, sf_t + 4 * kSf + sf + shift, kk > 0 ? 1u : (uint32_t)(ks - k0));
          }
          umma_commit(&empty[ring.s]);
          if (ks == k1 - 1) umma_commit(&acc_full[b]);
        }
        __syncwarp();
      }
    }
    __syncwarp();
    if (elect_one()) umma_commit(mma_done);
    __syncwarp();
    mbar_wait_drain(mma_done, 0, P.err, kErrWaitTimeout, P.wait_ns);
  } else if (warp >= 4) {
    using E = Epilogue<F32, SW>;
    E e(P, warp, lane);
    Item t{};
    int li = 0;
    bool ok = true;  // no wait of this warp has run out
    for (int it = first; it < items; it += step, ++li) {
      item_at<NT>(t, it, P.mblocks, off, pre, P.E);
      const int b = li & 1, use = li >> 1;
      const int f0 = t.mb * E::kFeatures, nf = min(E::kFeatures, P.n_out - f0);
      ok = ok && warp_wait(&acc_full[b], use & 1, abort_flag, P);
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      if (SPLIT) {
        // [token][weight row] to the stages' memory: all copies have landed and all MMAs that read it are done
        float* const part = reinterpret_cast<float*>(smem);
        for (int c0 = e.h * kTokens; ok && c0 < t.n; c0 += 2 * kTokens) {
          uint32_t v[kTokens];
          tmem_ld32_async(tmem + ((uint32_t)(e.q * 32) << 16) + c0, v);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
          for (int j = 0; j < kTokens; ++j) part[(c0 + j) * kPartPitch + e.q * 32 + lane] = __uint_as_float(v[j]);
        }
      } else {
        ok = e.item(P.y, tmem + b * NT, t.row0, t.n, f0, nf, 0, ok, li, [&](bool, bool last) {
          if (last && lane == 0) mbar_arrive(&acc_empty[b]);
        });
      }
    }
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  if (SPLIT) {
    cluster_sync();  // every CTA's partial sums (and its abort flag) are written
    Item t{};
    if (first < items) {
      item_at<NT>(t, first, P.mblocks, off, pre, P.E);
      sum_parts<F32, SW>(P, smem_u32(smem), smem_u32(const_cast<int*>(abort_flag)), rank, t.row0, t.n, t.mb, warp, lane);
    }
    cluster_sync();  // no CTA leaves while another may still read its sums
  }
  if (warp == 1) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
}

template <typename F>
constexpr int code_bytes(int K) {  // of a row
  return F::kMmaK == 64 ? K / 2 : K;
}

template <typename F>
bool make_w_map(const moe_fp4_mm_dims& d, const uint8_t* w, CUtensorMap* map) {
  const uint32_t pair = d.swiglu ? 2 : 1;
  const uint64_t row = code_bytes<F>(d.K);
  const uint64_t dims[4] = {row, pair, (uint64_t)d.N / pair, (uint64_t)d.E};
  const uint64_t strides[3] = {(d.N / pair) * row, row, (uint64_t)d.N * row};
  const uint32_t box[4] = {128, pair, 128 / pair, 1};
  return make_map_4d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, w, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <typename F>
bool make_a_map(const moe_fp4_mm_dims& d, const uint8_t* a, int rows, CUtensorMap* map) {
  const uint64_t row = code_bytes<F>(d.K);
  return make_map_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, a, row, d.M, row, 128, rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <typename F, int NT, bool F32, bool SW>
cudaError_t launch_as(const CUtensorMap& map_w, const CUtensorMap& map_a, const MmParams& P, int items,
                      cudaStream_t st) {
  auto* k = P.split > 1 ? mm_kernel<F, NT, F32, SW, true> : mm_kernel<F, NT, F32, SW, false>;
  const cudaError_t e = ensure_smem_optin(reinterpret_cast<const void*>(k), Cfg<F, NT>::kSmem);
  if (e != cudaSuccess) return e;
  const int grid = P.split > 1 ? items * P.split : std::min(items, num_sms());
  return launch_cluster_early(k, grid, P.split, kThreads, Cfg<F, NT>::kSmem, st, map_w, map_a, P);
}

template <typename F, int NT>
cudaError_t launch_nt(const moe_fp4_mm_dims& d, const uint8_t* a, const uint8_t* w, const MmParams& P,
                      cudaStream_t st) {
  CUtensorMap map_w, map_a;
  if (!make_w_map<F>(d, w, &map_w) || !make_a_map<F>(d, a, NT, &map_a)) return cudaErrorInvalidValue;
  // exactly, or for groups at most
  const int64_t tiles = P.offsets ? (int64_t)d.M / NT + std::min(d.E, d.M) : ((int64_t)d.M + NT - 1) / NT;
  const int items = (int)std::min<int64_t>(tiles * P.mblocks, INT32_MAX);
  if (P.f32)
    return P.swiglu ? launch_as<F, NT, true, true>(map_w, map_a, P, items, st)
                    : launch_as<F, NT, true, false>(map_w, map_a, P, items, st);
  return P.swiglu ? launch_as<F, NT, false, true>(map_w, map_a, P, items, st)
                  : launch_as<F, NT, false, false>(map_w, map_a, P, items, st);
}

template <typename F>
cudaError_t launch_pairs(const moe_fp4_mm_dims& d, const uint8_t* a, const uint8_t* w, const MmParams& P,
                         cudaStream_t st) {
  CUtensorMap map_w, map_a, map_a128, map_ws, map_as;
  const uint64_t ws_tiles = (uint64_t)d.E * P.mblocks * P.kt, as_tiles = (uint64_t)(d.M / 128 + d.E) * P.kt;
  if (!make_w_map<F>(d, w, &map_w) || !make_a_map<F>(d, a, 32, &map_a) || !make_a_map<F>(d, a, 128, &map_a128) ||
      !make_map_2d(&map_ws, CU_TENSOR_MAP_DATA_TYPE_INT32, P.w_scales, kSfTile / 4, ws_tiles, kSfTile, kSfTile / 4, F::kSfTiles,
                   CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !make_map_2d(&map_as, CU_TENSOR_MAP_DATA_TYPE_INT32, P.a_scales, kSfTile / 4, as_tiles, kSfTile, kSfTile / 4, F::kSfTiles,
                   CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;
  return launch_mm_pairs<F>(map_w, map_a, map_a128, map_ws, map_as, P, st);
}

int check_mm(const moe_fp4_mm_dims& d) {
  if (d.M < 0 || d.N < 1 || d.K <= 0 || d.K % 32 != 0 || d.K > 32768 || d.E < 1 || d.E > kMaxGroups ||
      d.swiglu < 0 || d.swiglu > 1 || (d.swiglu && d.N % 2 != 0) ||
      (d.y_type != MOE_FP4_TYPE_BF16 && d.y_type != MOE_FP4_TYPE_F32))
    return MOE_FP4_ERR_INVALID_ARG;
  // item counts and tensor-map extents stay below 2^31
  const int64_t mb = ((int64_t)d.N + 127) / 128;
  if (d.N > kMaxFeatures || (int64_t)d.M * d.K >= (1LL << 35) || ((int64_t)d.M / 64 + d.E) * mb >= (1LL << 30)) return MOE_FP4_ERR_UNSUPPORTED;
  return MOE_FP4_OK;
}

int check_mm_pointers(const moe_fp4_mm_dims& d, const void* w, const void* ws, const void* y, const void* offsets) {
  if (!w || !ws || !y || (!offsets && d.E != 1)) return MOE_FP4_ERR_INVALID_ARG;
  const uintptr_t ya = d.y_type == MOE_FP4_TYPE_F32 ? 3 : 1;
  if (((uintptr_t)w & 15) || ((uintptr_t)ws & 15) || ((uintptr_t)y & ya) || ((uintptr_t)offsets & 3))
    return MOE_FP4_ERR_INVALID_ARG;
  return MOE_FP4_OK;
}

MmParams params(const moe_fp4_mm_dims& d, const uint8_t* as, const int32_t* offsets, const uint8_t* ws, void* y) {
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
  P.vec = P.n_out % 2 == 0 && ((uintptr_t)y & 3) == 0;
  P.split = 1;
  P.fault = fault_site() == MOE_FP4_FAULT_TC_TOKEN_TILE;
  P.wait_ns = wait_limit_ns();
  return P;
}

// Few rows of one matrix have a kernel of their own, which quantises them itself and needs no workspace: that, the
// interface's promise, decides, whatever N is.  16 x 4096 x 4096 takes 5.8 us in it, 17 rows in the others 6.2; one row
// 4.8.  With a wide N it is the slower one: 16 x 16384 x 4096 11.1 us, 17 rows 8.7.
bool few_rows(const moe_fp4_mm_dims& d, const int32_t* offsets) { return !offsets && d.M <= kFewRows; }

template <typename F>
cudaError_t launch_few(const moe_fp4_mm_dims& d, const MmParams& P, const MxRows* x, const uint8_t* codes,
                       const uint8_t* w, cudaStream_t st) {
  CUtensorMap map_w;
  if (!make_w_map<F>(d, w, &map_w)) return cudaErrorInvalidValue;
  return launch_mm_few<F>(map_w, P, x, codes, st);
}

// The kernel and tile of a product with more than a few rows: the one whose
// time, rounds over the SMs x (stages x time of a stage + fixed time of an
// item), is least.  Fitted in us to products of 64 .. 13073 rows, N = 512 .. 8192, K
// = 128 .. 4096, with and without SwiGLU, and of ragged groups of 32 .. 1000 rows: a
// stage takes 0.23, 0.24 and 0.25, an item 0.6, 1.05 and 2.2 (SwiGLU 2.8) beside
// them, with tiles of 128 weight rows x 64 and 128 token rows on an SM and of 256 x
// 256 on a pair; the kernels' fixed times differ by 0.15 and 1.3.  (The choice is
// off the best of the three by 0.3% in the mean and 15% at most.  M = 256, N = K =
// 4096: 9.4, 10.1 and 13.6 us; M = N = 4096, K = 2048: 35, 22 and 18; M = 8192, N =
// 4096, K = 128: 24, 19 and 19.)  The tiles of a group are estimated from the mean of the
// groups' rows, half a standard deviation of a uniform routing taken off.  A
// dense product may split K over clusters of 2 or 4 CTAs (of 8, too few fit the
// GPCs: 32 x 4096 x 2048 10 us), which costs 0.8 and 0.017 a token row.  (N = K =
// 4096: M = 17 8.0 -> 6.3, 64 8.0 -> 7.1; K = 8192: M = 64 11.6 -> 8.7 us.)
struct Choice {
  int rows, split;
};

template <typename F>
Choice choose_tile(const moe_fp4_mm_dims& d, bool grouped) {
  const int nks = (d.K + F::kStageK - 1) / F::kStageK, sms = num_sms();
  const double mean = (double)d.M / d.E;
  double best = 0;
  Choice choice{0, 1};
  const struct {
    int rows, wrows, sms;
    double stage, item, launch;
  } kernels[] = {{64, 128, 1, 0.23, 0.6, 0}, {128, 128, 1, 0.24, 1.05, 0.15}, {256, 256, 2, 0.25, d.swiglu ? 2.8 : 2.2, 1.3}};
  for (const auto& k : kernels) {
    const double rows = grouped ? std::max(mean - 0.5 * std::sqrt(mean), 1.0) : mean;
    const double tiles = std::min(std::ceil(rows / k.rows) * d.E, (double)d.M);
    const double items = tiles * ((d.N + k.wrows - 1) / k.wrows);
    for (int split = 1; split <= 4; split *= 2) {
      if (split > 1 && (grouped || k.sms > 1 || split * items > 0.85 * sms || nks < 2 * split)) break;
      const double t = k.launch + (split > 1 ? 0.8 + 0.017 * std::min(d.M, k.rows) : 0) +
                       std::ceil(items * k.sms / sms) * ((nks + split - 1) / split * k.stage + k.item);
      if (choice.rows == 0 || t < best) best = t, choice = {k.rows, split};
    }
  }
  return choice;
}

// rows_ahead: the kernel ahead of this one quantises the rows, to a and as
template <typename F>
cudaError_t launch_mm(const moe_fp4_mm_dims& d, const uint8_t* a, const uint8_t* as, const int32_t* offsets,
                      const uint8_t* w, const uint8_t* ws, void* y, bool rows_ahead, cudaStream_t st) {
  MmParams P = params(d, as, offsets, ws, y);
  P.rows_ahead = rows_ahead;
  if (few_rows(d, offsets)) return launch_few<F>(d, P, nullptr, a, w, st);
  const Choice c = choose_tile<F>(d, offsets != nullptr);
  P.split = c.split;
  switch (c.rows) {
    case 64: return launch_nt<F, 64>(d, a, w, P, st);
    case 128: return launch_nt<F, 128>(d, a, w, P, st);
    default: return launch_pairs<F>(d, a, w, P, st);
  }
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

// Bytes of the lists with which rows of x that are used several times are
// quantised once; 0 where that does not pay, having two launches more.  Quantiser and
// a product of 64 features, every row gathered / each source row once, us: 36864 rows of 2048
// with 8 uses each 32.1 / 23.5, 65536 of 512 with 2 uses 35.7 / 31.6, 32768 of 512 with 4 19.8 /
// 16.9, 9362 of 7168 with 4 30.0 / 26.0, 16384 of 1024 with 8 12.9 / 13.5; below the bounds
// 16384 of 512 with 8 11.9 / 12.3, 8192 of 4096 with 8 18.4 / 20.5, 65536 of 256 with 4 24.0 / 25.3.
// Beyond a mean of 32 uses most places would be on the shared list.
size_t once_bytes(const MxRows& R) {
  if (!R.row_index || R.rows < 2 * R.x_rows || R.rows > 32 * R.x_rows || R.K < 512) return 0;
  const int64_t n = R.rows * R.K;
  if (!(R.rows >= (1 << 14) && n >= (1LL << 24)) && !(R.rows >= (1 << 13) && n >= (3LL << 24))) return 0;
  return (size_t)once_lists(R) * sizeof(int32_t);
}

}  // namespace

cudaError_t ops_mm_error(int32_t** word) { return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_mm_err); }

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
  return launch_mm<Fp4>(d, a, a_scales, offsets, w, w_scales, y, false, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess
             ? MOE_FP4_OK
             : MOE_FP4_ERR_CUDA;
}

size_t moe_fp4_mxfp4_linear_workspace_bytes(const moe_fp4_mm_dims* dims) {
  if (!dims || check_mm(*dims) != MOE_FP4_OK) return 0;
  return align256((size_t)dims->M * (dims->K / 2)) + moe_fp4_mxfp4_tiled_scale_bytes(dims->M, dims->E, dims->K);
}

size_t moe_fp4_mxfp4_gathered_workspace_bytes(const moe_fp4_mm_dims* dims, int64_t x_rows) {
  const size_t base = moe_fp4_mxfp4_linear_workspace_bytes(dims);
  if (base == 0 || x_rows < 0) return 0;
  MxRows R{};
  int32_t any = 0;
  R.row_index = &any;
  R.rows = dims->M;
  R.x_rows = x_rows;
  R.K = dims->K;
  const size_t once = once_bytes(R);
  return once == 0 ? base : align256(base) + once;
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
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (few_rows(d, offsets))
    return launch_few<Fp4>(d, params(d, nullptr, nullptr, w_scales, y), &R, nullptr, w, st) == cudaSuccess ? MOE_FP4_OK
                                                                                                     : MOE_FP4_ERR_CUDA;
  if (!workspace || ((uintptr_t)workspace & 255)) return MOE_FP4_ERR_INVALID_ARG;
  if (workspace_bytes < moe_fp4_mxfp4_linear_workspace_bytes(dims)) return MOE_FP4_ERR_WORKSPACE;
  uint8_t* codes = static_cast<uint8_t*>(workspace);
  uint8_t* scales = codes + align256((size_t)d.M * (d.K / 2));
  const size_t base = align256(moe_fp4_mxfp4_linear_workspace_bytes(dims)), once = once_bytes(R);
  const cudaError_t e =
      once != 0 && workspace_bytes >= base + once
          ? launch_mxfp4_quantize_once(R, reinterpret_cast<int32_t*>(codes + base), codes, scales, st)
          : launch_mxfp4_quantize(R, codes, scales, true, true, st);
  if (e != cudaSuccess) return MOE_FP4_ERR_CUDA;
  return launch_mm<Fp4>(d, codes, scales, offsets, w, w_scales, y, true, st) == cudaSuccess ? MOE_FP4_OK : MOE_FP4_ERR_CUDA;
}

size_t moe_fp4_fp8_linear_workspace_bytes(const moe_fp4_mm_dims* dims) {
  if (!dims || check_mm(*dims) != MOE_FP4_OK) return 0;
  return align256((size_t)dims->M * dims->K) + moe_fp4_mxfp4_tiled_scale_bytes(dims->M, dims->E, dims->K);
}

int moe_fp4_fp8_linear(const moe_fp4_mm_dims* dims, const void* x, int x_type, int64_t x_rows, int64_t x_stride,
                       const int32_t* offsets, const uint8_t* w, const uint8_t* w_scales, void* y, void* workspace,
                       size_t workspace_bytes, void* cuda_stream) {
  if (!dims || (x_type != MOE_FP4_TYPE_BF16 && x_type != MOE_FP4_TYPE_F32)) return MOE_FP4_ERR_INVALID_ARG;
  const moe_fp4_mm_dims d = *dims;
  int rc = check_mm(d);
  if (rc != MOE_FP4_OK) return rc;
  const MxRows R{x, x_rows, x_stride, nullptr, offsets, d.M, d.K, 1, d.E, x_type == MOE_FP4_TYPE_F32};
  rc = check_mx_rows(R);
  if (rc != MOE_FP4_OK || d.M == 0) return rc;
  rc = check_mm_pointers(d, w, w_scales, y, offsets);
  if (rc != MOE_FP4_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (few_rows(d, offsets))
    return launch_few<Fp8>(d, params(d, nullptr, nullptr, w_scales, y), &R, nullptr, w, st) == cudaSuccess
               ? MOE_FP4_OK
               : MOE_FP4_ERR_CUDA;
  if (!workspace || ((uintptr_t)workspace & 255)) return MOE_FP4_ERR_INVALID_ARG;
  if (workspace_bytes < moe_fp4_fp8_linear_workspace_bytes(dims)) return MOE_FP4_ERR_WORKSPACE;
  uint8_t* codes = static_cast<uint8_t*>(workspace);
  uint8_t* scales = codes + align256((size_t)d.M * d.K);
  if (launch_fp8_quantize(R, codes, scales, st) != cudaSuccess) return MOE_FP4_ERR_CUDA;
  return launch_mm<Fp8>(d, codes, scales, offsets, w, w_scales, y, true, st) == cudaSuccess ? MOE_FP4_OK
                                                                                           : MOE_FP4_ERR_CUDA;
}

}  // extern "C"
