// Products of MXFP4 matrices on pairs of SMs (tcgen05 cta_group::2), for many
// token rows.
//
// The mathematics and the operands' way to the tensor core are those of the
// one-SM kernel (mxfp4_mm.cu); an MMA here covers two SMs: M = 256 weight rows,
// 128 in each CTA of a cluster pair, by up to 256 token rows, whose codes the
// CTAs hold half each.  What bounds the product of 128 x 256 tiles on one SM is
// shared memory: an MMA of K = 64 takes 129 cycles when the operands are there
// (measured), in which its 12 KB have to be written by the copies and read by
// the tensor core, 190 bytes a cycle; a pair needs 8 KB on each SM, 128 bytes a
// cycle.
//
// Tensor memory: two accumulators of 256 columns and three slots of scales
// (24 columns each: weights 2 x 4, tokens 2 x 8) are 72 columns more than there
// are, so the accumulators overlap: columns [0, 256) and [184, 440).  The
// epilogue reads the shared columns first and then releases them
// (`part_free`), so that the MMAs of the next item start while it reads the
// rest.  (Two whole accumulators of 192 columns instead: 8192 x 4096 x 8192 86 us
// against 82.)  Measured: 8192 x 4096 x 8192 80 us, 6.8 PFLOP/s; 16384 x 8192 x
// 8192 274 us, 8.0 PFLOP/s, what four times the measured bf16 rate comes to.  A
// layer's W2 for 256 experts of 144 rows each, K = 2048, N = 4096, is bound by
// HBM: 220 us, 6.6 TB/s.
//
// Roles, in both CTAs: warp 0 the TMA producer of the CTA's own codes (its 128
// weight rows, its half of the token rows), warp 2 that of the scales (issuing
// a copy takes ~80 cycles: one warp for both is slower than the MMAs), warp 1 of
// the leader (rank 0) the MMA issuer, warp 3 of the leader the issuer of the
// scales' copies to tensor memory (in one warp with the MMAs they made it the
// bound for tiles of fewer than 256 tokens), warps 4..11 the epilogue of the
// CTA's own accumulator lanes.  The follower's copies complete on the leader's barrier
// (its producers announce their bytes there), so that the issuer waits for
// both halves at once.  (A warp of the follower that waits and
// arrives on the leader's barrier instead needs ~1,300 cycles a stage for the
// cluster-wide release, more than twice the stage's MMAs: measured.)
//
// All waits are bounded; the producers leave the number of their issued stages
// in the leader, which waits for them and for the MMAs before either CTA gives
// memory back.
#include <cuda.h>

#include <algorithm>

#include "mxfp4_mm.cuh"

namespace moe_fp4 {
namespace {

using namespace tc;
using namespace mm;

__device__ int32_t g_mm2_err[4];

constexpr int kThreads = 384;
constexpr int kNT = 256;                                 // token rows per item
constexpr int kBoxRows = 32;                             // token rows per small TMA box; a large one has 128
constexpr int kATile = kBM * 128;
constexpr int kBTile = kNT / 2 * 128;                    // this CTA's half
constexpr int kFixed = 1024 + 512 + 2 * (kMaxGroups + 1) * 4;
constexpr uint32_t kAcc1 = 184;                          // first column of accumulator 1
constexpr uint32_t kSfBase = 440;
constexpr int kSfSlots = 3;
template <typename F>
struct Cfg {
  static constexpr int kSf = F::kSfTiles;
  // scales of a stage: weight tiles, and token tiles of two 128 rows (to whole KB)
  static constexpr int kStage = kATile + kBTile + (3 * kSf + (kSf & 1)) * kSfTile;
  static constexpr int kStages = (kSmemMax - kFixed) / kStage;
  static constexpr int kSmem = kStages * kStage + kFixed;
  static constexpr uint32_t kSfCols = 12 * kSf;
  static_assert(kStage % 1024 == 0 && kStages >= 4, "ring");
  static_assert(kSfBase + kSfSlots * kSfCols <= kTmemCols, "tensor memory columns");
};
static_assert(kNT - kAcc1 <= 128 - 32 && kNT - kAcc1 / 32 * 32 <= 128, "the shared columns are in the first round's reads");
static_assert(kSfBase >= kAcc1 + kNT, "tensor memory columns");

// Arrive on the barrier at the same offset in the leader CTA: this warp's reads
// of tensor memory have ended (tcgen05.wait::ld, the fence before it), and that
// is all the leader's MMAs wait for.
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
      "mbarrier.arrive.shared::cluster.b64 _, [a];\n}" ::"r"(smem_u32(bar))
      : "memory");
}
// the address, in the cluster's shared memory, of p's place in the leader CTA
__device__ __forceinline__ uint32_t in_leader(const void* p) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
  return r;
}
// announce `bytes` of this CTA's copies on a barrier of the cluster (an arrival)
__device__ __forceinline__ void expect_tx_cl(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
// TMA loads into this CTA that complete on a barrier of either CTA of the pair
__device__ __forceinline__ void tma2_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma2_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w,
                                             uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3, "
      "%4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}
// commit of this thread's MMAs to the barrier at this offset in both CTAs
__device__ __forceinline__ void commit_both(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

// ... of its tensor-core operations to a barrier of this CTA
__device__ __forceinline__ void commit_one(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

template <typename F, bool F32, bool SW>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
mm2_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_a,
           const __grid_constant__ CUtensorMap map_a128, const __grid_constant__ CUtensorMap map_ws,
           const __grid_constant__ CUtensorMap map_as, MmParams P) {
  P.err = &g_mm2_err[0];
  constexpr int kStage = Cfg<F>::kStage, kStages = Cfg<F>::kStages, kStageK = F::kStageK, kSf = F::kSfTiles;
  constexpr uint32_t kSfCols = Cfg<F>::kSfCols;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* tail = smem + kStages * kStage;
  uint64_t* full = reinterpret_cast<uint64_t*>(tail);    // [stage] leader: both CTAs' bytes landed
  uint64_t* empty = full + kStages;                      // [stage] both: the stage's MMAs completed
  uint64_t* acc_full = empty + kStages;                  // [2] both
  uint64_t* acc_empty = acc_full + 2;                    // [2] leader: both epilogues read all of the accumulator
  uint64_t* part_free = acc_empty + 2;                   // [2] leader: ... its columns that the other one shares
  uint64_t* sf_full = part_free + 2;                     // [slot] leader: a stage's scales are in tensor memory
  uint64_t* sf_done = sf_full + kSfSlots;                // leader
  uint64_t* mma_done = sf_done + 1;                      // both
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* issued = abort_flag + 1;                 // [4] leader: stages issued by each producer
  int* off = reinterpret_cast<int*>(tail + 512);
  int* pre = off + kMaxGroups + 1;
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int rank = uniform((int)cluster_rank());

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 4);  // one expect_tx of each producer, of both CTAs
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 2 * kEpiWarps);
      mbar_init(&part_free[b], 2 * kEpiWarps);
    }
    for (int i = 0; i < kSfSlots; ++i) mbar_init(&sf_full[i], 1);
    mbar_init(sf_done, 1);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  __syncwarp();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  // behind the quantiser of its rows (rows_ahead) only the rows are waited for, by their producers
  if (!P.rows_ahead) griddep_wait();
  if (warp == 4) group_tables<kNT>(P, off, pre, lane);
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are initialised
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
  const int mblocks2 = (P.mblocks + 1) / 2;  // pairs of 128-row blocks
  const int items = uniform(pre[P.E]) * mblocks2;
  const int nks = (P.K + kStageK - 1) / kStageK;
  const int first = blockIdx.x >> 1, step = gridDim.x >> 1;

  if (warp == 0 || warp == 2) {
    Item t{};
    Ring<kStages> ring;
    int g = 0;
    bool ok = true;
    griddep_begin();  // the kernel ahead writes the rows' codes and scales
    for (int it = first; it < items && ok; it += step) {
      item_at<kNT>(t, it, mblocks2, off, pre, P.E);
      const int mb = 2 * t.mb + rank;           // may be one past the last block: its rows read as 0,
      const int mb_sf = min(mb, P.mblocks - 1);  // with any scales
      const int half = ((t.n + 31) & ~31) / 2;   // token rows of this CTA
      const int boxes = half > 96 ? 0 : (half + kBoxRows - 1) / kBoxRows;  // 0: one large box
      const uint32_t b_bytes = boxes == 0 ? kBTile : boxes * kBoxRows * 128;
      const int wrow = mb * (SW ? 64 : 128), arow = t.row0 + rank * half;
      // first scale tiles: of the weight rows, of the token rows, of their next 128 (which may lie past the end)
      const int ws = (t.g * P.mblocks + mb_sf) * P.kt;
      const int as = ((uniform(off[t.g]) >> 7) + t.g + (t.local >> 7)) * P.kt;
      for (int ks = 0; ks < nks; ++ks, ++g, ring.next()) {
        if (!warp_wait(&empty[ring.s], ring.phase ^ 1, abort_flag, P)) {
          ok = false;
          break;
        }
        if (P.fault && blockIdx.x <= 1 && g == 0) continue;
        uint8_t* st = smem + ring.s * kStage;
        const uint32_t bar = in_leader(&full[ring.s]);
        if (warp == 0) {
          if (elect_one()) {
            expect_tx_cl(bar, kATile + b_bytes);
            tma2_load_4d(st, &map_w, ks * 128, 0, wrow, t.g, bar);
            if (boxes == 0)
              tma2_load_2d(st + kATile, &map_a128, ks * 128, arow, bar);
            else
              for (int i = 0; i < boxes; ++i)
                tma2_load_2d(st + kATile + i * kBoxRows * 128, &map_a, ks * 128, arow + i * kBoxRows, bar);
          }
        } else if (elect_one()) {
          // a stage's tiles a box; the second (Fp4) of the last stage may be the next row tile's: not used then
          uint8_t* sf = st + kATile + kBTile;
          expect_tx_cl(bar, 3 * kSf * kSfTile);
          tma2_load_2d(sf, &map_ws, 0, ws + kSf * ks, bar);
          tma2_load_2d(sf + kSf * kSfTile, &map_as, 0, as + kSf * ks, bar);
          tma2_load_2d(sf + 2 * kSf * kSfTile, &map_as, 0, as + P.kt + kSf * ks, bar);
        }
        __syncwarp();
      }
    }
    if (lane == 0)
      asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(in_leader(const_cast<int*>(&issued[rank * 2 + (warp >> 1)]))),
                   "r"(g)
                   : "memory");
  } else if (warp == 1) {
    // the follower's warp goes on to the cluster barrier below, where the
    // leader arrives once its MMAs, which read both CTAs' memory, are done
    if (rank == 0) {
      Item t{};
      Ring<kStages> ring;
      Ring<kSfSlots> slot;
      int li = 0, prev_n = 0;
      bool ok = true;
      const uint32_t lo0 = desc_lo(smem_u32(smem));
      for (int it = first; it < items && ok; it += step, ++li) {
        item_at<kNT>(t, it, mblocks2, off, pre, P.E);
        const int b = li & 1, use = li >> 1;
        const int n_mma = (t.n + 31) & ~31;
        // the other accumulator's columns that this one shares, where its item has values in them
        const bool shared = li > 0 && (b ? prev_n > (int)kAcc1 : n_mma > (int)kAcc1);
        prev_n = n_mma;
        if (!warp_wait(&acc_empty[b], (use & 1) ^ 1, abort_flag, P) ||
            (shared && !warp_wait(&part_free[b ^ 1], ((li - 1) >> 1) & 1, abort_flag, P)))
          break;
        const uint32_t d_tmem = tmem + b * kAcc1;
        uint32_t id[4];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) id[kk] = idesc_mx<F>(2 * kBM, n_mma, kk);
        for (int ks = 0; ks < nks; ++ks, ring.next(), slot.next()) {
          if (!warp_wait(&sf_full[slot.s], slot.phase, abort_flag, P)) {
            ok = false;
            break;
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          if (elect_one()) {
            const uint32_t lo = lo0 + ring.s * (kStage >> 4);
            const uint32_t a_lo = lo | kDescLoSw128, b_lo = (lo + (kATile >> 4)) | kDescLoSw128;
            const uint32_t sf_t = tmem + kSfBase + slot.s * kSfCols;
            const int steps = (P.K - ks * kStageK + F::kMmaK - 1) / F::kMmaK;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              const int c = kk * F::kMmaK / 128;  // this MMA's scale tile
              if (kk < steps)
                umma_mx<F, 2>(d_tmem, desc(a_lo + 2 * kk, kDescHiSw128), desc(b_lo + 2 * kk, kDescHiSw128), id[kk],
                              sf_t + 4 * c, sf_t + 4 * kSf + 8 * c, kk > 0 ? 1u : (uint32_t)ks);
            }
            commit_both(&empty[ring.s]);
            if (ks == nks - 1) commit_both(&acc_full[b]);
          }
          __syncwarp();
        }
      }
      __syncwarp();
      if (elect_one()) commit_both(mma_done);
      __syncwarp();
      mbar_wait_drain(mma_done, 0, P.err, kErrWaitTimeout, P.wait_ns);
    }
  } else if (warp == 3) {
    if (rank == 0) {
      // scales of each landed stage to a slot of tensor memory
      Ring<kStages> ring, behind;  // behind: the stage that last used this stage's slot
      Ring<kSfSlots> slot;
      const uint32_t lo0 = desc_lo(smem_u32(smem)) + ((kATile + kBTile) >> 4);
      int g = 0;
      bool ok = true;
      for (int it = first; it < items && ok; it += step)
        for (int ks = 0; ks < nks; ++ks, ++g, ring.next(), slot.next()) {
          if (!warp_wait(&full[ring.s], ring.phase, abort_flag, P)) {
            ok = false;
            break;
          }
          if (g >= kSfSlots) {  // the MMAs that read this slot have completed
            if (!warp_wait(&empty[behind.s], behind.phase, abort_flag, P)) {
              ok = false;
              break;
            }
            behind.next();
          }
          asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
          if (elect_one()) {
            const uint32_t sf_lo = lo0 + ring.s * (kStage >> 4);
            const uint32_t sf_t = tmem + kSfBase + slot.s * kSfCols;
#pragma unroll
            for (int c = 0; c < kSf; ++c) {
              tmem_cp_scales<2>(sf_t + 4 * c, sf_lo + c * (kSfTile >> 4));
              tmem_cp_scales<2>(sf_t + 4 * kSf + 8 * c, sf_lo + (kSf + c) * (kSfTile >> 4));
              tmem_cp_scales<2>(sf_t + 4 * kSf + 4 + 8 * c, sf_lo + (2 * kSf + c) * (kSfTile >> 4));
            }
            commit_one(&sf_full[slot.s]);
          }
          __syncwarp();
        }
      // every copy has completed before tensor memory is given back
      __syncwarp();
      if (elect_one()) commit_one(sf_done);
      __syncwarp();
      mbar_wait_drain(sf_done, 0, P.err, kErrWaitTimeout, P.wait_ns);
    }
  } else if (warp >= 4) {
    using E = Epilogue<F32, SW>;
    E e(P, warp, lane);
    Item t{};
    int li = 0;
    bool ok = true;  // no wait of this warp has run out
    for (int it = first; it < items; it += step, ++li) {
      item_at<kNT>(t, it, mblocks2, off, pre, P.E);
      const int b = li & 1, use = li >> 1;
      const int f0 = (2 * t.mb + rank) * E::kFeatures, nf = max(0, min(E::kFeatures, P.n_out - f0));
      ok = ok && warp_wait(&acc_full[b], use & 1, abort_flag, P);
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      // the columns shared with the other accumulator are read in the first round: accumulator 0's from kAcc1 on,
      // so its chunks are taken from there; accumulator 1's first 256 - kAcc1
      const int chunks = (t.n + kTokens - 1) / kTokens, from = kAcc1 / kTokens;
      const int start = b == 0 && chunks > from ? from : 0;
      ok = e.item(P.y, tmem + b * kAcc1, t.row0, t.n, f0, nf, start, ok, li, [&](bool round0, bool last) {
        if (lane != 0) return;
        if (round0) arrive_leader(&part_free[b]);
        if (last) arrive_leader(&acc_empty[b]);
      });
    }
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();  // every role has ended, in both CTAs
  if (rank == 0 && warp == 0) {
    // all copies of both CTAs have landed, if every item was done; if a wait ran out, what was issued is given
    // the time of a bounded wait
    const int g = max(max(issued[0], issued[1]), max(issued[2], issued[3]));
    for (int q = g > kStages ? g - kStages : 0; q < g; ++q)
      mbar_wait_drain(&full[q % kStages], (q / kStages) & 1, P.err, kErrWaitTimeout, P.wait_ns);
  }
  cluster_sync();  // no CTA leaves while its peer may still reach into it
  if (warp == 1) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
}

}  // namespace

namespace {

template <typename F, bool F32, bool SW>
cudaError_t launch_as(const CUtensorMap& map_w, const CUtensorMap& map_a, const CUtensorMap& map_a128,
                      const CUtensorMap& map_ws, const CUtensorMap& map_as, const MmParams& P, int pairs,
                      cudaStream_t st) {
  const cudaError_t e = ensure_smem_optin(reinterpret_cast<const void*>(mm2_kernel<F, F32, SW>), Cfg<F>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_early(mm2_kernel<F, F32, SW>, dim3(2 * pairs), dim3(kThreads), Cfg<F>::kSmem, st, map_w, map_a, map_a128, map_ws,
                      map_as, P);
}

}  // namespace

template <typename F>
cudaError_t launch_mm_pairs(const CUtensorMap& map_w, const CUtensorMap& map_a, const CUtensorMap& map_a128,
                            const CUtensorMap& map_ws, const CUtensorMap& map_as, const MmParams& P, cudaStream_t st) {
  const int64_t most = ((int64_t)P.M / kNT + std::min(P.E, P.M)) * ((P.mblocks + 1) / 2);
  const int pairs = (int)std::min<int64_t>(most, num_sms() / 2);
  if (P.f32)
    return P.swiglu ? launch_as<F, true, true>(map_w, map_a, map_a128, map_ws, map_as, P, pairs, st)
                    : launch_as<F, true, false>(map_w, map_a, map_a128, map_ws, map_as, P, pairs, st);
  return P.swiglu ? launch_as<F, false, true>(map_w, map_a, map_a128, map_ws, map_as, P, pairs, st)
                  : launch_as<F, false, false>(map_w, map_a, map_a128, map_ws, map_as, P, pairs, st);
}

template cudaError_t launch_mm_pairs<Fp4>(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                          const CUtensorMap&, const MmParams&, cudaStream_t);
template cudaError_t launch_mm_pairs<Fp8>(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                          const CUtensorMap&, const MmParams&, cudaStream_t);

cudaError_t ops_mm2_error(int32_t** word) { return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_mm2_err); }

}  // namespace moe_fp4
