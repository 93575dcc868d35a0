// Dense products of MXFP4 matrices for few rows (a decoded token, a small
// batch): y = a w^T with M <= 16.
//
// The time is that of reading w once, and for most layers less than that: a
// launch and a chain of latencies.  So everything is in one kernel.  Rows that
// come unquantised are quantised by the warps that later do the epilogue,
// straight into the stages the tensor core reads (each CTA needs its share of K
// alone, so that little work is done twice), while the weights are on their
// way; and K is split over the CTAs of a cluster, as many as fill the SMs,
// whose partial sums are added in rank order through distributed shared memory.
// One token, 4096 x 4096 with SwiGLU: 4.9 us, against 8.8 us for a quantiser and
// a product without the split.
//
// Tile, scales and SwiGLU as in mxfp4_mm.cu.  Warps: 0 the TMA producer of the
// weights (its first stages are under way before tensor memory is allocated),
// 1 the MMA issuer, 4..11 the writers of the rows and the epilogue.  Waits are
// bounded; every copy has landed and every MMA completed before memory is given
// back.
#include <cuda.h>

#include <algorithm>

#include "mxfp4_mm.cuh"

namespace moe_fp4 {
namespace {

using namespace tc;
using namespace mm;

__device__ int32_t g_mm1_err[4];

constexpr int kThreads = 384;
constexpr int kWriters = 8;
constexpr int kRows = kFewRows;
constexpr int kATile = kBM * 128;
constexpr int kBTile = kRows * 128;
constexpr int kStage = kATile + kBTile + 4 * kSfTile;
// Ring stages: 5 where a CTA has no more (two CTAs then fit an SM, and the next
// launch is set up while this one runs), else 10.
template <int S>
struct Cfg {
  static constexpr int kOffPart = S * kStage;
  static constexpr int kOffBar = kOffPart + kRows * kPartPitch * 4;
  static constexpr int kSmem = kOffBar + 512 + 1024;
  static_assert(kSmem <= (S <= 5 ? kSmemMax / 2 : kSmemMax) && kRows + 16 * S <= 256, "layout");
};
constexpr uint32_t kCols1 = 256;     // tensor memory: 16 accumulator columns, 16 of scales a stage
static_assert(kStage % 1024 == 0, "stages stay 1 KB aligned for the 128-byte swizzle");

struct Mm1Params {
  MmParams m;
  const void* x;             // rows: bf16, fp32 or codes
  int64_t x_rows, x_stride;  // stride in elements (codes: in elements too, two a byte)
  const int32_t* row_index;
  int div, align;            // align: MxRows::align()
};

// SRC 0: bf16 rows, 1: fp32 rows, 2: codes with tiled scales
template <int kStages, int SRC, bool F32, bool SW>
__global__ void __launch_bounds__(kThreads, kStages <= 5 ? 2 : 1)
mm1_kernel(const __grid_constant__ CUtensorMap map_w, Mm1Params Q) {
  MmParams& P = Q.m;
  P.err = &g_mm1_err[0];
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* part = reinterpret_cast<float*>(smem + Cfg<kStages>::kOffPart);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg<kStages>::kOffBar);  // [stage]: weights landed
  uint64_t* written = full + kStages;                            // [stage]: rows written
  uint64_t* empty = written + kStages;                           // [stage]: its MMAs completed
  uint64_t* acc_full = empty + kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = warp_index(), lane = threadIdx.x & 31;
  const int rank = uniform((int)cluster_rank());
  const int mb = blockIdx.x / P.split;
  const int nks = (P.K + kStageK - 1) / kStageK;
  const int k0 = (int)((int64_t)nks * rank / P.split), k1 = (int)((int64_t)nks * (rank + 1) / P.split);

  auto load_weights = [&](int ks, int s) {
    if (elect_one()) {
      uint8_t* st = smem + s * kStage;
      const uint32_t sf_bytes = min(2, P.kt - 2 * ks) * kSfTile;
      mbar_expect_tx(&full[s], kATile + sf_bytes);
      tma_load_4d(st, &map_w, ks * 128, 0, mb * (SW ? 64 : 128), 0, &full[s]);
      bulk_load(st + kATile + kBTile, P.w_scales + ((size_t)mb * P.kt + 2 * ks) * kSfTile, sf_bytes, &full[s]);
    }
    __syncwarp();
  };

  if (warp == 0) {
    if (lane == 0) {
      for (int s = 0; s < kStages; ++s) {
        mbar_init(&full[s], 1);
        mbar_init(&written[s], kWriters);
        mbar_init(&empty[s], 1);
      }
      mbar_init(acc_full, 1);
      *abort_flag = 0;
      mbar_fence_init();
    }
    __syncwarp();
    griddep_wait();
    for (int i = 0; i < min(kStages, k1 - k0); ++i)
      if (!(P.fault && blockIdx.x == 0 && i == 0)) load_weights(k0 + i, i);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kCols1));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  griddep_begin();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
  const uint32_t sf_base = tmem + kRows;

  if (warp == 0) {
    Ring<kStages> ring;
    int g = min(kStages, k1 - k0);
    bool ok = true;
    for (; g < k1 - k0 && ok; ++g, ring.next()) {
      ok = warp_wait(&empty[ring.s], ring.phase, abort_flag, P);
      if (ok) load_weights(k0 + g, ring.s);
    }
    if (!ok) --g;
    // every issued copy has landed before shared memory is given back
    for (int q = g > kStages ? g - kStages : 0; q < g; ++q)
      mbar_wait_drain(&full[q % kStages], (q / kStages) & 1, P.err, kErrWaitTimeout, P.wait_ns);
  } else if (warp == 1) {
    Ring<kStages> ring;
    const uint32_t lo0 = desc_lo(smem_u32(smem));
    const uint32_t id0 = idesc_mxf4(kBM, kRows, 0), id1 = idesc_mxf4(kBM, kRows, 1);
    for (int ks = k0; ks < k1; ++ks, ring.next()) {
      if (!warp_wait(&written[ring.s], ring.phase, abort_flag, P) ||
          !warp_wait(&full[ring.s], ring.phase, abort_flag, P))
        break;
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      if (elect_one()) {
        const uint32_t lo = lo0 + ring.s * (kStage >> 4);
        const uint32_t a_lo = lo | kDescLoSw128, b_lo = (lo + (kATile >> 4)) | kDescLoSw128;
        const uint32_t sf_lo = lo + ((kATile + kBTile) >> 4);
        const uint32_t sf_t = sf_base + ring.s * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i)  // weights' two K chunks, then the rows'
          tmem_cp_scales<1>(sf_t + 4 * i, sf_lo + i * (kSfTile >> 4));
        const int steps = (P.K - ks * kStageK + 63) / 64;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          if (kk < steps)
            umma_mxf4<1>(tmem, desc(a_lo + 2 * kk, kDescHiSw128), desc(b_lo + 2 * kk, kDescHiSw128),
                         (kk & 1) ? id1 : id0, sf_t + 4 * (kk >> 1), sf_t + 8 + 4 * (kk >> 1),
                         kk > 0 ? 1u : (uint32_t)(ks - k0));
        umma_commit(&empty[ring.s]);
      }
      __syncwarp();
    }
    if (elect_one()) umma_commit(acc_full);
    __syncwarp();
    mbar_wait_drain(acc_full, 0, P.err, kErrWaitTimeout, P.wait_ns);
  } else if (warp >= 4) {
    // ---------------- writers: rows into the stages ----------------
    // A pass covers 256 chunks of 16 elements (8 bytes of codes): 16 a row and
    // stage, so that with few rows one pass covers several stages.  A pass's
    // rows are loaded two passes before they are quantised.
    const int tid = threadIdx.x - 128;
    int per_log = 4;                                           // chunks of a stage: its rows, rounded up to a
    while ((16 << (per_log - 4)) < 16 * P.M) ++per_log;        // power of two, times 16
    const int group = min(1 << (8 - per_log), 4);              // stages of a pass
    const int sub = tid >> per_log, c = tid & 15, row = (tid & ((1 << per_log) - 1)) >> 4;
    const bool mine = sub < group && row < P.M;
    int64_t src = -1;                                          // first element of this thread's row, -1: a zero row
    if (mine) {
      src = row;
      if (SRC != 2 && Q.row_index) {
        src = Q.row_index[row];
        src = src < 0 ? -1 : src / Q.div;
        if (src < 0 || src >= Q.x_rows) {
          atomicOr(P.err, kErrBadExpertId);
          src = -1;
        }
      }
      if (src > 0) src *= Q.x_stride;
    }
    uint32_t next[2][16];
    auto load = [&](int ks, uint32_t (&raw)[16]) {  // this thread's chunk of the pass from stage ks on
#pragma unroll
      for (int j = 0; j < 16; ++j) raw[j] = 0;
      const int k = (ks + sub) * kStageK + c * 16;
      if (src < 0 || ks + sub >= k1 || k >= P.K) return;
      if (SRC == 2) {
        const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(Q.x) + (src + k) / 2);
        raw[0] = q.x, raw[1] = q.y;
        raw[2] = P.a_scales[(size_t)(k >> 7) * kSfTile + 16 * row + ((k >> 5) & 3)];
      } else if (Q.align == 32) {
        load16_raw<SRC == 1, 32>(Q.x, src + k, raw);
      } else if (Q.align == 16) {
        load16_raw<SRC == 1, 16>(Q.x, src + k, raw);
      } else {
        load16_raw<SRC == 1, 0>(Q.x, src + k, raw);
      }
    };
    load(k0, next[0]);
    load(k0 + group, next[1]);
    Ring<kStages> ring;
    bool ok = true;
    for (int ks = k0; ks < k1 && ok; ks += group) {
      const int here = min(group, k1 - ks);
      uint32_t cur[16], sb;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        cur[j] = next[0][j];
        next[0][j] = next[1][j];
      }
      load(ks + 2 * group, next[1]);
      uint2 q;
      if (SRC == 2) {
        q = make_uint2(cur[0], cur[1]);
        sb = cur[2];
      } else {
        q = quantize16<SRC == 1>(cur, sb);
      }
      // the stages of this pass are free
      Ring<kStages> at = ring;
      for (int i = 0; i < here && ok; ++i, at.next())
        if (ks - k0 + i >= kStages) ok = warp_wait(&empty[at.s], at.phase ^ 1, abort_flag, P);
      if (!ok) break;
      if (mine && sub < here) {
        uint8_t* st = smem + (ring.s + sub < kStages ? ring.s + sub : ring.s + sub - kStages) * kStage;
        // 128-byte swizzle: the 16-byte chunk at (c / 2) ^ (row % 8); past the end of K codes and scales are 0
        *reinterpret_cast<uint2*>(st + kATile + row * 128 + (((c >> 1) ^ (row & 7)) << 4) + (c & 1) * 8) = q;
        if ((c & 1) == 0) st[kATile + kBTile + (2 + (c >> 3)) * kSfTile + 16 * row + ((c >> 1) & 3)] = (uint8_t)sb;
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      for (int i = 0; i < here; ++i, ring.next())
        if (lane == 0) mbar_arrive(&written[ring.s]);
    }
    // ---------------- partial sums: [token][feature], fp32 ----------------
    if (warp < 8 && warp_wait(acc_full, 0, abort_flag, P)) {
      asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
      uint32_t v[32];
      const int q = warp & 3;
      tmem_ld32_async(tmem + ((uint32_t)(q * 32) << 16), v);
      asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
      for (int j = 0; j < kRows; ++j)
        if (j < P.M) part[j * kPartPitch + q * 32 + lane] = __uint_as_float(v[j]);
    }
  }
  __syncwarp();
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
  __syncthreads();
  cluster_sync();  // every CTA's partial sums (and its abort flag) are written
  sum_parts<F32, SW>(P, smem_u32(part), smem_u32(const_cast<int*>(abort_flag)), rank, 0, P.M, mb, warp, lane);
  cluster_sync();  // no CTA leaves while another may still read its sums
  if (warp == 1) {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols1));
  }
}

template <int S, int SRC, bool F32, bool SW>
cudaError_t launch_as(const CUtensorMap& map_w, const Mm1Params& Q, cudaStream_t st) {
  auto* k = mm1_kernel<S, SRC, F32, SW>;
  const cudaError_t e = ensure_smem_optin(reinterpret_cast<const void*>(k), Cfg<S>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_cluster_early(k, Q.m.mblocks * Q.m.split, Q.m.split, kThreads, Cfg<S>::kSmem, st, map_w, Q);
}

template <int SRC, bool F32, bool SW>
cudaError_t launch_stages(const CUtensorMap& map_w, const Mm1Params& Q, cudaStream_t st) {
  const int nks = (Q.m.K + kStageK - 1) / kStageK;
  return (nks + Q.m.split - 1) / Q.m.split <= 5 ? launch_as<5, SRC, F32, SW>(map_w, Q, st)
                                                : launch_as<10, SRC, F32, SW>(map_w, Q, st);
}

template <int SRC>
cudaError_t launch_src(const CUtensorMap& map_w, const Mm1Params& Q, cudaStream_t st) {
  if (Q.m.f32)
    return Q.m.swiglu ? launch_stages<SRC, true, true>(map_w, Q, st) : launch_stages<SRC, true, false>(map_w, Q, st);
  return Q.m.swiglu ? launch_stages<SRC, false, true>(map_w, Q, st) : launch_stages<SRC, false, false>(map_w, Q, st);
}

}  // namespace

cudaError_t launch_mm_few(const CUtensorMap& map_w, const MmParams& P, const MxRows* x, const uint8_t* codes,
                          cudaStream_t st) {
  Mm1Params Q{};
  Q.m = P;
  // CTAs of a cluster: as many as the SMs take, with two stages of K each at least
  const int nks = (P.K + kStageK - 1) / kStageK;
  Q.m.split = 1;
  while (Q.m.split < 8 && 2 * Q.m.split * P.mblocks <= num_sms() && 4 * Q.m.split <= nks) Q.m.split *= 2;
  if (x == nullptr) {
    Q.x = codes;
    Q.x_rows = P.M;
    Q.x_stride = P.K;
    return launch_src<2>(map_w, Q, st);
  }
  Q.x = x->x;
  Q.x_rows = x->x_rows;
  Q.x_stride = x->x_stride;
  Q.row_index = x->row_index;
  Q.div = x->div;
  Q.align = x->align();
  return x->f32 ? launch_src<1>(map_w, Q, st) : launch_src<0>(map_w, Q, st);
}

cudaError_t ops_mm1_error(int32_t** word) { return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_mm1_err); }

}  // namespace moe_fp4
