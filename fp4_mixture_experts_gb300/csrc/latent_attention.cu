// Latent attention in its expanded form, for the new tokens of a ragged batch:
//
//   s[h, i, j] = scale (qn[i, h] . kn[j, h] + qr[i, h] . kr[j])     (128 and 64)
//   out[i, h] = sum_j softmax(s[h, i])_j v[j, h],                   j <= i + nk - nq
//
// kn and v of a head lie side by side, [Tk, H, 256], as the up projection of the
// latent vectors writes them; kr is one vector a token that all heads share: the
// third slab of every head's keys is loaded from there, so that no [Tk, H, 192]
// is ever put together.
//
// An item is 256 queries of a head, two tiles of 128 that take turns: while the
// tensor cores do one's P V and next Q K^T, the other's softmax runs (128 x 128
// scores are 512 + 768 cycles of MMAs and, at 16 exponentials a cycle, 1,024 of
// exponentials).  S lies in tensor memory, a query a lane, so that maximum and sum
// need no other thread; P overwrites it as bf16 and is the MMA's A operand from
// there; V is the B operand as it lies (MN-major).
//
// The running maximum moves only when a score exceeds it by more than 2^8: then a
// warp multiplies its lanes of O, in tensor memory, before it gives P to the MMAs;
// until then P may grow up to 2^8, which costs bf16 nothing.
//
// Shared memory: Q 2 x 3 slabs of [128][64] (96 KB), keys two stages of 3 slabs,
// values one of 2.  Warps: 0 loads, 1 issues the MMAs (and clears what the last tile
// of values holds behind the sequence's end: a zero of P must not meet an infinity
// there), 4..7 and 8..11 are the tiles' softmax and results.  Items are dealt out to
// one CTA an SM, long ones of a sequence first.  Waits are bounded; results are
// stored only by warps none of whose waits ran out.
#include <algorithm>

#include "latent.cuh"

namespace moe_fp4 {
namespace {

using namespace latent;
using tc::umma_commit;

__device__ int32_t g_attention_err[4];

constexpr int kThreads = 384;
constexpr int kQ = 128, kK = 128;             // queries and keys of a tile
constexpr int kSlab = 128 * 128;              // [128 rows][64 elements]
constexpr int kQSlabs = 3, kVSlabs = 2;
constexpr int kKStages = 2;
constexpr int kKStage = kQSlabs * kSlab, kVStage = kVSlabs * kSlab;
constexpr int kOffK = 2 * kQSlabs * kSlab;
constexpr int kOffV = kOffK + kKStages * kKStage;
constexpr int kOffTail = kOffV + kVStage;
constexpr int kSmem = kOffTail + 1024 + 1024;
static_assert(kSmem <= kSmemMax, "shared memory");
constexpr uint32_t kCols = 512;               // S of both tiles, O of both
constexpr uint32_t kColO = 256;
constexpr float kGrow = 8.f;                  // log2 of what P may grow to

struct AttentionParams {
  const int32_t* q_offsets;
  const int32_t* k_offsets;
  uint16_t* out;
  int32_t* err;
  int B, H, Tq, Tk;
  int causal;
  float scale_log2;
  int fault;
  uint64_t wait_ns;
};

// The items of a CTA, in ascending number: tile number x heads, tiles numbered
// through over the sequences.  Whole warp; 32 sequences at a time.
struct Items {
  int item, step;
  int base;               // first sequence of the 32 in the lanes
  int before;             // tiles before them
  int q0_, nq_, c_, end_; // this lane's sequence: first query, queries, its tiles, tiles up to its end
  // the item
  int h, q0, rows, k0, nk, lim[2], n[2];  // lim: keys that the first query of a tile sees; n: tiles of keys
  __device__ __forceinline__ void start(int first, int step_) {
    item = first - step_, step = step_, base = -32, before = 0, c_ = 0, end_ = 0;
  }
  __device__ __forceinline__ bool next(const AttentionParams& P) {
    const int lane = threadIdx.x & 31;
    item += step;
    const int tile = item / P.H;
    h = item - tile * P.H;
    while (tile >= __shfl_sync(0xFFFFFFFFu, end_, 31)) {
      before = __shfl_sync(0xFFFFFFFFu, end_, 31);
      base += 32;
      if (base >= P.B) return false;
      const int b = base + lane;
      q0_ = b < P.B ? min(max(P.q_offsets[b], 0), P.Tq) : 0;
      nq_ = b < P.B ? max(0, min(P.q_offsets[b + 1], P.Tq) - q0_) : 0;
      c_ = (nq_ + 2 * kQ - 1) / (2 * kQ);
      int s = c_;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, s, d);
        if (lane >= d) s += v;
      }
      end_ = before + s;
    }
    const int l = __popc(__ballot_sync(0xFFFFFFFFu, end_ <= tile));
    const int b = base + l;
    // the sequence's tiles from its end on: under a causal mask the long ones come first
    const int t = __shfl_sync(0xFFFFFFFFu, end_, l) - 1 - tile;
    const int nq = __shfl_sync(0xFFFFFFFFu, nq_, l);
    q0 = __shfl_sync(0xFFFFFFFFu, q0_, l) + t * 2 * kQ;
    rows = min(2 * kQ, nq - t * 2 * kQ);
    k0 = min(max(P.k_offsets[b], 0), P.Tk);
    nk = max(0, min(P.k_offsets[b + 1], P.Tk) - k0);
    k0 = uniform(k0), nk = uniform(nk);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = min(rows, (i + 1) * kQ) - i * kQ;  // queries of the tile
      lim[i] = P.causal ? t * 2 * kQ + i * kQ + 1 + nk - nq : nk;
      const int most = P.causal ? min(nk, lim[i] + r - 1) : nk;  // what its last one sees
      n[i] = r > 0 && most > 0 ? (most + kK - 1) / kK : 0;
    }
    return true;
  }
};

// Registers of a thread: the loads and MMAs give theirs up to the softmax, which
// holds a row of S.  The launch brings kThreads x 168 (checked before the first
// launch), the split asks for no more.
constexpr int kRegsFew = 72, kRegsMany = 208, kRegsLaunch = 168;
static_assert(128 * kRegsFew + 256 * kRegsMany <= kThreads * kRegsLaunch, "registers");
template <int R>
__device__ __forceinline__ void set_registers_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void set_registers_fewer() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

__global__ void __launch_bounds__(kThreads, 1)
latent_attention_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_kv,
                        const __grid_constant__ CUtensorMap map_rope, AttentionParams P) {
  P.err = &g_attention_err[0];
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* q_full = reinterpret_cast<uint64_t*>(smem + kOffTail);
  uint64_t* q_empty = q_full + 1;
  uint64_t* k_full = q_empty + 1;       // [stage]
  uint64_t* k_empty = k_full + kKStages;
  uint64_t* v_full = k_empty + kKStages;
  uint64_t* v_empty = v_full + 1;
  uint64_t* s_full = v_empty + 1;       // [tile]
  uint64_t* p_full = s_full + 2;        // [tile], four warps
  uint64_t* o_full = p_full + 2;        // [tile]
  uint64_t* o_free = o_full + 2;        // [tile], four warps
  uint64_t* mma_done = o_free + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1), mbar_init(q_empty, 1);
    for (int s = 0; s < kKStages; ++s) mbar_init(&k_full[s], 1), mbar_init(&k_empty[s], 1);
    mbar_init(v_full, 1), mbar_init(v_empty, 1);
    for (int t = 0; t < 2; ++t)
      mbar_init(&s_full[t], 1), mbar_init(&p_full[t], 4), mbar_init(&o_full[t], 1), mbar_init(&o_free[t], 4);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  __syncwarp();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  griddep_begin();
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
  const Waits wait{abort_flag, P.err, P.wait_ns};
  Items w;
  w.start(blockIdx.x, gridDim.x);

  if (warp < 4) {
    set_registers_fewer<kRegsFew>();
    if (warp == 0) {
      // ---------------- loads ----------------
      int items = 0, g = 0;  // items with keys, tiles of keys
      bool ok = true;
      while (ok && w.next(P)) {
        const int n = max(w.n[0], w.n[1]);
        if (n == 0) continue;
        if (!(ok = wait(q_empty, (items & 1) ^ 1))) break;
        const int tiles = w.rows > kQ ? 2 : 1;
        if (elect_one()) {
          mbar_expect_tx(q_full, tiles * kQSlabs * kSlab);
          for (int t = 0; t < tiles; ++t)
            for (int s = 0; s < kQSlabs; ++s)
              tma_load_3d(smem + (t * kQSlabs + s) * kSlab, &map_q, s * 64, w.h, w.q0 + t * kQ, q_full);
        }
        __syncwarp();
        ++items;
        for (int i = 0; i < n; ++i, ++g) {
          const int s = g % kKStages;
          if (!(ok = wait(&k_empty[s], ((g / kKStages) & 1) ^ 1))) break;
          if (!(P.fault && blockIdx.x == 0 && g == 0) && elect_one()) {
            uint8_t* st = smem + kOffK + s * kKStage;
            mbar_expect_tx(&k_full[s], kKStage);
            tma_load_3d(st, &map_kv, 0, w.h, w.k0 + i * kK, &k_full[s]);
            tma_load_3d(st + kSlab, &map_kv, 64, w.h, w.k0 + i * kK, &k_full[s]);
            tma_load_3d(st + 2 * kSlab, &map_rope, 0, 0, w.k0 + i * kK, &k_full[s]);
          }
          __syncwarp();
          if (!(ok = wait(v_empty, (g & 1) ^ 1))) {
            ++g;  // its keys are under way
            break;
          }
          if (elect_one()) {
            mbar_expect_tx(v_full, kVStage);
            tma_load_3d(smem + kOffV, &map_kv, 128, w.h, w.k0 + i * kK, v_full);
            tma_load_3d(smem + kOffV + kSlab, &map_kv, 192, w.h, w.k0 + i * kK, v_full);
          }
          __syncwarp();
        }
      }
      // every issued copy has landed before shared memory is given back
      __syncwarp();
      for (int q = max(0, g - kKStages); q < g; ++q) wait.drain(&k_full[q % kKStages], (q / kKStages) & 1);
      if (g > 0) wait.drain(v_full, (g - 1) & 1);
      if (items > 0) wait.drain(q_full, (items - 1) & 1);
    } else if (warp == 1) {
      // ---------------- MMAs ----------------
      const uint32_t base = smem_u32(smem);
      constexpr uint32_t id_qk = idesc_bf16(kQ, kK, false, false), id_pv = idesc_bf16(kQ, kValue, false, true);
      int items = 0, g = 0, use[2] = {0, 0}, turn[2] = {0, 0};  // of O's and of P's barriers
      bool ok = true;
      auto qk = [&](int t, int gk) {
        if (elect_one()) {
          const uint32_t q_lo = desc_lo(base + t * kQSlabs * kSlab, 16);
          const uint32_t k_lo = desc_lo(base + kOffK + (gk % kKStages) * kKStage, 16);
#pragma unroll
          for (int k = 0; k < (kNope + kRope) / 16; ++k) {
            const uint32_t at = ((k / 4) * kSlab + (k % 4) * 32) >> 4;
            umma_ss(tmem + t * kK, desc(q_lo + at), desc(k_lo + at), id_qk, k > 0);
          }
          umma_commit(&s_full[t]);
        }
        __syncwarp();
      };
      while (ok && w.next(P)) {
        const int n = max(w.n[0], w.n[1]);
        if (n == 0) continue;
        const bool clean = n * kK > w.nk;  // the last tile's end is behind the sequence's
        if (!(ok = wait(q_full, items & 1)) || !(ok = wait(&k_full[g % kKStages], (g / kKStages) & 1))) break;
        tmem_fence_after();
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (w.n[t] > 0) qk(t, g);
        if (elect_one()) {
          umma_commit(&k_empty[g % kKStages]);
          if (n == 1) umma_commit(q_empty);
        }
        __syncwarp();
        for (int i = 0; i < n && ok; ++i, ++g) {
          if (!(ok = wait(v_full, g & 1))) break;
          if (clean && i == n - 1) {
            const int from = w.nk - i * kK;
            for (int c = lane; c < (kK - from) * kVSlabs * 8; c += 32) {
              const int row = from + c / (kVSlabs * 8), s = (c >> 3) % kVSlabs;
              *reinterpret_cast<uint4*>(smem + kOffV + s * kSlab + row * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async();
            __syncwarp();
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (i >= w.n[t] || !ok) continue;
            ok = wait(&p_full[t], turn[t] & 1);
            if (ok && i == 0) ok = wait(&o_free[t], (use[t] & 1) ^ 1), ++use[t];
            if (!ok) break;
            ++turn[t];
            tmem_fence_after();
            if (elect_one()) {
              const uint32_t v_lo = desc_lo(base + kOffV, kSlab);
#pragma unroll
              for (int k = 0; k < kK / 16; ++k)
                tc::umma_tmem_a(tmem + kColO + t * kValue, tmem + t * kK + 8 * k, desc(v_lo + ((k * 2048) >> 4)), id_pv,
                                i > 0 || k > 0);
              if (i == w.n[t] - 1) umma_commit(&o_full[t]);
            }
            __syncwarp();
            if (i + 1 < w.n[t]) {
              if (!(ok = wait(&k_full[(g + 1) % kKStages], ((g + 1) / kKStages) & 1))) break;
              tmem_fence_after();
              qk(t, g + 1);
            }
          }
          if (!ok) break;
          if (elect_one()) {
            umma_commit(v_empty);
            if (i + 1 < n) umma_commit(&k_empty[(g + 1) % kKStages]);
            if (i + 2 == n) umma_commit(q_empty);
          }
          __syncwarp();
        }
        ++items;
      }
      __syncwarp();
      if (elect_one()) umma_commit(mma_done);
      __syncwarp();
      wait.drain(mma_done, 0);
    }
  } else {
    set_registers_more<kRegsMany>();
    // ---------------- softmax, rescaling, results ----------------
    const int t = (warp >> 2) - 1, row = (warp & 3) * 32 + lane;  // tile; this thread's query of it
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + t * kK + lanes, o_col = tmem + kColO + t * kValue + lanes;
    int turn = 0, use = 0;
    bool ok = true;
    while (ok && w.next(P)) {
      const int here = min(w.rows - t * kQ, kQ);  // queries of the tile
      const int seen = P.causal ? min(w.nk, w.lim[t] + row) : w.nk;  // keys that this query sees
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < w.n[t]; ++i, ++turn) {
        if (!(ok = wait(&s_full[t], turn & 1))) break;
        tmem_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_col + 32 * c, s[c]);
        tmem_wait_ld();
        // a tile that some query of the warp does not see whole
        const int left = seen - i * kK;
        if (__any_sync(0xFFFFFFFFu, left < kK)) {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c >= left) s[c / 32][c % 32] = __float_as_uint(-INFINITY);
        }
        float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 128; ++c) top4[c & 3] = fmaxf(top4[c & 3], __uint_as_float(s[c / 32][c % 32]));
        float top = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
        top *= P.scale_log2;  // (positive)
        if (__any_sync(0xFFFFFFFFu, top > m + kGrow)) {
          const float to = fmaxf(m, top);
          const float f = to == m ? 1.f : exp2_fast(m - to);  // the first maximum: 0
          m = to, l *= f;
          if (i > 0) {
            // this warp's lanes of O; the MMAs before this S have ended
#pragma unroll 1
            for (int c = 0; c < kValue; c += 32) {
              uint32_t o[32];
              tmem_ld32(o_col + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tc::tmem_st32(o_col + c, o);
            }
          }
        }
        const float off = m == -INFINITY ? 0.f : -m;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t p[32];
#pragma unroll
          for (int c = 0; c < 64; c += 2) {
            const int at = 64 * half + c;
            const float a = exp2_fast(fmaf(__uint_as_float(s[at / 32][at % 32]), P.scale_log2, off));
            const float b = exp2_fast(fmaf(__uint_as_float(s[at / 32][at % 32 + 1]), P.scale_log2, off));
            sum[c & 2] += a, sum[(c & 2) + 1] += b;
            p[c / 2] = pack_bf16(a, b);
          }
          tc::tmem_st32(s_col + 32 * half, p);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_wait_st();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t]);
      }
      if (!ok) break;
      if (here <= 0) continue;
      uint16_t* const out = P.out + ((int64_t)(w.q0 + t * kQ + row) * P.H + w.h) * kValue;
      const bool mine = row < here;
      if (w.n[t] == 0) {
        if (mine)
          for (int c = 0; c < kValue; c += 8) *reinterpret_cast<uint4*>(out + c) = make_uint4(0, 0, 0, 0);
        continue;
      }
      if (!(ok = wait(&o_full[t], use & 1))) break;
      ++use;
      tmem_fence_after();
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;  // a query that sees nothing: zeros
#pragma unroll 1
      for (int c = 0; c < kValue; c += 32) {
        uint32_t o[32];
        tmem_ld32(o_col + c, o);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          uint32_t v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            v[k] = pack_bf16(__uint_as_float(o[j + 2 * k]) * inv, __uint_as_float(o[j + 2 * k + 1]) * inv);
          if (mine) *reinterpret_cast<uint4*>(out + c + j) = make_uint4(v[0], v[1], v[2], v[3]);
        }
      }
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&o_free[t]);
    }
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == 1) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols));
  }
}

// The kernel's limits on the current device, once; an error if it was compiled to
// fewer registers than its split needs (the softmax's warps would wait for ever).
cudaError_t ready() {
  const void* const k = reinterpret_cast<const void*>(latent_attention_kernel);
  static const bool enough = [k] {
    cudaFuncAttributes a;
    return cudaFuncGetAttributes(&a, k) == cudaSuccess && a.numRegs >= kRegsLaunch;
  }();
  return enough ? ensure_smem_optin(k, kSmem) : cudaErrorLaunchOutOfResources;
}

}  // namespace

cudaError_t latent_attention_error(int32_t** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_attention_err);
}

}  // namespace moe_fp4

using namespace moe_fp4;

extern "C" int moe_fp4_latent_attention(const moe_fp4_latent_attention_args* args, void* cuda_stream) {
  if (!args) return MOE_FP4_ERR_INVALID_ARG;
  const moe_fp4_latent_attention_args a = *args;
  if (a.B < 0 || a.H < 1 || a.H > MOE_FP4_LATENT_MAX_HEADS || a.Tq < 0 || a.Tk < 0 || !(a.scale > 0.f) || a.scale > 3e38f ||
      a.causal < 0 || a.causal > 1)
    return MOE_FP4_ERR_INVALID_ARG;
  // items and TMA coordinates are counted in 32 bits
  const int64_t tiles = a.Tq / (2 * kQ) + std::min<int64_t>(a.B, a.Tq);
  if (a.Tq > INT32_MAX - 4 * kQ || a.Tk > INT32_MAX - 2 * kK || (tiles + num_sms()) * a.H >= (1LL << 30)) return MOE_FP4_ERR_UNSUPPORTED;
  if (a.B == 0 || a.Tq == 0) return MOE_FP4_OK;
  const auto rows = [](const void* p, int64_t stride, int64_t head_stride, int64_t width) {
    return p && ((uintptr_t)p & 15) == 0 && stride >= width && head_stride >= width && stride % 8 == 0 && head_stride % 8 == 0 &&
           stride < (1LL << 38) && head_stride < (1LL << 38);
  };
  if (!rows(a.q, a.q_stride, a.q_head_stride, kNope + kRope) || !a.q_offsets || !a.k_offsets || !a.out ||
      ((uintptr_t)a.q_offsets & 3) || ((uintptr_t)a.k_offsets & 3) || ((uintptr_t)a.out & 15))
    return MOE_FP4_ERR_INVALID_ARG;
  if (a.Tk > 0 && (!rows(a.kv, a.kv_stride, a.kv_head_stride, kNope + kValue) || !rows(a.k_rope, a.rope_stride, kRope, kRope)))
    return MOE_FP4_ERR_INVALID_ARG;
  AttentionParams P{};
  P.q_offsets = a.q_offsets, P.k_offsets = a.k_offsets, P.out = static_cast<uint16_t*>(a.out);
  P.B = a.B, P.H = a.H, P.Tq = (int)a.Tq, P.Tk = (int)a.Tk, P.causal = a.causal;
  P.scale_log2 = a.scale * 1.4426950408889634f;
  P.fault = fault_site() == MOE_FP4_FAULT_TC_TOKEN_TILE;
  P.wait_ns = wait_limit_ns();
  CUtensorMap map_q, map_kv, map_rope;
  const uint32_t box[3] = {64, 1, 128};
  const uint64_t H = a.H, qd[3] = {kNope + kRope, H, (uint64_t)a.Tq};
  const uint64_t qs[2] = {(uint64_t)a.q_head_stride * 2, (uint64_t)a.q_stride * 2};
  if (!make_map_3d(&map_q, a.q, qd, qs, box)) return MOE_FP4_ERR_CUDA;
  if (a.Tk > 0) {
    const uint64_t kd[3] = {kNope + kValue, H, (uint64_t)a.Tk}, ks[2] = {(uint64_t)a.kv_head_stride * 2, (uint64_t)a.kv_stride * 2};
    const uint64_t rd[3] = {kRope, 1, (uint64_t)a.Tk}, rs[2] = {(uint64_t)a.rope_stride * 2, (uint64_t)a.rope_stride * 2};
    if (!make_map_3d(&map_kv, a.kv, kd, ks, box) || !make_map_3d(&map_rope, a.k_rope, rd, rs, box)) return MOE_FP4_ERR_CUDA;
  } else {
    map_kv = map_rope = map_q;  // nothing is loaded through them
  }
  if (ready() != cudaSuccess) return MOE_FP4_ERR_CUDA;
  const int grid = (int)std::min<int64_t>(num_sms(), tiles * a.H);
  return launch_early(latent_attention_kernel, dim3(grid), dim3(kThreads), kSmem, static_cast<cudaStream_t>(cuda_stream), map_q,
                      map_kv, map_rope, P) == cudaSuccess
             ? MOE_FP4_OK
             : MOE_FP4_ERR_CUDA;
}
