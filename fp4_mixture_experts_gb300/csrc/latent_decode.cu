// Latent attention of one new token a sequence (the absorbed form) over a paged
// cache of the latent vectors:
//
//   s[h, j] = scale q[b, h] . c[b, j]          (576: latent 512 and rotary 64)
//   out[b, h] = sum_j softmax(s[h])_j c[b, j][0 .. 511]
//
// All heads read the same vectors, so a tile of tokens that is in shared memory
// once serves 2 x 64 heads x (576 + 512) multiply-adds a token: with up to 64 heads
// reading the cache bounds it, with 128 the tensor cores come close.
//
// A tile is 64 tokens, 9 slabs of 64 elements ([64 tokens][128 bytes], 128-byte
// swizzle).  S = Q K^T has heads as M = 64 and tokens as N = 64, so that a head's
// scores lie in one row of tensor memory and a softmax needs two shuffles; P goes to
// shared memory as [head][token].  The sums are transposed, O^T = V^T P^T: M = 128
// elements of the latent vector (two slabs of the same tile, MN-major), four of
// them, N = the heads.  O as [64 heads][512] would take all 512 columns of tensor
// memory and leave none for S.
//
// The running maximum moves only when a score exceeds it by more than 2^8: then
// O^T is multiplied, column by column, in tensor memory; until then P may grow up
// to 2^8, which costs bf16 nothing.
//
// The tiles of all sequences are numbered through and dealt out in equal ranges,
// one a CTA, whatever the lengths are; a sequence that is cut leaves unnormalised
// sums (fp32) and its maximum and sum in the workspace, which a second kernel
// joins in the ranges' order.  The same lengths give the same bits.
//
// Warps: 0 and 1 load (tokens; 0 the queries too), 2 issues the MMAs, 4..7 are the
// softmax, the rescaling and the results.  Waits are bounded; a piece whose wait ran
// out stores nothing, and a sequence with such a piece is not joined.
#include <algorithm>
#include <numeric>

#include "latent.cuh"

namespace moe_fp4 {
namespace {

using namespace latent;
using tc::umma_commit;

__device__ int32_t g_decode_err[4];

constexpr int kThreads = 256;
constexpr int kTile = 64;                     // tokens of a tile
constexpr int kHeads = 64;                    // heads of a CTA, at most
constexpr int kSlab = kTile * 128;
constexpr int kSlabs = kRow / 64, kValueSlabs = kLatent / 64;
constexpr int kStage = kSlabs * kSlab;
constexpr int kStages = 2;
constexpr int kOffQ = kStages * kStage;
constexpr int kOffP = kOffQ + kSlabs * kHeads * 128;
constexpr int kOffTail = kOffP + kHeads * 128;
constexpr int kSmem = kOffTail + 1024 + 1024;
static_assert(kSmem <= kSmemMax, "shared memory");
constexpr uint32_t kCols = 512;
constexpr uint32_t kColS = 4 * kHeads;        // O^T: 4 x 64 columns, then two buffers of S
constexpr float kGrow = 8.f;                  // log2 of what P may grow to
constexpr int kMinTiles = 4;                  // of a range
constexpr int kMaxRanges = 256;               // (threads of the join kernel, at most)

struct DecodeParams {
  const int32_t* table;
  const int32_t* lengths;
  uint16_t* out;
  int32_t* err;
  int4* cut;           // [range]: the sequence at its start, tiles of it before, all of its tiles, tiles of a range
  int32_t* done;       // [slot]: its piece is in the workspace
  float2* ml;          // [slot][heads]: maximum (log2) and sum
  float* sums;         // [slot][heads][512]
  int64_t table_stride;
  int B, H, groups, heads;  // heads: of a group
  int page, width, pages, box;  // box: tokens of a copy
  int ranges;
  float scale_log2;
  int fault;
  uint64_t wait_ns;
};

// A sequence's length, kept to what its row of the table holds.
__device__ __forceinline__ int length_at(const DecodeParams& P, int b) {
  const int64_t most = (int64_t)P.width * P.page;
  const int n = P.lengths[b];
  return (int)min((int64_t)max(n, 0), most);
}
__device__ __forceinline__ int tiles_of(int n) { return n / kTile + (n % kTile != 0); }

// Tiles of a range: the ranges' even share, a few at least.
__device__ __forceinline__ int64_t share(const DecodeParams& P, int64_t total) {
  const int64_t even = (total + P.ranges - 1) / P.ranges;
  return even > kMinTiles ? even : kMinTiles;
}

// The pieces of this CTA's range, sequence by sequence; every warp walks them with
// its own cursor and holds the lengths of 32 sequences.
struct Walk {
  int b, t0, left;     // sequence, its first tile here, tiles left of the range
  int nt, len, all;    // of the piece: tiles, length of the sequence and its tiles
  int base, mine;
  __device__ __forceinline__ void start(int b_, int t_, int left_) {
    b = b_, t0 = t_, left = left_, nt = 0, base = -32;
  }
  __device__ __forceinline__ bool next(const DecodeParams& P) {
    if (nt > 0) ++b, t0 = 0;
    for (; left > 0 && b < P.B; ++b, t0 = 0) {
      if (b >= base + 32) {
        base = b;
        const int i = b + (threadIdx.x & 31);
        mine = i < P.B ? length_at(P, i) : 0;
      }
      len = __shfl_sync(0xFFFFFFFFu, mine, b - base);
      all = tiles_of(len);
      if (all == 0) continue;
      nt = min(all - t0, left);
      left -= nt;
      return true;
    }
    return false;
  }
};

// The sum of v over the block; scratch: a word of 64 bits for each warp.
__device__ int64_t block_sum(int64_t v, int64_t* scratch) {
  const int warp = threadIdx.x >> 5;
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, s);
  if ((threadIdx.x & 31) == 0) scratch[warp] = v;
  __syncthreads();
  int64_t sum = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) sum += scratch[w];
  __syncthreads();
  return sum;
}

// Where tile number `at` (below the total) is: its sequence, and its number there.
__device__ void find_tile(const DecodeParams& P, int64_t at, int64_t* scratch, int* b_out, int* t_out) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int64_t before = 0;
  for (int b0 = 0; b0 < P.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    const int n = b < P.B ? tiles_of(length_at(P, b)) : 0;
    int64_t c = n;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int64_t v = __shfl_up_sync(0xFFFFFFFFu, c, s);
      if (lane >= s) c += v;
    }
    if (lane == 31) scratch[warp] = c;
    __syncthreads();
    int64_t first = before, all = before;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) first += scratch[w];
      all += scratch[w];
    }
    first += c - n;
    if (n > 0 && first <= at && at < first + n) *b_out = b, *t_out = (int)(at - first);
    __syncthreads();
    before = all;
    if (before > at) break;
  }
  __syncthreads();
}

__global__ void __launch_bounds__(kThreads, 1)
latent_decode_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_c, DecodeParams P) {
  P.err = &g_decode_err[0];
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(smem + kOffTail);  // [stage]: bytes landed
  uint64_t* kv_empty = kv_full + kStages;                            // [stage]: its MMAs completed
  uint64_t* s_full = kv_empty + kStages;                             // [2]
  uint64_t* s_free = s_full + 2;                                     // [2]: read by the four warps
  uint64_t* q_full = s_free + 2;
  uint64_t* q_empty = q_full + 1;
  uint64_t* p_full = q_empty + 1;                                    // P (and O^T) written by the four warps
  uint64_t* pv_done = p_full + 1;
  uint64_t* o_free = pv_done + 1;                                    // O^T read by the four warps
  uint64_t* mma_done = o_free + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* where = reinterpret_cast<int*>(tmem_slot + 2);                // [2]
  float* factor = reinterpret_cast<float*>(smem + kOffTail + 256);   // [heads]
  int64_t* scratch = reinterpret_cast<int64_t*>(smem + kOffTail + 512);
  const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&kv_full[s], P.box == kTile ? 1 : 2), mbar_init(&kv_empty[s], 1);
    for (int s = 0; s < 2; ++s) mbar_init(&s_full[s], 1), mbar_init(&s_free[s], 4);
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(p_full, 4);
    mbar_init(pv_done, 1);
    mbar_init(o_free, 4);
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    mbar_fence_init();
  }
  __syncwarp();
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  griddep_begin();
  const int group = blockIdx.x % P.groups, range = blockIdx.x / P.groups;
  const int head0 = group * P.heads, live = min(P.heads, P.H - head0);  // this CTA's heads
  const int slot0 = (2 * range) * P.groups + group;
  if (threadIdx.x < 2) P.done[slot0 + threadIdx.x * P.groups] = 0;
  // this range's tiles
  int64_t mine = 0;
  bool bad = false;
  for (int b = threadIdx.x; b < P.B; b += kThreads) {
    const int n = length_at(P, b);
    bad |= n != P.lengths[b];
    mine += tiles_of(n);
  }
  if (bad && blockIdx.x == 0) atomicOr(P.err, kErrBadExpertId);
  tmem_fence_before();
  const int64_t total = block_sum(mine, scratch);
  tmem_fence_after();
  const int64_t per = share(P, total), first = per * range, last = min(total, first + per);
  const int left = (int)max(last - first, (int64_t)0);
  if (left > 0) find_tile(P, first, scratch, &where[0], &where[1]);
  if (group == 0 && threadIdx.x == 0)
    P.cut[range] = left > 0 ? make_int4(where[0], where[1], tiles_of(length_at(P, where[0])), (int)per) : make_int4(0, 0, 0, 0);
  // sequences of no tokens
  for (int b = blockIdx.x; b < P.B; b += gridDim.x)
    if (length_at(P, b) == 0)
      for (int64_t i = threadIdx.x; i < (int64_t)P.H * (kLatent / 8); i += kThreads)
        reinterpret_cast<uint4*>(P.out + (int64_t)b * P.H * kLatent)[i] = make_uint4(0, 0, 0, 0);
  Walk w;
  w.start(left > 0 ? where[0] : P.B, left > 0 ? where[1] : 0, left);
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
  const Waits wait{abort_flag, P.err, P.wait_ns};
  const int n_mma = (live + 15) & ~15;

  if (warp < 2) {
    // ---------------- loads ----------------
    const int copies = kTile / P.box;  // of a slab
    int g = 0, piece = 0;
    bool ok = true;
    while (ok && w.next(P)) {
      if (warp == 0) {
        ok = wait(q_empty, (piece & 1) ^ 1);
        if (!ok) break;
        if (elect_one()) {
          mbar_expect_tx(q_full, kSlabs * kHeads * 128);
          for (int s = 0; s < kSlabs; ++s)
            tma_load_3d(smem + kOffQ + s * kHeads * 128, &map_q, s * 64, head0, w.b, q_full);
        }
        __syncwarp();
        ++piece;
      }
      // the tokens' first row in the cache, for copy `lane` of a tile; a tile ahead.  A page outside the cache reads
      // as zeros.
      const int none = P.pages * P.page;
      auto row_of = [&](int t) {
        const int token = t * kTile + lane * P.box;
        if (lane >= copies || token >= w.len) return none;
        const int page = P.table[w.b * P.table_stride + token / P.page];
        if (page < 0 || page >= P.pages) {
          atomicOr(P.err, kErrBadExpertId);
          return none;
        }
        return page * P.page + token % P.page;
      };
      int row = row_of(w.t0);
      for (int i = 0; i < w.nt; ++i, ++g) {
        const int next = i + 1 < w.nt ? row_of(w.t0 + i + 1) : 0;
        const int s = g % kStages;
        ok = wait(&kv_empty[s], ((g / kStages) & 1) ^ 1);
        if (!ok) break;
        if (!(P.fault && blockIdx.x == 0 && g == 0)) {
          uint8_t* st = smem + s * kStage;
          const int here = min(copies, (w.len - (w.t0 + i) * kTile + P.box - 1) / P.box);
          const int r0 = __shfl_sync(0xFFFFFFFFu, row, 0);
          if (copies == 1) {
            if (warp == 0 && elect_one()) {
              mbar_expect_tx(&kv_full[s], kStage);
              tma_load_3d(st, &map_c, 0, r0, 0, &kv_full[s]);
            }
          } else {
            // either warp's share of the slabs
            if (elect_one()) mbar_expect_tx(&kv_full[s], (kSlabs / 2 + (warp == 0)) * here * P.box * 128);
            __syncwarp();
            for (int c = 0; c < here; ++c) {
              const int r = __shfl_sync(0xFFFFFFFFu, row, c);
              if (elect_one())
                for (int sl = warp; sl < kSlabs; sl += 2)
                  tma_load_3d(st + sl * kSlab + c * P.box * 128, &map_c, 0, r, sl, &kv_full[s]);
              __syncwarp();
            }
          }
          __syncwarp();
        }
        row = next;
      }
    }
    // every issued copy has landed before shared memory is given back
    __syncwarp();
    if (warp == 0 || copies > 1) {
      for (int q = max(0, g - kStages); q < g; ++q) wait.drain(&kv_full[q % kStages], (q / kStages) & 1);
      if (piece > 0) wait.drain(q_full, (piece - 1) & 1);
    }
  } else if (warp == 2) {
    // ---------------- MMAs ----------------
    const uint32_t base = smem_u32(smem);
    const uint32_t q_lo = desc_lo(base + kOffQ, 16), p_lo = desc_lo(base + kOffP, 16);
    const uint32_t id_qk = idesc_bf16(kHeads, kTile, false, false), id_pv = idesc_bf16(128, n_mma, true, false);
    int g0 = 0, piece = 0;
    bool ok = true;
    while (ok && w.next(P)) {
      ok = wait(q_full, piece & 1);
      if (!ok) break;
      int qi = 0, pi = 0;  // tiles whose scores, whose sums have been issued
      uint64_t since = 0;
      while (pi < w.nt) {
        const int gq = g0 + qi, gp = g0 + pi;
        if (qi < w.nt && qi < pi + 2 && mbar_test(&kv_full[gq % kStages], (gq / kStages) & 1) &&
            mbar_test(&s_free[gq & 1], ((gq >> 1) & 1) ^ 1)) {
          tmem_fence_after();
          if (elect_one()) {
            const uint32_t k_lo = desc_lo(base + (gq % kStages) * kStage, 16);
            const uint32_t d = tmem + kColS + (gq & 1) * kTile;
#pragma unroll
            for (int k = 0; k < kRow / 16; ++k) {
              const uint32_t at = ((k / 4) * kSlab + (k % 4) * 32) >> 4;
              umma_ss(d, desc(q_lo + at), desc(k_lo + at), id_qk, k > 0);
            }
            umma_commit(&s_full[gq & 1]);
            if (qi == w.nt - 1) umma_commit(q_empty);
          }
          __syncwarp();
          ++qi;
          since = 0;
        } else if (pi < qi && mbar_test(p_full, gp & 1) && (pi > 0 || mbar_test(o_free, (piece & 1) ^ 1))) {
          tmem_fence_after();
          if (elect_one()) {
            const uint32_t v_lo = desc_lo(base + (gp % kStages) * kStage, kSlab);
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
#pragma unroll
              for (int j = 0; j < 4; ++j)
                umma_ss(tmem + j * kHeads, desc(v_lo + ((2 * j * kSlab + k * 2048) >> 4)), desc(p_lo + ((k * 32) >> 4)),
                        id_pv, pi > 0 || k > 0);
            umma_commit(pv_done);
            umma_commit(&kv_empty[gp % kStages]);
          }
          __syncwarp();
          ++pi;
          since = 0;
        } else {
          const uint64_t now = global_timer_ns();
          if (since == 0) since = now;
          const bool out_of_time = now - since > P.wait_ns;
          if (__any_sync(0xFFFFFFFFu, out_of_time || *abort_flag)) {
            if (lane == 0) {
              if (!*abort_flag) atomicOr(P.err, kErrWaitTimeout);
              *abort_flag = 1;
            }
            ok = false;
            break;
          }
        }
      }
      g0 += w.nt;
      ++piece;
    }
    __syncwarp();
    if (elect_one()) umma_commit(mma_done);
    __syncwarp();
    wait.drain(mma_done, 0);
  } else if (warp >= 4) {
    // ---------------- softmax, rescaling, results ----------------
    const int q = warp & 3, tid = threadIdx.x - 128;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    const bool rows_live = 16 * q < n_mma;
    const int r0 = 16 * q + (lane >> 2);  // this thread's heads: r0 and r0 + 8
    int g = 0, piece = 0;
    bool ok = true;  // no wait of this warp has run out; with one, the warp walks on without waits and stores
    while (w.next(P)) {
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
      for (int i = 0; i < w.nt; ++i, ++g) {
        const int n = min(kTile, w.len - (w.t0 + i) * kTile);  // tokens here
        ok = ok && wait(&s_full[g & 1], (g >> 1) & 1);
        tmem_fence_after();
        uint32_t raw[32];
        if (rows_live) {
          tmem_ld_rows16(tmem + kColS + (g & 1) * kTile + lanes, raw);
          tmem_wait_ld();
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&s_free[g & 1]);
        // rows behind the sequence's end count as zeros: whatever is there must not meet a zero of P
        if (n < kTile && ok) {
          uint8_t* st = smem + (g % kStages) * kStage;
          for (int c = tid; c < (kTile - n) * kValueSlabs * 8; c += 128) {
            const int row = n + c / (kValueSlabs * 8), s = (c >> 3) % kValueSlabs;
            *reinterpret_cast<uint4*>(st + s * kSlab + row * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        float s[2][16], top[2] = {-INFINITY, -INFINITY};
        if (rows_live) {
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const int token = 8 * (c >> 1) + 2 * (lane & 3) + (c & 1);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float v = __uint_as_float(raw[4 * (c >> 1) + 2 * r + (c & 1)]) * P.scale_log2;
              s[r][c] = token < n ? v : -INFINITY;
              top[r] = fmaxf(top[r], s[r][c]);
            }
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            top[r] = fmaxf(top[r], __shfl_xor_sync(0xFFFFFFFFu, top[r], 1));
            top[r] = fmaxf(top[r], __shfl_xor_sync(0xFFFFFFFFu, top[r], 2));
          }
        }
        const bool grow = rows_live && (top[0] > m[0] + kGrow || top[1] > m[1] + kGrow);
        if (any_at_barrier(grow, 1, 128)) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float to = fmaxf(m[r], top[r]);
            const float f = to == m[r] ? 1.f : exp2_fast(m[r] - to);  // the first maximum: 0
            if (rows_live && (lane & 3) == 0) factor[r0 + 8 * r] = f;
            m[r] = to, l[r] *= f;
          }
          if (i > 0) {
            ok = ok && wait(pv_done, (g - 1) & 1);
            any_at_barrier(false, 1, 128);  // the factors are written
            tmem_fence_after();
            for (int c0 = 0; ok && c0 < 4 * kHeads; c0 += 32) {
              if ((c0 & (kHeads - 1)) >= n_mma) continue;
              uint32_t o[32];
              tmem_ld32(tmem + lanes + c0, o);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j)
                o[j] = __float_as_uint(__uint_as_float(o[j]) * factor[(c0 & (kHeads - 1)) + j]);
              tc::tmem_st32(tmem + lanes + c0, o);
            }
            tmem_wait_st();
            tmem_fence_before();
            any_at_barrier(false, 1, 128);  // and read: the next ones may follow
          }
        }
        uint32_t p[2][8];
        if (rows_live) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float off = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
            for (int c = 0; c < 16; c += 2) {
              const float a = exp2_fast(s[r][c] - off), b = exp2_fast(s[r][c + 1] - off);
              l[r] += a + b;
              p[r][c / 2] = pack_bf16(a, b);
            }
          }
        }
        if (i > 0) ok = ok && wait(pv_done, (g - 1) & 1);  // P's last readers
        if (rows_live && ok) {
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int row = r0 + 8 * r;
#pragma unroll
            for (int c = 0; c < 8; ++c)
              *reinterpret_cast<uint32_t*>(smem + kOffP + row * 128 + ((c ^ (row & 7)) << 4) + (lane & 3) * 4) = p[r][c];
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(p_full);
      }
      // ---- the piece's results ----
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 1);
        l[r] += __shfl_xor_sync(0xFFFFFFFFu, l[r], 2);
      }
      const bool whole = w.nt == w.all;
      const int slot = slot0 + (piece > 0 ? P.groups : 0);
      if (rows_live && (lane & 3) == 0) {
#pragma unroll
        for (int r = 0; r < 2; ++r) factor[r0 + 8 * r] = whole ? 1.f / l[r] : 1.f;
      }
      ok = ok && wait(pv_done, (g - 1) & 1);
      const bool all_ok = !any_at_barrier(!ok, 1, 128);
      tmem_fence_after();
      if (all_ok) {
        const int dim0 = q * 32 + lane;
        uint16_t* const out = P.out + ((int64_t)w.b * P.H + head0) * kLatent + dim0;
        float* const sums = P.sums + (int64_t)slot * P.heads * kLatent + dim0;
        for (int c0 = 0; c0 < 4 * kHeads; c0 += 32) {
          const int h0 = c0 & (kHeads - 1), dim = (c0 / kHeads) * 128;
          if (h0 >= live) continue;
          uint32_t o[32];
          tmem_ld32(tmem + lanes + c0, o);
          tmem_wait_ld();
          if (whole) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (h0 + j < live)
                out[(int64_t)(h0 + j) * kLatent + dim] = f32_to_bf16_rn(__uint_as_float(o[j]) * factor[h0 + j]);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (h0 + j < live) sums[(int64_t)(h0 + j) * kLatent + dim] = __uint_as_float(o[j]);
          }
        }
        if (!whole && rows_live && (lane & 3) == 0) {
#pragma unroll
          for (int r = 0; r < 2; ++r)
            if (r0 + 8 * r < live) P.ml[(int64_t)slot * P.heads + r0 + 8 * r] = make_float2(m[r], l[r]);
        }
      }
      tmem_fence_before();
      any_at_barrier(false, 1, 128);  // the factors are read, the piece's results stored
      if (tid == 0 && all_ok && !whole) P.done[slot] = 1;
      if (lane == 0 && all_ok) mbar_arrive(o_free);
      ok = all_ok;
      ++piece;
    }
  }
  __syncwarp();
  tmem_fence_before();
  __syncthreads();
  if (warp == 2) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols));
  }
}

// The pieces of cut sequences, joined: a CTA a sequence and head at a time, four
// groups of 128 threads that take the pieces in turn, four elements a thread.
__global__ void __launch_bounds__(512) latent_join_kernel(DecodeParams P) {
  griddep_begin();
  __shared__ int4 list[kMaxRanges];  // sequence, first and last range, first slot's number
  __shared__ uint32_t found[kMaxRanges / 32];
  __shared__ float4 part[4][128];
  __shared__ float part_l[4];
  // A range that starts inside a sequence cuts it, the first such one names it; in the ranges' order, the same list
  // in every CTA.
  const int rr = threadIdx.x;
  int4 cut = make_int4(0, 0, 0, 0);
  if (rr < P.ranges) cut = P.cut[rr];
  const bool names = cut.y > 0 && cut.y <= cut.w;
  const uint32_t mask = __ballot_sync(0xFFFFFFFFu, names);
  if (rr < kMaxRanges && (rr & 31) == 0) found[rr >> 5] = mask;
  __syncthreads();
  int count = 0, at = __popc(mask & ((1u << (rr & 31)) - 1));
  for (int i = 0; i < kMaxRanges / 32; ++i) {
    if (i < rr >> 5) at += __popc(found[i]);
    count += __popc(found[i]);
  }
  if (names) {
    const int64_t start = (int64_t)rr * cut.w - cut.y;
    list[at] = make_int4(cut.x, rr - 1, (int)((start + cut.z - 1) / cut.w), 2 * (rr - 1) + (cut.y < cut.w ? 1 : 0));
  }
  __syncthreads();
  const int tid = threadIdx.x & 127, part_of = threadIdx.x >> 7;
  for (int item = blockIdx.x; item < count * P.H; item += gridDim.x) {
    const int4 c = list[item / P.H];
    const int h = item % P.H, group = h / P.heads, hh = h % P.heads;
    const int first = c.y, last = c.z;
    auto slot_of = [&](int r) { return (int64_t)(r == first ? c.w : 2 * r) * P.groups + group; };
    float top = -INFINITY;
    bool complete = true;
    for (int r = first; r <= last; ++r) {
      const int64_t s = slot_of(r);
      complete &= P.done[s] != 0;
      top = fmaxf(top, P.ml[s * P.heads + hh].x);
    }
    if (!complete) continue;  // a wait ran out; the same in all threads
    if (top == -INFINITY) top = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll 4
    for (int r = first + part_of; r <= last; r += 4) {
      const int64_t s = slot_of(r) * P.heads + hh;
      const float2 ml = P.ml[s];
      const float f = exp2f(ml.x - top);
      const float4 v = reinterpret_cast<const float4*>(P.sums + s * kLatent)[tid];
      o.x += f * v.x, o.y += f * v.y, o.z += f * v.z, o.w += f * v.w;
      l += f * ml.y;
    }
    part[part_of][tid] = o;
    if (tid == 0) part_l[part_of] = l;
    __syncthreads();
    if (threadIdx.x < 128) {
      l = 0.f;
      o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = part[i][tid];
        o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
        l += part_l[i];
      }
      const float inv = 1.f / l;
      reinterpret_cast<uint2*>(P.out + ((int64_t)c.x * P.H + h) * kLatent)[tid] =
          make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    }
    __syncthreads();
  }
}

struct Shape {
  int groups, heads, ranges;
  int64_t slots;
};

// Groups of up to 64 heads, even ones; as many ranges as there are SMs for them.
Shape shape_of(int H) {
  Shape s;
  s.groups = (H + kHeads - 1) / kHeads;
  s.heads = ((H + s.groups - 1) / s.groups + 15) & ~15;
  s.groups = (H + s.heads - 1) / s.heads;
  s.ranges = std::min(kMaxRanges, std::max(1, num_sms() / s.groups));
  s.slots = 2LL * s.ranges * s.groups;
  return s;
}

size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace

cudaError_t latent_decode_error(int32_t** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_decode_err);
}

}  // namespace moe_fp4

using namespace moe_fp4;

extern "C" {

size_t moe_fp4_latent_decode_workspace_bytes(int32_t H) {
  if (H < 1 || H > MOE_FP4_LATENT_MAX_HEADS) return 0;
  const Shape s = shape_of(H);
  return align256(kMaxRanges * sizeof(int4)) + align256(s.slots * sizeof(int32_t)) + align256(s.slots * s.heads * sizeof(float2)) +
         (size_t)s.slots * s.heads * kLatent * sizeof(float);
}

int moe_fp4_latent_decode(const moe_fp4_latent_decode_args* args, void* workspace, size_t workspace_bytes,
                          void* cuda_stream) {
  if (!args) return MOE_FP4_ERR_INVALID_ARG;
  const moe_fp4_latent_decode_args a = *args;
  if (a.B < 0 || a.H < 1 || a.H > MOE_FP4_LATENT_MAX_HEADS || a.page < 16 || a.page % 16 != 0 || a.pages < 1 || a.width < 1 ||
      !(a.scale == a.scale) || a.table_stride < a.width)
    return MOE_FP4_ERR_INVALID_ARG;
  if ((int64_t)a.pages * a.page >= (1LL << 31) || (int64_t)a.width * a.page >= (1LL << 31) || (int64_t)a.B * a.H >= (1LL << 31))
    return MOE_FP4_ERR_UNSUPPORTED;
  if (a.B == 0) return MOE_FP4_OK;
  if (!a.q || !a.cache || !a.table || !a.lengths || !a.out || ((uintptr_t)a.q & 15) || ((uintptr_t)a.cache & 15) ||
      ((uintptr_t)a.table & 3) || ((uintptr_t)a.lengths & 3) || ((uintptr_t)a.out & 15) || a.q_head_stride < kRow ||
      a.q_head_stride % 8 != 0 || a.q_stride < kRow || a.q_stride % 8 != 0 || a.q_stride >= (1LL << 38) || a.q_head_stride >= (1LL << 38))
    return MOE_FP4_ERR_INVALID_ARG;
  if (!workspace || ((uintptr_t)workspace & 255)) return MOE_FP4_ERR_INVALID_ARG;
  if (workspace_bytes < moe_fp4_latent_decode_workspace_bytes(a.H)) return MOE_FP4_ERR_WORKSPACE;
  const Shape s = shape_of(a.H);
  DecodeParams P{};
  P.table = a.table, P.lengths = a.lengths, P.out = static_cast<uint16_t*>(a.out);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  P.cut = reinterpret_cast<int4*>(ws);
  ws += align256(kMaxRanges * sizeof(int4));
  P.done = reinterpret_cast<int32_t*>(ws);
  ws += align256(s.slots * sizeof(int32_t));
  P.ml = reinterpret_cast<float2*>(ws);
  ws += align256(s.slots * s.heads * sizeof(float2));
  P.sums = reinterpret_cast<float*>(ws);
  P.table_stride = a.table_stride;
  P.B = a.B, P.H = a.H, P.groups = s.groups, P.heads = s.heads, P.ranges = s.ranges;
  P.page = a.page, P.width = a.width, P.pages = a.pages, P.box = std::gcd(a.page, kTile);
  P.scale_log2 = a.scale * 1.4426950408889634f;
  P.fault = fault_site() == MOE_FP4_FAULT_TC_TOKEN_TILE;
  P.wait_ns = wait_limit_ns();
  CUtensorMap map_q, map_c;
  const uint64_t qd[3] = {kRow, (uint64_t)a.H, (uint64_t)a.B}, qs[2] = {(uint64_t)a.q_head_stride * 2, (uint64_t)a.q_stride * 2};
  const uint32_t qb[3] = {64, kHeads, 1};
  const uint64_t cd[3] = {64, (uint64_t)a.pages * a.page, kSlabs}, cs[2] = {kRow * 2, 128};
  const uint32_t cb[3] = {64, (uint32_t)P.box, P.box == kTile ? (uint32_t)kSlabs : 1u};
  if (!make_map_3d(&map_q, a.q, qd, qs, qb) || !make_map_3d(&map_c, a.cache, cd, cs, cb)) return MOE_FP4_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (ensure_smem_optin(reinterpret_cast<const void*>(latent_decode_kernel), kSmem) != cudaSuccess) return MOE_FP4_ERR_CUDA;
  if (launch_early(latent_decode_kernel, dim3(s.ranges * s.groups), dim3(kThreads), kSmem, st, map_q, map_c, P) != cudaSuccess)
    return MOE_FP4_ERR_CUDA;
  // at most a sequence is cut for each range but the first
  const int64_t items = (int64_t)std::min(a.B, s.ranges - 1) * a.H;
  if (items == 0) return MOE_FP4_OK;
  return launch_early(latent_join_kernel, dim3((unsigned)std::min<int64_t>(items, 2 * num_sms())), dim3(512), 0, st, P) ==
                 cudaSuccess
             ? MOE_FP4_OK
             : MOE_FP4_ERR_CUDA;
}

}  // extern "C"
