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
// What it takes: an MMA of 16 elements of K 61 cycles for QK (M = N = 64) and 75 for PV
// (M = 128, N = 64), 3,396 a tile, 1.8 us, where HBM brings an SM's tile in 1.7: 4
// sequences of 131072 tokens, 64 heads, 114 us, 5.3 TB/s; with 128 heads every tile is read
// by two CTAs, 188 us.  There is room for two tiles, each held from its first byte to its
// last MMA; the one behind them is fetched to L2 meanwhile (without: 124 and 206 us; two
// ahead are no better).  One sequence of 4608 tokens 14.6 us: the first tile's scores
// are there after 5, its sums after 7.
//
// Warps: 0 and, for tiles of many copies, 1 load (tokens; 0 the queries too), 2 issues the MMAs, 3 writes the
// results of sequences without tokens, 4..7 are the softmax, the rescaling and the
// results.  Waits are bounded; a piece whose wait ran
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
constexpr int kSlabs = kRow / 64;
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
constexpr int kMaxRanges = 256;

struct DecodeParams {
  const int32_t* table;
  const int32_t* lengths;
  uint16_t* out;
  int32_t* err;
  int4* cut;           // [range]: the sequence at its start, tiles of it before, all of its tiles, tiles of a range
  int32_t* done;       // [slot]: its piece is in the workspace
  float2* ml;          // [slot][heads]: maximum (log2) and sum
  float* sums;         // [slot][4 x 128 elements][32 heads][4 x 32 elements][8 x 4 heads][32 elements][4 heads]
  int64_t table_stride;
  int B, H, groups, heads;  // heads: of a group
  int page, width, pages, box;  // box: tokens of a copy
  int ranges;
  float scale_log2;
  int fault;
  uint64_t wait_ns;
};

// A sequence's length, kept to what its row of the table holds.
__device__ __forceinline__ int length_of(const DecodeParams& P, int n) { return min(max(n, 0), P.width * P.page); }
__device__ __forceinline__ int length_at(const DecodeParams& P, int b) { return length_of(P, P.lengths[b]); }
__device__ __forceinline__ int tiles_of(int n) { return n / kTile + (n % kTile != 0); }

// Tiles of a range: the ranges' even share.  Fewer and longer ranges where that
// leaves many pieces of few sequences: a tile takes about 1.25 us, a piece of a
// sequence 0.1 us in its joining, so that sqrt(0.08 tiles) of a sequence are best.  (72
// tiles, 64 heads, in ranges of 1, 2, 3, 4, 8: 19.3, 16.7, 17.7, 18.5, 23.5 us; 256
// tiles, of 2, 3, 4, 6, 8: 25.7, 24.5, 21.8, 23.1, 25.1.)
__device__ __forceinline__ int64_t share(const DecodeParams& P, int64_t total) {
  const bool small = total >> 31 == 0;  // (a division of 64 bits takes 0.3 us)
  const int64_t even = small ? ((uint32_t)total + P.ranges - 1) / (uint32_t)P.ranges : (total + P.ranges - 1) / P.ranges;
  const int64_t best = (int64_t)(sqrtf(0.08f * ((float)total / (float)P.B)) + 0.5f);
  return max(even, max(best, (int64_t)1));
}

// The pieces of this CTA's range, sequence by sequence; every warp walks them with
// its own cursor and holds the lengths of 32 sequences.
struct Walk {
  int b, t0, left;     // sequence, its first tile here, tiles left of the range
  int nt, len, all;    // of the piece: tiles, length of the sequence and its tiles
  int base, mine;
  __device__ __forceinline__ void load(const DecodeParams& P) {
    base = b;
    const int i = b + (threadIdx.x & 31);
    mine = i < P.B ? P.lengths[i] : 0;  // (as loaded: nothing waits for it here)
  }
  // from tile t_ of sequence b_, whose length is known
  __device__ __forceinline__ void start(const DecodeParams& P, int b_, int t_, int len_, int left_) {
    b = b_, t0 = t_, len = len_, left = left_, nt = 0;
    load(P);  // (needed for the second piece)
  }
  __device__ __forceinline__ bool next(const DecodeParams& P) {
    if (left <= 0) return false;
    if (nt > 0) {
      t0 = 0;
      do {
        if (++b >= P.B) return false;
        if (b >= base + 32) load(P);
        len = length_of(P, __shfl_sync(0xFFFFFFFFu, mine, b - base));
      } while (len == 0);
    }
    all = tiles_of(len);
    nt = min(all - t0, left);
    left -= nt;
    return true;
  }
};

// Inclusive sums of v over the block's threads; *total: over all of them.
// scratch: a word of 64 bits for each warp.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* scratch, int64_t* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int64_t u = __shfl_up_sync(0xFFFFFFFFu, v, s);
    if (lane >= s) v += u;
  }
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  int64_t all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == warp) v += all;
    all += scratch[w];
  }
  __syncthreads();
  *total = all;
  return v;
}

// A range: its sequence at the start, that one's tiles before it and length, its tiles.
struct Range {
  int b, t, len, left;
};

// This CTA's range, to *out in shared memory; whole block.  With up to kThreads
// sequences their lengths are loaded once and summed up once.
__device__ void find_range(const DecodeParams& P, int range, bool names, int64_t* scratch, Range* out) {
  int64_t total = 0, upto = 0;
  int mine = 0;
  bool bad = false;
  if (P.B <= kThreads) {
    if ((int)threadIdx.x < P.B) mine = length_at(P, threadIdx.x), bad = mine != P.lengths[threadIdx.x];
    upto = block_scan(tiles_of(mine), scratch, &total);
  } else {
    for (int b = threadIdx.x; b < P.B; b += kThreads) {
      const int n = length_at(P, b);
      bad |= n != P.lengths[b];
      upto += tiles_of(n);
    }
    block_scan(upto, scratch, &total);
  }
  if (bad && blockIdx.x == 0) atomicOr(P.err, kErrBadExpertId);
  const int64_t per = share(P, total), first = per * range;
  if (first >= total) {
    if (threadIdx.x == 0) {
      *out = Range{0, 0, 0, 0};
      if (names) P.cut[range] = make_int4(0, 0, 0, 0);
    }
  } else {
    int64_t before = 0;
    for (int b0 = 0; b0 < P.B; b0 += kThreads) {
      const int b = b0 + threadIdx.x;
      int64_t all = total;
      if (P.B > kThreads) {
        mine = b < P.B ? length_at(P, b) : 0;
        upto = block_scan(tiles_of(mine), scratch, &all);
      }
      const int64_t end = before + upto, begin = end - tiles_of(mine);
      if (begin <= first && first < end) {
        *out = Range{b, (int)(first - begin), mine, (int)min(per, total - first)};
        if (names) P.cut[range] = make_int4(b, (int)(first - begin), tiles_of(mine), (int)per);
      }
      before += all;
      if (before > first) break;
    }
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
  Range* where = reinterpret_cast<Range*>(tmem_slot + 2);
  float* factor = reinterpret_cast<float*>(smem + kOffTail + 256);   // [heads]
  int64_t* scratch = reinterpret_cast<int64_t*>(smem + kOffTail + 512);
  const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
  // Load warps: the second one where a tile is many copies.  Each that waits for a stage announces its next copies: one
  // that did not could be overtaken by two phases of the stage, and would wait for ever.
  const int loaders = P.box == kTile ? 1 : 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&kv_full[s], loaders), mbar_init(&kv_empty[s], 1);
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
  griddep_wait();
  const int group = blockIdx.x % P.groups, range = blockIdx.x / P.groups;
  const int head0 = group * P.heads, live = min(P.heads, P.H - head0);  // this CTA's heads
  const int slot0 = (2 * range) * P.groups + group;
  if (threadIdx.x < 2) P.done[slot0 + threadIdx.x * P.groups] = 0;
  tmem_fence_before();
  find_range(P, range, group == 0, scratch, where);
  tmem_fence_after();
  Walk w;
  w.start(P, where->b, where->t, where->len, where->left);
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
  const Waits wait{abort_flag, P.err, P.wait_ns};
  const int n_mma = (live + 15) & ~15;

  if (warp < 2) {
    // ---------------- loads ----------------
    const int copies = kTile / P.box;  // of a slab
    int g = 0, piece = 0;
    bool ok = true;
    while (ok && warp < loaders && w.next(P)) {
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
            if (elect_one()) {
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
        if (warp == 0 && i == 0) {  // behind the first tile: its way is longer
          ok = wait(q_empty, (piece & 1) ^ 1);
          if (!ok) {
            ++g;
            break;
          }
          if (elect_one()) {
            mbar_expect_tx(q_full, kSlabs * kHeads * 128);
            tma_load_4d(smem + kOffQ, &map_q, 0, head0, w.b, 0, q_full);
          }
          __syncwarp();
          ++piece;
        }
        row = next;
        // The next tile comes to L2 while no stage is free for it.
        if (i >= kStages - 1 && i + 1 < w.nt) {
          if (copies == 1) {
            const int r = __shfl_sync(0xFFFFFFFFu, row, 0);
            if (r != none && elect_one()) tma_prefetch_3d(&map_c, 0, r, 0);
          } else {
            for (int c = 0; c < copies; ++c) {
              const int r = __shfl_sync(0xFFFFFFFFu, row, c);
              if (r != none && elect_one())
                for (int sl = warp; sl < kSlabs; sl += 2) tma_prefetch_3d(&map_c, 0, r, sl);
            }
          }
          __syncwarp();
        }
      }
    }
    // every issued copy has landed before shared memory is given back
    __syncwarp();
    if (warp < loaders) {
      for (int q = max(0, g - kStages); q < g; ++q) wait.drain(&kv_full[q % kStages], (q / kStages) & 1);
      if (piece > 0) wait.drain(q_full, (piece - 1) & 1);
    }
  } else if (warp == 2) {
    // ---------------- MMAs ----------------
    const uint32_t base = smem_u32(smem);
    const uint32_t q_lo = desc_lo(base + kOffQ, 16), p_lo = desc_lo(base + kOffP, 16);
    const uint32_t id_pv = idesc_bf16(128, n_mma, true, false);
    int g0 = 0, piece = 0;
    bool ok = true;
    while (ok && w.next(P)) {
      ok = wait(q_full, piece & 1);
      if (!ok) break;
      int qi = 0, pi = 0;  // tiles whose scores, whose sums have been issued
      uint64_t since = 0;
      // tokens of a tile, to whole MMA steps: the sequence's last one may have fewer
      auto tokens16 = [&](int i) { return min(kTile, (w.len - (w.t0 + i) * kTile + 15) & ~15); };
      while (pi < w.nt) {
        const int gq = g0 + qi, gp = g0 + pi;
        if (qi < w.nt && qi < pi + 2 && mbar_test(&kv_full[gq % kStages], (gq / kStages) & 1) &&
            mbar_test(&s_free[gq & 1], ((gq >> 1) & 1) ^ 1)) {
          tmem_fence_after();
          if (elect_one()) {
            const uint32_t k_lo = desc_lo(base + (gq % kStages) * kStage, 16);
            const uint32_t d = tmem + kColS + (gq & 1) * kTile, id_qk = idesc_bf16(kHeads, tokens16(qi), false, false);
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
            const int steps = tokens16(pi) / 16;
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k)
              if (k < steps)
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
  } else if (warp == 3) {
    // ---------------- sequences of no tokens ----------------
    for (int b = blockIdx.x; b < P.B; b += gridDim.x)
      if (length_at(P, b) == 0)
        for (int64_t i = lane; i < (int64_t)P.H * (kLatent / 8); i += 32)
          reinterpret_cast<uint4*>(P.out + (int64_t)b * P.H * kLatent)[i] = make_uint4(0, 0, 0, 0);
  } else {
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
        // Rows behind the sequence's end that the last MMA step takes in are zeros: whatever is there must not meet a
        // zero of P.
        if (n % 16 != 0 && ok) {
          uint8_t* st = smem + (g % kStages) * kStage + (tid >> 4) * kSlab + (tid & 7) * 16;
          for (int row = n + ((tid >> 3) & 1); row < ((n + 15) & ~15); row += 2)
            *reinterpret_cast<uint4*>(st + row * 128) = make_uint4(0, 0, 0, 0);
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
        // 32 heads at a time, two quarters of the latent vector
        const int halves = (P.heads + 31) / 32;
#pragma unroll 1
        for (int c = 0; c < 2 * halves; ++c) {
          const int h0 = c / 2 * 32, j0 = (c & 1) * 2;
          if (h0 >= live) break;
          uint32_t o[2][32];
          if (whole) {
            // Elements lie across lanes, heads across columns; a head's elements are wanted side by side.  Read as
            // fragments of 8 x 8 and stored transposed to this warp's rows of P, [head][32 elements] (16-byte chunk c of
            // head h at c ^ (h / 2) % 4), then 16 bytes a lane.
            const int i0 = lane >> 3, column = 8 * i0 + (lane & 7);  // the matrix and head whose address this lane gives
            uint8_t* const turn = smem + kOffP + q * 2048;
            float2 f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = *reinterpret_cast<const float2*>(factor + h0 + 8 * i + 2 * (lane & 3));
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                tmem_ld_rows16_half(tmem + lanes + ((uint32_t)(16 * h) << 16) + (j0 + u) * kHeads + h0, o[u] + 16 * h);
            tmem_wait_ld();
            uint16_t* const out = P.out + ((int64_t)w.b * P.H + head0 + h0 + (lane >> 2)) * kLatent + j0 * 128 + q * 32 + (lane & 3) * 8;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
              for (int c8 = 0; c8 < 4; ++c8) {  // elements 8 c8 .. 8 c8 + 7 of the 32
                uint32_t p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int at = 16 * (c8 >> 1) + 4 * i + 2 * (c8 & 1);
                  p[i] = pack_bf16(__uint_as_float(o[u][at]) * f[i].x, __uint_as_float(o[u][at + 1]) * f[i].y);
                }
                stmatrix4_trans(turn + column * 64 + ((c8 ^ ((column >> 1) & 3)) << 4), p[0], p[1], p[2], p[3]);
              }
              __syncwarp();
              uint4 v[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int h = i * 8 + (lane >> 2);
                v[i] = *reinterpret_cast<const uint4*>(turn + h * 64 + (((lane & 3) ^ ((h >> 1) & 3)) << 4));
              }
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (h0 + i * 8 + (lane >> 2) < live) *reinterpret_cast<uint4*>(out + i * 8 * kLatent + u * 128) = v[i];
              __syncwarp();
            }
          } else {
            // [quarter of the latent vector][32 heads][warp][4 heads] of 32 elements x 4 heads: 16 bytes a lane
            float4* const sums = reinterpret_cast<float4*>(P.sums) +
                                 ((((int64_t)slot * 4 + j0) * halves + h0 / 32) * 4 + q) * 8 * 32 + lane;
#pragma unroll
            for (int u = 0; u < 2; ++u) tmem_ld32(tmem + lanes + (j0 + u) * kHeads + h0, o[u]);
            tmem_wait_ld();
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int j = 0; j < 32; j += 4)
                if (h0 + j < live)
                  sums[u * halves * 4 * 8 * 32 + j / 4 * 32] =
                      make_float4(__uint_as_float(o[u][j]), __uint_as_float(o[u][j + 1]), __uint_as_float(o[u][j + 2]),
                                  __uint_as_float(o[u][j + 3]));
          }
        }
        if (!whole && rows_live && (lane & 3) == 0) {
#pragma unroll
          for (int r = 0; r < 2; ++r)
            P.ml[(int64_t)slot * P.heads + r0 + 8 * r] = make_float2(m[r], l[r]);
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
  // the joining kernel is let in here: waiting from the start it costs more than it saves (one sequence of 4608 tokens
  // 17.1 us, 16.3 so; of 32768, 16 heads, 27.5 and 24.6)
  griddep_launch_dependents();
  if (warp == 2) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols));
  }
}

// The pieces of cut sequences, joined: an item is four heads and a quarter of the
// latent vector of a sequence, an element and four heads a thread, as the pieces
// lie, every fourth piece a part of the CTA.  A part's lanes find the factors of its
// pieces (to its own maximum), 32 at a time, the first kAhead pieces' sums on their way
// meanwhile; the parts meet in shared memory.
template <int kJoinParts, int kAhead>
__global__ void __launch_bounds__(128 * kJoinParts) latent_join_kernel(DecodeParams P) {
  griddep_begin();
  __shared__ int4 list[kMaxRanges];  // sequence, first and last range, first slot's number
  __shared__ uint32_t found[kMaxRanges / 32];
  // A range that starts inside a sequence cuts it, the first such one names it; in the ranges' order, the same list
  // in every CTA.
  __shared__ float4 part_o[kJoinParts][128];
  __shared__ float part_top[kJoinParts][4], part_l[kJoinParts][4];
  constexpr int kThreads = 128 * kJoinParts, kRounds = (kMaxRanges + kThreads - 1) / kThreads;
  int at[kRounds], count = 0;
#pragma unroll
  for (int i = 0; i < kRounds; ++i) {
    const int r = i * kThreads + threadIdx.x;
    int4 cut = make_int4(0, 0, 0, 0);
    if (r < P.ranges) cut = P.cut[r];
    const bool names = cut.y > 0 && cut.y <= cut.w;
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, names);
    if (r < kMaxRanges && (r & 31) == 0) found[r >> 5] = mask;
    at[i] = names ? __popc(mask & ((1u << (r & 31)) - 1)) : -1;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kMaxRanges / 32; ++k) {
#pragma unroll
    for (int i = 0; i < kRounds; ++i)
      if (at[i] >= 0 && k < (i * kThreads + (int)threadIdx.x) >> 5) at[i] += __popc(found[k]);
    count += __popc(found[k]);
  }
#pragma unroll
  for (int i = 0; i < kRounds; ++i)
    if (at[i] >= 0) {
      const int r = i * kThreads + threadIdx.x;
      const int4 cut = P.cut[r];
      const int64_t start = (int64_t)r * cut.w - cut.y;
      list[at[i]] = make_int4(cut.x, r - 1, (int)((start + cut.z - 1) / cut.w), 2 * (r - 1) + (cut.y < cut.w ? 1 : 0));
    }
  __syncthreads();
  const int lane = threadIdx.x & 31, q = (threadIdx.x >> 5) & 3, part = threadIdx.x >> 7, halves = (P.heads + 31) / 32;
  const int quads = P.heads / 4, items = count * P.groups * quads * 4;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    int i = item;
    const int j0 = i & 3;
    i >>= 2;
    const int quad = i % quads;
    i /= quads;
    const int group = i % P.groups;
    const int4 c = list[i / P.groups];
    const int h0 = quad * 4, live = min(P.heads, P.H - group * P.heads);
    if (h0 >= live) continue;
    const int first = c.y, last = c.z;
    auto slot_of = [&](int r) { return (int64_t)(r == first ? c.w : 2 * r) * P.groups + group; };
    float o[4] = {0.f, 0.f, 0.f, 0.f}, l[4] = {0.f, 0.f, 0.f, 0.f};
    float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
    bool complete = true;
    const float4* const sums = reinterpret_cast<const float4*>(P.sums) + (quad & 7) * 32 + lane;
    for (int r0 = first + part; r0 <= last; r0 += 32 * kJoinParts) {
      const int r = r0 + lane * kJoinParts, n = min(32, (last - r0) / kJoinParts + 1);
      const auto sums_at = [&](int k) {
        return sums[((slot_of(r0 + k * kJoinParts) * 4 + j0) * halves + h0 / 32) * 4 * 8 * 32 + q * 8 * 32];
      };
      // the first ones are on their way while the factors are found
      float4 ahead[kAhead > 0 ? kAhead : 1];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (k < n) ahead[k] = sums_at(k);
      float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY}, s[4] = {0.f, 0.f, 0.f, 0.f}, f[4];
      if (r <= last) {
        complete &= P.done[slot_of(r)] != 0;
        const float4* const ml = reinterpret_cast<const float4*>(P.ml + slot_of(r) * P.heads + h0);
        const float4 a = ml[0], b = ml[1];
        m[0] = a.x, m[1] = a.z, m[2] = b.x, m[3] = b.z;
        s[0] = a.y, s[1] = a.w, s[2] = b.y, s[3] = b.w;
      }
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        float to = fmaxf(top[h], m[h]);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) to = fmaxf(to, __shfl_xor_sync(0xFFFFFFFFu, to, d));
        const float off = to == -INFINITY ? 0.f : to, was = exp2f(top[h] - off);
        f[h] = exp2f(m[h] - off);
        o[h] *= was;
        l[h] = l[h] * was + f[h] * s[h];
        top[h] = to;
      }
      const auto add = [&](int k, const float4& v) {
        o[0] += __shfl_sync(0xFFFFFFFFu, f[0], k) * v.x;
        o[1] += __shfl_sync(0xFFFFFFFFu, f[1], k) * v.y;
        o[2] += __shfl_sync(0xFFFFFFFFu, f[2], k) * v.z;
        o[3] += __shfl_sync(0xFFFFFFFFu, f[3], k) * v.w;
      };
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (k < n) add(k, ahead[k]);
#pragma unroll 8
      for (int k = kAhead; k < n; ++k) add(k, sums_at(k));
    }
#pragma unroll
    for (int h = 0; h < 4; ++h) {
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], d);
      if (q == 0 && lane == 0) part_top[part][h] = top[h], part_l[part][h] = l[h];
    }
    part_o[part][q * 32 + lane] = make_float4(o[0], o[1], o[2], o[3]);
    if (__syncthreads_or(!complete)) continue;  // a wait ran out (what is written above is not read)
    // a part adds up a head of the four, or all
#pragma unroll
    for (int h = part; h < 4; h += kJoinParts) {
      float all = -INFINITY, sum = 0.f, den = 0.f;
#pragma unroll
      for (int p = 0; p < kJoinParts; ++p) all = fmaxf(all, part_top[p][h]);
      if (all == -INFINITY) all = 0.f;
#pragma unroll
      for (int p = 0; p < kJoinParts; ++p) {
        const float f = exp2f(part_top[p][h] - all);
        sum += f * reinterpret_cast<const float*>(&part_o[p][q * 32 + lane])[h];
        den += f * part_l[p][h];
      }
      if (h0 + h < live)
        P.out[((int64_t)c.x * P.H + group * P.heads + h0 + h) * kLatent + j0 * 128 + q * 32 + lane] = f32_to_bf16_rn(sum / den);
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
         (size_t)s.slots * ((s.heads + 31) & ~31) * kLatent * sizeof(float);
}

int moe_fp4_latent_decode(const moe_fp4_latent_decode_args* args, void* workspace, size_t workspace_bytes,
                          void* cuda_stream) {
  if (!args) return MOE_FP4_ERR_INVALID_ARG;
  const moe_fp4_latent_decode_args a = *args;
  if (a.B < 0 || a.H < 1 || a.H > MOE_FP4_LATENT_MAX_HEADS || a.page < 16 || a.page % 16 != 0 || a.pages < 1 || a.width < 1 ||
      !finite_scale(a.scale) || a.table_stride < a.width)
    return MOE_FP4_ERR_INVALID_ARG;
  if (a.B > kMaxSequences || (int64_t)a.pages * a.page >= (1LL << 31) || (int64_t)a.width * a.page >= (1LL << 31) || (int64_t)a.B * a.H >= (1LL << 31))
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
  const uint64_t qd[4] = {64, (uint64_t)a.H, (uint64_t)a.B, kSlabs};
  const uint64_t qs[3] = {(uint64_t)a.q_head_stride * 2, (uint64_t)a.q_stride * 2, 128};
  const uint32_t qb[4] = {64, kHeads, 1, kSlabs};
  const uint64_t cd[3] = {64, (uint64_t)a.pages * a.page, kSlabs}, cs[2] = {kRow * 2, 128};
  const uint32_t cb[3] = {64, (uint32_t)P.box, P.box == kTile ? (uint32_t)kSlabs : 1u};
  if (!make_map_4d(&map_q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B) || !make_map_3d(&map_c, a.cache, cd, cs, cb)) return MOE_FP4_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  if (ensure_smem_optin(reinterpret_cast<const void*>(latent_decode_kernel), kSmem) != cudaSuccess) return MOE_FP4_ERR_CUDA;
  if (launch_early(latent_decode_kernel, dim3(s.ranges * s.groups), dim3(kThreads), kSmem, st, map_q, map_c, P) != cudaSuccess)
    return MOE_FP4_ERR_CUDA;
  // at most a sequence is cut for each range but the first
  const int64_t items = (int64_t)std::min(a.B, s.ranges - 1) * s.groups * s.heads;  // a quarter of four heads each
  if (items == 0) return MOE_FP4_OK;
  // Four parts share a sequence's pieces where these are many for the items: the ranges are 20 and more a sequence, or
  // 8 where the items leave a CTA an SM, which then has the registers for loads ahead.  (64 heads, with one part and with
  // four: 6 sequences of 16000 tokens 47.1 and 46.1 us, 8 of 8000 31.0 and 34.7, 16 of 4000 31.9 and 38.6; 16 heads, 8 of
  // 1000 19.5 and 14.4.  Loads ahead: a sequence of 4608 tokens, 64 heads, 16.2 and 14.6; four of 131072 124 and 126.)
  const bool few = items <= num_sms(), many = s.ranges >= (few ? 8 : 20) * (int64_t)a.B;
  auto* const join = !many ? latent_join_kernel<1, 1> : few ? latent_join_kernel<4, 8> : latent_join_kernel<4, 0>;
  const unsigned grid = (unsigned)std::min<int64_t>(items, (many ? 4 : 16) * num_sms());
  return launch_early(join, dim3(grid), dim3(many ? 512 : 128), 0, st, P) == cudaSuccess
             ? MOE_FP4_OK
             : MOE_FP4_ERR_CUDA;
}

}  // extern "C"
