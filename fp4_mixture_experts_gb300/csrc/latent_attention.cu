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
// tensor cores do one's P V and next Q K^T, the other's softmax runs.  An MMA of 128 x
// 128 x 16 takes 105 cycles with A in shared memory (Q) and 73 with A in tensor memory
// (P), so that 128 x 128 scores are 1,260 + 584 cycles of MMAs and, at 16 exponentials
// a cycle, 1,024 of exponentials: the MMAs bound it (8192 tokens, 64 heads, causal:
// 920 us in short runs, 1.49 PFLOP/s, about 1,930 cycles, without any softmax 880; 990 to
// 1030 in a long loop of calls, under the power cap).  S lies in
// tensor memory, a query a lane, so that maximum and sum need no other thread; P
// overwrites it as bf16 and is the MMA's A operand from there; V is the B operand as
// it lies (MN-major).
//
// The running maximum moves only when a score exceeds it by more than 2^8: then a
// warp multiplies its lanes of O, in tensor memory, before it gives P to the MMAs;
// until then P may grow up to 2^8, which costs bf16 nothing.
//
// Shared memory: Q 2 x 3 slabs of [128][64] (96 KB) and a ring of 8 slabs, through
// which 3 of keys and 2 of values go for each step, given back in that order.  (Two
// stages of keys and one of values take the same 128 KB, but a step's values are
// then on their way only when the last one's are used: 8192 tokens, 64 heads 1130 us,
// 1080 without any softmax.)  Warps: 0 loads, 1 issues the MMAs, 2 finds the pieces of
// work and hands them to the others, 3 looks for offsets that are no sequences' (in one
// CTA), 4..7 and 8..11 are the tiles' softmax and results.  The code is about as long as
// an SM's instruction cache is large: what makes it longer costs 1 to 2 us an item.
//
// Items are dealt out to one CTA an SM; where there are few, by their cost: all
// items' steps are numbered through, in the order of sequences, heads and queries,
// and cut into even ranges, wherever that is in an item of some length; its pieces
// leave their sums (fp32), maxima and row sums in the workspace, which a second
// kernel joins in the ranges' order (64 queries behind 30000 tokens, 16 heads: 403 us on
// 16 SMs, 62 so).  The same lengths give the same bits.  Waits are bounded; results
// are stored only by warps none of whose waits ran out.
#include <algorithm>
#include <cfloat>

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
constexpr int kStepSlabs = kQSlabs + kVSlabs;  // of keys, then of values, of a step
constexpr int kRing = 8;                      // slabs
constexpr int kOffRing = 2 * kQSlabs * kSlab;
constexpr int kOffTail = kOffRing + kRing * kSlab;
constexpr int kSmem = kOffTail + 1024 + 1024;
static_assert(kSmem <= kSmemMax, "shared memory");
constexpr uint32_t kCols = 512;               // S of both tiles, O of both
constexpr uint32_t kColO = 256;
constexpr float kGrow = 8.f;                  // log2 of what P may grow to

constexpr int kMinSplit = 8;                  // steps of an item that may be cut
constexpr int kCut = 4;                       // where: at multiples of this
constexpr int kCostTwo = 6, kCostOne = 5;     // see step_cost
constexpr int kMaxRanges = 256;
constexpr int kRows = 2 * kQ;                 // queries of an item

// Sequences of few queries and keys, which have a kernel of their own.
constexpr int kFewQueries = 8, kFewKeys = 32, kFewItems = 12;  // items an SM
__host__ __device__ inline bool few(int64_t nq, int64_t nk) {
  return nq <= kFewQueries && nk <= kFewKeys;
}

struct AttentionParams {
  const int32_t* q_offsets;
  const int32_t* k_offsets;
  uint16_t* out;
  int32_t* err;
  int4* info;          // [range]: flags, first query, queries and head of the item that its last piece leaves unfinished
  int32_t* done;       // [slot][8]: a warp's part of the piece is in the workspace
  float2* ml;          // [slot][queries]: maximum (log2) and sum
  float4* sums;        // [slot][32][queries] of 4 elements
  int B, H, Tq, Tk;
  int ranges, causal;
  int dealt;           // no item is cut, and each CTA has one at most
  int others;          // sequences of few queries and keys are the other kernel's
  float scale_log2;
  int fault;
  uint64_t wait_ns;
};
// a range: it has pieces; the first one begins inside its item; the last one ends before its item does; it is the first
constexpr int kHasPieces = 1, kContinues = 2, kUnfinished = 4, kOnePiece = 8;

struct Sequence {
  int q0, nq, k0, nk;
};
// its four offsets as they are, and taken into the rows
__device__ __forceinline__ int4 offsets_at(const AttentionParams& P, int b) {
  return b < P.B ? make_int4(P.q_offsets[b], P.q_offsets[b + 1], P.k_offsets[b], P.k_offsets[b + 1]) : make_int4(0, 0, 0, 0);
}
__device__ __forceinline__ Sequence sequence_of(const AttentionParams& P, int4 o) {
  Sequence s;
  s.q0 = min(max(o.x, 0), P.Tq), s.nq = max(0, min(o.y, P.Tq) - s.q0);
  s.k0 = min(max(o.z, 0), P.Tk), s.nk = max(0, min(o.w, P.Tk) - s.k0);
  if (P.others && few(s.nq, s.nk)) s.nq = 0;
  return s;
}
// offsets below the ones before them, or behind the rows (INT32_MAX: the rows' end)
__device__ __forceinline__ bool misplaced(const AttentionParams& P, int4 o) {
  const auto behind = [](int v, int rows) { return v > rows && v != INT32_MAX; };
  return o.y < o.x || o.w < o.z || behind(o.x, P.Tq) || behind(o.y, P.Tq) || behind(o.z, P.Tk) || behind(o.w, P.Tk);
}
__device__ __forceinline__ Sequence sequence_at(const AttentionParams& P, int b) { return sequence_of(P, offsets_at(P, b)); }
__device__ __forceinline__ int items_of(const Sequence& s) { return s.nq / kRows + (s.nq % kRows != 0); }

// Steps (tiles of keys) of item t of a sequence's head: what its last query sees.
__device__ __forceinline__ int steps_of(const AttentionParams& P, const Sequence& s, int t) {
  const int behind = P.causal ? max(s.nq - (t + 1) * kRows, 0) : 0;  // queries, each of which sees one key more
  return (max(s.nk - behind, 0) + kK - 1) / kK;
}

// An item costs its steps and one more for its beginning and end; a step of one tile
// of queries, 1.6 us, is to one of two tiles, 2.0 us, as kCostOne to kCostTwo.
__device__ __forceinline__ int step_cost(const Sequence& s, int t) { return s.nq - t * kRows > kQ ? kCostTwo : kCostOne; }
// Cost of the items before t of a sequence's head, t <= items_of(s): under a causal
// mask item u < items - 1 has max(0, 2 (u + 1) + ceil((nk - nq) / 128)) steps.
__device__ __forceinline__ int64_t cost_before(const AttentionParams& P, const Sequence& s, int t) {
  if (t == 0) return 0;
  const int items = items_of(s), whole = min(t, items - 1);
  int64_t cost = whole;
  if (!P.causal) {
    cost += (int64_t)whole * steps_of(P, s, 0);
  } else {
    const int64_t off = (int64_t)s.nk - s.nq, a = off >= 0 ? (off + kK - 1) / kK : -(-off / kK);
    const int64_t u1 = whole;                         // u + 1 = 1 .. u1, from u0 on above 0
    const int64_t u0 = a >= 0 ? 1 : -a / 2 + 1;
    if (u0 <= u1) cost += u1 * (u1 + 1) - (u0 - 1) * u0 + a * (u1 - u0 + 1);
  }
  cost *= kCostTwo;
  if (t == items) cost += (int64_t)(steps_of(P, s, items - 1) + 1) * step_cost(s, items - 1);
  return cost;
}

// A place in the work of all items, in the order of sequences, heads and items: an
// item and a step in it, or behind its last one.  Only items of more than kMinSplit
// steps are cut, at multiples of kCut; a place is the nearest one there is (those
// of several ranges may then be the same).
struct Place {
  int b, h, t, x;
};

// A CTA's share of the work: where it begins (with that sequence) and ends; or, with
// many items, every gridDim.x-th whole one.
struct Range {
  Place from, to;
  Sequence first;
  int strided, snake;
};
constexpr int kManyItems = 6;   // items a CTA
constexpr int kLongSequence = 8;  // items a sequence's head, in the mean

// Inclusive sums over the block's threads; *total: over all of them.  scratch: two
// words for each warp.
__device__ __forceinline__ longlong2 block_scan(longlong2 v, longlong2* scratch, longlong2* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const long long x = __shfl_up_sync(0xFFFFFFFFu, v.x, s), y = __shfl_up_sync(0xFFFFFFFFu, v.y, s);
    if (lane >= s) v.x += x, v.y += y;
  }
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  longlong2 all = make_longlong2(0, 0);
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == warp) v.x += all.x, v.y += all.y;
    all.x += scratch[w].x, all.y += scratch[w].y;
  }
  __syncthreads();
  *total = all;
  return v;
}

// a / b, by a division of 32 bits where that does
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return (uint64_t)a >> 32 == 0 && (uint64_t)b >> 32 == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// The nearest place to `cost` behind an item's beginning.
__device__ __forceinline__ Place place_in(const AttentionParams& P, const Sequence& s, int b, int h, int t, int cost) {
  const int n = steps_of(P, s, t), c = step_cost(s, t);
  int x = 2 * cost > (n + 1) * c ? n : 0;
  if (n > kMinSplit) {
    x = (cost / c + kCut / 2) / kCut * kCut;
    if (x + kCut / 2 > n) x = n;
  }
  return Place{b, h, t, x};
}

// This CTA's range, to *out in shared memory; whole block.
//
// With kManyItems items for each CTA they stay whole and are dealt out in turn, a
// sequence's last queries first, its heads side by side: what runs at the same time
// then reads the same keys (8192 tokens, 64 heads, 13.5 items a CTA: 1129 us, 1285 with
// even ranges of whole heads; 4608 tokens, 7.6 items: 393 and 449).  Under a causal
// mask a long sequence's items cost less one after the other, so that every second
// round is dealt out backwards (4608 tokens 343 -> 321 us, 8192 974 -> 936, 16384 with 16 heads
// 1025 -> 924; 32 sequences of 2 items 126 -> 131, so these are not; before the results' wider stores).
__device__ void find_range(const AttentionParams& P, int range, longlong2* scratch, Range* out) {
  const bool once = P.B <= kThreads;  // each sequence has its thread
  Sequence s{};
  longlong2 sum = make_longlong2(0, 0), total, upto;  // items, and their cost
  int64_t each = 0;                                   // a head's cost of this thread's sequence
  if (threadIdx.x == 0) out->from = out->to = Place{P.B, 0, 0, 0};
  auto look = [&](int b) {
    s = sequence_at(P, b);
    each = cost_before(P, s, items_of(s));
    return make_longlong2((long long)items_of(s) * P.H, each * P.H);
  };
  for (int b = threadIdx.x; b < (once ? kThreads : P.B); b += kThreads) {
    const longlong2 v = look(b);
    sum.x += v.x, sum.y += v.y;
  }
  upto = block_scan(sum, scratch, &total);
  const bool strided = total.x >= (long long)kManyItems * gridDim.x;
  if (threadIdx.x == 0) {
    out->strided = strided;
    out->snake = P.causal && total.x >= (long long)kLongSequence * P.B * P.H;
  }
  if (strided) {
    if (threadIdx.x == 0) {
      out->from = Place{0, 0, 0, 0};
      out->first = sequence_at(P, 0);
    }
  } else {
    const int64_t even = quotient(total.y, P.ranges), rest = total.y - even * P.ranges;
    int64_t at[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) at[i] = even * (range + i) + min((int64_t)(range + i), rest);
    int64_t before = 0;
    for (int b0 = 0; b0 < P.B; b0 += kThreads) {
      longlong2 all = total;
      if (!once) upto = block_scan(look(b0 + threadIdx.x), scratch, &all);
      const int64_t end = before + upto.y, begin = end - each * P.H;
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {
        if (!(begin <= at[i] && at[i] < end)) continue;
        const int64_t y = at[i] - begin, h = quotient(y, each), z = y - h * each;
        int lo = 0, hi = items_of(s);  // the last item that begins at or before z
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (cost_before(P, s, mid) <= z)
            lo = mid;
          else
            hi = mid;
        }
        (i == 0 ? out->from : out->to) = place_in(P, s, b0 + (int)threadIdx.x, (int)h, lo, (int)(z - cost_before(P, s, lo)));
        if (i == 0) out->first = s;
      }
      before += all.y;
      if (before > at[1]) break;
    }
  }
  __syncthreads();
}

// The same by one warp, for up to 32 sequences, a lane each: without the block's
// barriers, and with the search for an item in one step.
__device__ __forceinline__ Range find_range_by_warp(const AttentionParams& P, int range) {
  const int lane = threadIdx.x & 31;
  Range out;
  const Sequence mine = sequence_at(P, lane);
  out.first = Sequence{__shfl_sync(0xFFFFFFFFu, mine.q0, 0), __shfl_sync(0xFFFFFFFFu, mine.nq, 0),
                       __shfl_sync(0xFFFFFFFFu, mine.k0, 0), __shfl_sync(0xFFFFFFFFu, mine.nk, 0)};
  out.from = out.to = Place{0, 0, 0, 0};
  out.strided = 1, out.snake = 0;
  if (P.dealt) return out;
  const int64_t each = cost_before(P, mine, items_of(mine));
  longlong2 upto = make_longlong2((long long)items_of(mine) * P.H, each * P.H);
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(0xFFFFFFFFu, upto.x, d), y = __shfl_up_sync(0xFFFFFFFFu, upto.y, d);
    if (lane >= d) upto.x += x, upto.y += y;
  }
  const int64_t items = __shfl_sync(0xFFFFFFFFu, upto.x, 31), total = __shfl_sync(0xFFFFFFFFu, upto.y, 31);
  out.strided = items >= (int64_t)kManyItems * gridDim.x;
  out.snake = P.causal && items >= (int64_t)kLongSequence * P.B * P.H;
  if (out.strided) return out;
  out.from = out.to = Place{P.B, 0, 0, 0};
  const int64_t even = quotient(total, P.ranges), rest = total - even * P.ranges;
#pragma unroll 1
  for (int i = 0; i < 2; ++i) {
    const int64_t at = even * (range + i) + min((int64_t)(range + i), rest);
    const uint32_t where = __ballot_sync(0xFFFFFFFFu, upto.y - each * P.H <= at && at < upto.y);
    if (where == 0) continue;  // (behind all)
    const int b = __ffs(where) - 1;
    const Sequence s{__shfl_sync(0xFFFFFFFFu, mine.q0, b), __shfl_sync(0xFFFFFFFFu, mine.nq, b),
                     __shfl_sync(0xFFFFFFFFu, mine.k0, b), __shfl_sync(0xFFFFFFFFu, mine.nk, b)};
    const int64_t head = __shfl_sync(0xFFFFFFFFu, each, b), y = at - (__shfl_sync(0xFFFFFFFFu, upto.y, b) - head * P.H);
    const int h = (int)quotient(y, head);
    const int64_t z = y - h * head;
    int64_t before = 0;
    int lo = 0, n = items_of(s);  // the last item that begins at or before z is one of these
    do {
      const int step = (n + 31) / 32;
      const int64_t c = lane * step < n ? cost_before(P, s, lo + lane * step) : z + 1;
      const int k = 31 - __clz(__ballot_sync(0xFFFFFFFFu, c <= z));
      before = __shfl_sync(0xFFFFFFFFu, c, k);
      lo += k * step, n = min(step, n - k * step);
    } while (n > 1);
    (i == 0 ? out.from : out.to) = place_in(P, s, b, h, lo, (int)(z - before));
    if (i == 0) out.first = s;
  }
  return out;
}

// A piece of an item, as the warps hand it on in shared memory.
struct Piece {
  int h, q0, rows, k0, nk;  // rows 0: no more pieces
  int n, from, to;          // steps of the item, of the piece
  int lim[2], upto[2];      // of either tile: keys that its first query sees, where its steps end
  int slot;                 // of its sums, if it is not the whole item
  int g;                    // steps of the pieces before it
};
constexpr int kHanded = 3;  // pieces on their way

// The pieces of a CTA's share, item by item; one warp walks them and holds 32
// sequences, one a lane.
struct Pieces {
  Place at, end;      // at.t counts a sequence's items of all heads where they are dealt out in turn (begun: to an even one next)
  bool begun, strided;
  int step[2];        // to the next item of those dealt out in turn, from an even and from an odd one
  int base;
  int4 mine;          // this lane's sequence's offsets (as loaded: nothing waits for them here)
  Sequence s;         // the current one
  __device__ __forceinline__ void load(const AttentionParams& P) {
    base = at.b;
    mine = offsets_at(P, base + (threadIdx.x & 31));
  }
  __device__ __forceinline__ void start(const AttentionParams& P, const Range& r) {
    at = r.from, end = r.to, s = r.first, strided = r.strided;
    begun = at.x > 0 && at.x >= steps_of(P, s, at.t);  // behind its end: the next one begins
    const int n = gridDim.x, mine = blockIdx.x;
    step[0] = r.snake ? 2 * (n - 1 - mine) + 1 : n;
    step[1] = r.snake ? 2 * mine + 1 : n;
    if (strided) at.t = mine - step[1], begun = true;
    load(P);  // (needed from the second sequence on)
  }
  __device__ __forceinline__ void next_sequence(const AttentionParams& P) {
    if (++at.b >= base + 32) load(P);
    const int l = at.b - base;
    s = sequence_of(P, make_int4(__shfl_sync(0xFFFFFFFFu, mine.x, l), __shfl_sync(0xFFFFFFFFu, mine.y, l),
                                 __shfl_sync(0xFFFFFFFFu, mine.z, l), __shfl_sync(0xFFFFFFFFu, mine.w, l)));
  }
  __device__ __forceinline__ bool next(const AttentionParams& P, Piece& p) {
    int t;
    bool last = false;
    if (strided) {
      at.t += begun ? step[1] : step[0];
      begun = !begun;
      int count;
      while (at.b < P.B && at.t >= (count = items_of(s) * P.H)) {
        at.t -= count;
        next_sequence(P);
      }
      if (at.b >= P.B) return false;
      const int row = at.t / P.H;
      p.h = at.t - row * P.H;
      t = items_of(s) - 1 - row;
    } else {
      if (begun) {
        if (at.b == end.b && at.h == end.h && at.t == end.t) return false;
        at.x = 0;
        if (++at.t >= items_of(s)) {
          at.t = 0;
          if (++at.h == P.H) {
            at.h = 0;
            do next_sequence(P);
            while (at.b < P.B && s.nq == 0);
          }
        }
      }
      begun = true;
      last = at.b == end.b && at.h == end.h && at.t == end.t;
      if (at.b >= P.B || (last && at.x == end.x)) return false;
      p.h = at.h, t = at.t;
    }
    p.n = steps_of(P, s, t);
    p.q0 = s.q0 + t * kRows, p.rows = min(kRows, s.nq - t * kRows);
    p.k0 = s.k0, p.nk = s.nk;
    p.from = at.x, p.to = last ? end.x : p.n;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = min(p.rows, (i + 1) * kQ) - i * kQ;  // queries of the tile
      p.lim[i] = P.causal ? t * kRows + i * kQ + 1 + s.nk - s.nq : s.nk;
      const int most = P.causal ? min(s.nk, p.lim[i] + r - 1) : s.nk;  // what its last one sees
      p.upto[i] = r > 0 && most > 0 ? min((most + kK - 1) / kK, p.to) : 0;
    }
    return true;
  }
};

// 32 bytes, in one store where they start on as many.
__device__ __forceinline__ void store32(void* p, const uint4& a, const uint4& b, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
                 "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = a;
    static_cast<uint4*>(p)[1] = b;
  }
}

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
  uint64_t* k_full = q_empty + 1;       // [step % 2]: the step's keys have landed,
  uint64_t* v_full = k_full + 2;        // its values,
  uint64_t* k_empty = v_full + 2;       // and are given back
  uint64_t* v_empty = k_empty + 2;
  uint64_t* s_full = v_empty + 2;       // [tile]
  uint64_t* p_full = s_full + 2;        // [tile], four warps
  uint64_t* o_full = p_full + 2;        // [tile]
  uint64_t* o_free = o_full + 2;        // [tile], four warps
  uint64_t* mma_done = o_free + 2;
  uint64_t* piece_full = mma_done + 1;  // [handed]
  uint64_t* piece_empty = piece_full + kHanded;  // [handed], ten warps
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(piece_empty + kHanded);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Range* share = reinterpret_cast<Range*>(smem + kOffTail + 320);
  longlong2* scratch = reinterpret_cast<longlong2*>(smem + kOffTail + 384);
  Piece* handed = reinterpret_cast<Piece*>(smem + kOffTail + 640);   // [handed]
  const int warp = uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1), mbar_init(q_empty, 1);
    for (int s = 0; s < 8; ++s) mbar_init(&k_full[s], 1);  // (the four pairs)
    for (int t = 0; t < 2; ++t)
      mbar_init(&s_full[t], 1), mbar_init(&p_full[t], 4), mbar_init(&o_full[t], 1), mbar_init(&o_free[t], 4);
    mbar_init(mma_done, 1);
    for (int s = 0; s < kHanded; ++s) mbar_init(&piece_full[s], 1), mbar_init(&piece_empty[s], 10);
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
  const int slot0 = 2 * blockIdx.x;
  if (threadIdx.x < 16) P.done[slot0 * 8 + threadIdx.x] = 0;
  tmem_fence_before();
  const bool by_warp = P.B <= 32;  // (dealt is only so)
  if (by_warp)
    __syncthreads();
  else
    find_range(P, blockIdx.x, scratch, share);
  tmem_fence_after();
  const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
  const Waits wait{abort_flag, P.err, P.wait_ns};
  // the next piece, from the warp that walks them; false: there is none, or a wait ran out
  int seen_pieces = 0;
  bool ok = true;
  Piece w;
  auto next_piece = [&] {
    const int s = seen_pieces % kHanded;
    if (!(ok = wait(&piece_full[s], (seen_pieces / kHanded) & 1))) return false;
    w = handed[s];
    __syncwarp();
    if (lane == 0) mbar_arrive(&piece_empty[s]);
    ++seen_pieces;
    return w.rows > 0;
  };

  if (warp < 4) {
    set_registers_fewer<kRegsFew>();
    if (warp == 0) {
      // ---------------- loads ----------------
      int items = 0, g = 0;  // items with keys, steps
      // the step's slab j goes where the ring's eighth slab before it was
      auto given_back = [&](int j) {
        const int n = g * kStepSlabs + j - kRing, gn = n / kStepSlabs;
        if (n < 0) return true;
        return wait(n - gn * kStepSlabs < kQSlabs ? &k_empty[gn & 1] : &v_empty[gn & 1], (gn >> 1) & 1);
      };
      auto place = [&](int j) { return smem + kOffRing + (g * kStepSlabs + j) % kRing * kSlab; };
      int k_steps = 0, v_steps = 0;  // announced
      while (ok && next_piece()) {
        if (w.from >= w.to) continue;
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
        for (int i = w.from; i < w.to && ok; ++i, ++g) {
          const int row = w.k0 + i * kK;
          const bool withheld = P.fault && g == 0 && w.from == 0 && w.h == 0;
          for (int j = 0; j < kStepSlabs; ++j) {
            if (!(ok = given_back(j))) break;
            uint64_t* const bar = j < kQSlabs ? &k_full[g & 1] : &v_full[g & 1];
            if (j == 0 && withheld) continue;
            if (elect_one()) {
              if (j == 0 || (j == 1 && withheld)) mbar_expect_tx(bar, kQSlabs * kSlab);
              if (j == kQSlabs) mbar_expect_tx(bar, kVSlabs * kSlab);
              // 0, 1: keys, 2: their rotary part, 3, 4: values (which lie behind the keys)
              if (j == kQSlabs - 1)
                tma_load_3d(place(j), &map_rope, 0, 0, row, bar);
              else
                tma_load_3d(place(j), &map_kv, (j < kQSlabs ? j : j - 1) * 64, w.h, row, bar);
            }
            __syncwarp();
            if (j == 0 || (j == 1 && withheld)) ++k_steps;
            if (j == kQSlabs) ++v_steps;
          }
        }
      }
      // every issued copy has landed before shared memory is given back
      __syncwarp();
      for (int q = max(0, k_steps - 2); q < k_steps; ++q) wait.drain(&k_full[q & 1], (q >> 1) & 1);
      for (int q = max(0, v_steps - 2); q < v_steps; ++q) wait.drain(&v_full[q & 1], (q >> 1) & 1);
      if (items > 0) wait.drain(q_full, (items - 1) & 1);
    } else if (warp == 1) {
      // ---------------- MMAs ----------------
      const uint32_t base = smem_u32(smem);
      constexpr uint32_t id_pv = idesc_bf16(kQ, kValue, false, true), id_pv_half = idesc_bf16(kQ, kValue / 2, false, true);
      int items = 0, g = 0, use[2] = {0, 0}, turn[2] = {0, 0};  // items, steps, turns of O's and of P's barriers
      auto keys16 = [&](int i) { return min(kK, (w.nk - i * kK + 15) & ~15); };  // of a tile, to whole MMA steps
      // S of tile t with the keys of step gk of the ring
      auto qk = [&](int t, int gk, uint32_t id_qk) {
        if (elect_one()) {
          const uint32_t q_lo = desc_lo(base + t * kQSlabs * kSlab, 16);
#pragma unroll
          for (int j = 0; j < kQSlabs; ++j) {
            const uint32_t k_lo = desc_lo(base + kOffRing + (gk * kStepSlabs + j) % kRing * kSlab, 16);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_ss(tmem + t * kK, desc(q_lo + ((j * kSlab + k * 32) >> 4)), desc(k_lo + ((k * 32) >> 4)), id_qk, j > 0 || k > 0);
          }
          umma_commit(&s_full[t]);
        }
        __syncwarp();
      };
      while (ok && next_piece()) {
        if (w.from >= w.to) continue;
        if (!(ok = wait(q_full, items & 1) && wait(&k_full[g & 1], (g >> 1) & 1))) break;
        tmem_fence_after();
        uint32_t id_qk = idesc_bf16(kQ, keys16(w.from), false, false);
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (w.from < w.upto[t]) qk(t, g, id_qk);
        if (elect_one()) {
          umma_commit(&k_empty[g & 1]);
          if (w.to - w.from == 1) umma_commit(q_empty);
        }
        __syncwarp();
        for (int i = w.from; i < w.to && ok; ++i, ++g) {
          const bool more = i + 1 < w.to;
          const int steps = keys16(i) / 16;
          if (more) id_qk = idesc_bf16(kQ, keys16(i + 1), false, false);
          const uint32_t nv = g * kStepSlabs + kQSlabs;  // the values' slabs
          const uint32_t v_at[2] = {base + kOffRing + nv % kRing * kSlab, base + kOffRing + (nv + 1) % kRing * kSlab};
          // (not earlier: they may still be on their way while the keys' MMAs run)
          if (!(ok = wait(&v_full[g & 1], (g >> 1) & 1))) break;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (i >= w.upto[t] || !ok) continue;
            ok = wait(&p_full[t], turn[t] & 1);
            if (ok && i == w.from) ok = wait(&o_free[t], (use[t] & 1) ^ 1), ++use[t];
            if (!ok) break;
            ++turn[t];
            tmem_fence_after();
            if (elect_one()) {
              const uint32_t o = tmem + kColO + t * kValue, p = tmem + t * kK;
              if (v_at[1] > v_at[0] && steps == kK / 16) {
                const uint32_t v_lo = desc_lo(v_at[0], kSlab);
#pragma unroll
                for (int k = 0; k < kK / 16; ++k)
                  tc::umma_tmem_a(o, p + 8 * k, desc(v_lo + ((k * 2048) >> 4)), id_pv, i > w.from || k > 0);
              } else {
                // the ring's last slab and its first, or the sequence's last keys: half of the values at a time.  (A condition
                // on every MMA of the usual case costs 3% of a long prompt.)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                  const uint32_t v_lo = desc_lo(v_at[u], kSlab);
#pragma unroll 1
                  for (int k = 0; k < steps; ++k)
                    tc::umma_tmem_a(o + u * kValue / 2, p + 8 * k, desc(v_lo + ((k * 2048) >> 4)), id_pv_half, i > w.from || k > 0);
                }
              }
              if (i == w.upto[t] - 1) umma_commit(&o_full[t]);
              // the values are given back behind their last reader, ahead of the keys of the next step
              if (t == 1 || i >= w.upto[1]) umma_commit(&v_empty[g & 1]);
            }
            __syncwarp();
            if (i + 1 < w.upto[t]) {
              if (!(ok = wait(&k_full[(g + 1) & 1], ((g + 1) >> 1) & 1))) break;
              tmem_fence_after();
              qk(t, g + 1, id_qk);
            }
          }
          if (!ok) break;
          if (more && elect_one()) {
            umma_commit(&k_empty[(g + 1) & 1]);
            if (i + 2 == w.to) umma_commit(q_empty);
          }
          __syncwarp();
        }
        ++items;
      }
      __syncwarp();
      if (elect_one()) umma_commit(mma_done);
      __syncwarp();
      wait.drain(mma_done, 0);
    } else if (warp == 2) {
      // ---------------- the share's pieces ----------------
      Pieces all;
      all.start(P, by_warp ? find_range_by_warp(P, blockIdx.x) : *share);
      int count = 0, steps = 0, flags = 0;
      int4 unfinished = make_int4(0, 0, 0, 0);
      while (true) {
        Piece p{};
        const bool more = all.next(P, p);
        const int s = count % kHanded;
        if (more) {
          p.slot = slot0 + (count > 0 ? 1 : 0);
          p.g = steps;
          steps += p.to - p.from;
          flags |= kHasPieces | (count == 0 && p.from > 0 ? kContinues : 0);
          if (p.to < p.n) {
            flags |= kUnfinished | (count == 0 ? kOnePiece : 0);
            unfinished = make_int4(0, p.q0, p.rows, p.h);
          }
        }
        if (!ok || !(ok = wait(&piece_empty[s], ((count / kHanded) & 1) ^ 1))) {
          if (!more) break;
          continue;  // (the flags are needed still)
        }
        if (lane == 0) {
          handed[s] = p;
          mbar_arrive(&piece_full[s]);
        }
        ++count;
        if (!more) break;
      }
      if (lane == 0) P.info[blockIdx.x] = make_int4(flags, unfinished.y, unfinished.z, unfinished.w);
    } else if (__builtin_expect(blockIdx.x == 0, 0)) {
      // ---------------- offsets that are no sequences' ----------------
      // (out of the way and short: laid out among the other warps' code and unrolled it costs them 1 to 3%)
      bool bad = false;
#pragma unroll 1
      for (int b = lane; b < P.B; b += 32) bad |= misplaced(P, offsets_at(P, b));
      if (bad) atomicOr(P.err, kErrBadExpertId);
    }
  } else {
    set_registers_more<kRegsMany>();
    // ---------------- softmax, rescaling, results ----------------
    const int t = (warp >> 2) - 1, row = (warp & 3) * 32 + lane;  // tile; this thread's query of it
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + t * kK + lanes, o_col = tmem + kColO + t * kValue + lanes;
    int turn = 0, use = 0;
    while (ok && next_piece()) {
      const int here = min(w.rows - t * kQ, kQ);  // queries of the tile
      const int seen = P.causal ? min(w.nk, w.lim[t] + row) : w.nk;  // keys that this query sees
      const bool rows_here = (warp & 3) * 32 < here;  // (else nothing is read of what lies in this warp's lanes)
      float m = -INFINITY, l = 0.f;
      for (int i = w.from; i < w.upto[t]; ++i, ++turn) {
        if (!(ok = wait(&s_full[t], turn & 1))) break;
        tmem_fence_after();
        if (rows_here) {
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
            if (i > w.from) {
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
        }
        const int keys = w.nk - i * kK;
        if (keys < kK && keys % 16 != 0) {
          // Rows behind the sequence's end that the last MMA step takes in are zeros: whatever is there must not meet a
          // zero of P.  (Both tiles' warps may write them.)
          const int g = w.g + i - w.from, nv = g * kStepSlabs + kQSlabs;
          if (!(ok = wait(&v_full[g & 1], (g >> 1) & 1))) break;
          uint8_t* const v = smem + kOffRing + (nv + ((warp >> 1) & 1)) % kRing * kSlab + (lane & 7) * 16;
          for (int r = keys + (lane >> 3) + 4 * (warp & 1); r < ((keys + 15) & ~15); r += 8)
            *reinterpret_cast<uint4*>(v + r * 128) = make_uint4(0, 0, 0, 0);
          fence_proxy_async();
        }
        tmem_wait_st();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[t]);
      }
      if (!ok) break;
      const bool whole = w.from == 0 && w.to == w.n, any = w.from < w.upto[t], mine = row < here;
      uint16_t* const out = P.out + ((int64_t)(w.q0 + t * kQ + row) * P.H + w.h) * kValue;
      const bool wide = (reinterpret_cast<uintptr_t>(P.out) & 31) == 0;
      if (whole && !any) {
        if (mine)
          for (int c = 0; c < kValue; c += 8) *reinterpret_cast<uint4*>(out + c) = make_uint4(0, 0, 0, 0);
        continue;
      }
      if (any) {
        if (!(ok = wait(&o_full[t], use & 1))) break;
        ++use;
        tmem_fence_after();
        const float inv = seen > 0 ? 1.f / l : 0.f;  // a query that sees nothing: zeros
        float4* const sums = P.sums + (int64_t)w.slot * (kValue / 4) * kRows + t * kQ + row;
#pragma unroll 1
        for (int c = rows_here ? 0 : kValue; c < kValue; c += 32) {
          uint32_t o[32];
          tmem_ld32(o_col + c, o);
          tmem_wait_ld();
          if (whole) {
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t* const e = o + 8 * j;
              const auto two = [&](int k) { return pack_bf16(__uint_as_float(e[k]) * inv, __uint_as_float(e[k + 1]) * inv); };
              v[j] = make_uint4(two(0), two(2), two(4), two(6));
            }
            // A store touches a line for each of its lanes, so that 32 bytes a lane take half the time of 16 (2.6 and 1.5 us
            // an item; 64 bytes of a row on four lanes, by shuffles, 1.5 to 1.6).
            if (mine) store32(out + c, v[0], v[1], wide), store32(out + c + 16, v[2], v[3], wide);
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              sums[(c + j) / 4 * kRows] = make_float4(__uint_as_float(o[j]), __uint_as_float(o[j + 1]),
                                                      __uint_as_float(o[j + 2]), __uint_as_float(o[j + 3]));
          }
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&o_free[t]);
      }
      if (!whole) {
        // (a maximum above -infinity also where all scores are that: the query has seen something)
        P.ml[(int64_t)w.slot * kRows + t * kQ + row] = make_float2(seen > w.from * kK ? fmaxf(m, -FLT_MAX) : m, l);
        if (lane == 0) P.done[w.slot * 8 + warp - 4] = 1;
      }
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

// ---- sequences of few queries and keys ----
// A tile of 128 queries and 128 keys of a head takes the kernel above ~3 us on an SM,
// however few of them there are.  Here a warp takes a head of a sequence, four
// queries at a time, all its keys at once: for S a lane has a key and reads its row,
// the queries come from shared memory (fp32, the same word for all lanes); for P V a
// lane has four elements of the values and P comes by shuffles.  (64 sequences, 128
// heads, of 1 x 1, 4 x 16, 8 x 32 queries and keys: 24, 36, 112 us; with tensor cores 180 to
// 195; 33 of 1 or 2 tokens 20 and 103; one token, 16 heads, 4.5 and 9.4.  With 16 queries
// the sequences of a mixed batch take 74 us instead of 62, with more keys the rows'
// loads, 16 bytes a lane, take longer than the MMAs.)  For fewer than kFewItems heads of
// sequences an SM a launch more does not pay (10 sequences, 128 heads: 35 us, 46 with both),
// unless it is the only one.
struct FewParams {
  AttentionParams a;
  const uint16_t *q, *kv, *rope;
  int64_t q_stride, q_head_stride, kv_stride, kv_head_stride, rope_stride;
  int only;  // no other kernel looks at the offsets
};
constexpr int kFewWarps = 4, kFewGroup = 4;

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}

__global__ void __launch_bounds__(32 * kFewWarps) latent_attention_few_kernel(const FewParams P) {
  griddep_begin();
  constexpr int kD = kNope + kRope;
  __shared__ __align__(16) float queries[kFewWarps][kFewGroup][kD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quads = (P.a.H + kFewWarps - 1) / kFewWarps;
  const int b = blockIdx.x / quads, h = (blockIdx.x - b * quads) * kFewWarps + warp;
  AttentionParams all = P.a;
  all.others = 0;
  const int4 o4 = offsets_at(all, b);
  const Sequence s = sequence_of(all, o4);
  if (P.only && h == 0 && lane == 0 && misplaced(all, o4)) atomicOr(&g_attention_err[0], kErrBadExpertId);
  if (h >= P.a.H || !few(s.nq, s.nk)) return;  // (no barrier follows)
  float(&q)[kFewGroup][kD] = queries[warp];
  const int key = min(lane, max(s.nk - 1, 0));
  const uint16_t* const k_row = P.kv + (s.k0 + (int64_t)key) * P.kv_stride + h * P.kv_head_stride;
  const uint16_t* const r_row = P.rope + (s.k0 + (int64_t)key) * P.rope_stride;
  const uint16_t* const values = P.kv + (int64_t)s.k0 * P.kv_stride + h * P.kv_head_stride + kNope + lane * 4;
  for (int g0 = 0; g0 < s.nq; g0 += kFewGroup) {
    const int n = min(kFewGroup, s.nq - g0);
    __syncwarp();
    for (int i = lane; i < kFewGroup * (kD / 8); i += 32) {
      const int r = i / (kD / 8), c = i - r * (kD / 8);
      float f[8] = {};
      if (r < n) unpack8(*reinterpret_cast<const uint4*>(P.q + (s.q0 + (int64_t)g0 + r) * P.q_stride + h * P.q_head_stride + c * 8), f);
#pragma unroll
      for (int j = 0; j < 8; ++j) q[r][c * 8 + j] = f[j] * P.a.scale_log2;
    }
    __syncwarp();
    float p[kFewGroup] = {}, l[kFewGroup], o[kFewGroup][4] = {};
    if (lane < s.nk) {
#pragma unroll 8
      for (int c = 0; c < kD / 8; ++c) {
        float f[8];
        unpack8(c < kNope / 8 ? *reinterpret_cast<const uint4*>(k_row + c * 8)
                              : *reinterpret_cast<const uint4*>(r_row + (c - kNope / 8) * 8), f);
#pragma unroll
        for (int i = 0; i < kFewGroup; ++i) {
          const float4 a = *reinterpret_cast<const float4*>(&q[i][c * 8]), e = *reinterpret_cast<const float4*>(&q[i][c * 8 + 4]);
          p[i] = fmaf(a.x, f[0], fmaf(a.y, f[1], fmaf(a.z, f[2], fmaf(a.w, f[3], p[i]))));
          p[i] = fmaf(e.x, f[4], fmaf(e.y, f[5], fmaf(e.z, f[6], fmaf(e.w, f[7], p[i]))));
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kFewGroup; ++i) {
      const float v = lane < s.nk && (!P.a.causal || lane <= g0 + i + s.nk - s.nq) ? p[i] : -INFINITY;
      float top = v;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
      p[i] = exp2f(v - (top == -INFINITY ? 0.f : top));
      l[i] = p[i];
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], d);
    }
#pragma unroll 4
    for (int j = 0; j < s.nk; ++j) {
      const uint2 w = *reinterpret_cast<const uint2*>(values + j * P.kv_stride);
      const float v[4] = {__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                          __uint_as_float(w.y & 0xFFFF0000u)};
#pragma unroll
      for (int i = 0; i < kFewGroup; ++i) {
        const float pj = __shfl_sync(0xFFFFFFFFu, p[i], j);
#pragma unroll
        for (int d = 0; d < 4; ++d) o[i][d] = fmaf(pj, v[d], o[i][d]);
      }
    }
#pragma unroll
    for (int i = 0; i < kFewGroup; ++i) {
      const int seen = P.a.causal ? min(s.nk, g0 + i + 1 + s.nk - s.nq) : s.nk;
      const float inv = seen > 0 ? 1.f / l[i] : 0.f;  // a query that sees nothing: zeros
      if (i < n)
        *reinterpret_cast<uint2*>(P.a.out + ((s.q0 + (int64_t)g0 + i) * P.a.H + h) * kValue + lane * 4) =
            make_uint2(pack_bf16(o[i][0] * inv, o[i][1] * inv), pack_bf16(o[i][2] * inv, o[i][3] * inv));
    }
  }
}

// The pieces of items that several ranges share, joined in the ranges' order: a
// CTA an item and eight elements of its queries' results, a query a thread, the
// loads of kJoinAhead pieces at a time on their way (500 queries behind 20000 tokens, one
// head, 40 pieces an item: 34 us, 52 with one at a time).
constexpr int kJoinChunks = kValue / 8, kJoinAhead = 4;
__global__ void __launch_bounds__(kRows) latent_attention_join_kernel(AttentionParams P) {
  griddep_begin();
  constexpr int kWords = kMaxRanges / 32;
  __shared__ uint32_t first[kWords], has[kWords], ends[kWords];  // bits of the ranges
  __shared__ int busy[kMaxRanges];    // the ranges that have pieces
  __shared__ int4 chains[kMaxRanges]; // of each cut item: its head, its first range's slot and place in busy, its pieces
  __shared__ int2 queries[kMaxRanges];  // the first one, how many
  const int mine = threadIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;  // (kRows threads, a range each)
  const int4 info = mine < P.ranges ? P.info[mine] : make_int4(0, 0, 0, 0);
  const bool busy_range = info.x & kHasPieces, one = info.x & kOnePiece;
  // an item's first piece begins it and leaves it unfinished; the first pieces of the ranges behind follow, up to the
  // first that ends it
  const bool begins = (info.x & kUnfinished) && !((info.x & kContinues) && one);
  const uint32_t f = __ballot_sync(0xFFFFFFFFu, begins), h = __ballot_sync(0xFFFFFFFFu, busy_range);
  const uint32_t e = __ballot_sync(0xFFFFFFFFu, busy_range && !((info.x & kUnfinished) && one));
  if (lane == 0) first[warp] = f, has[warp] = h, ends[warp] = e;
  __syncthreads();
  const uint32_t below = (1u << lane) - 1;
  int count = 0, at = __popc(f & below), place = __popc(h & below), pieces = 1;
  bool open = true;  // the item's end has not been met
#pragma unroll
  for (int k = 0; k < kWords; ++k) {
    if (k < warp) at += __popc(first[k]), place += __popc(has[k]);
    count += __popc(first[k]);
    if (k >= warp && open) {
      const uint32_t behind = k == warp ? ~(below << 1 | 1u) : 0xFFFFFFFFu, end = ends[k] & behind;
      open = end == 0;
      pieces += __popc(has[k] & behind & (open ? 0xFFFFFFFFu : end ^ (end - 1)));
    }
  }
  if (busy_range) busy[place] = mine;
  if (begins) chains[at] = make_int4(info.w, 2 * mine + (one ? 0 : 1), place, pieces), queries[at] = make_int2(info.y, info.z);
  __syncthreads();
  const int row = threadIdx.x;
  for (int item = blockIdx.x; item < count * kJoinChunks; item += gridDim.x) {
    const int c = item % kJoinChunks;
    const int4 chain = chains[item / kJoinChunks];
    const int pieces = chain.w;
    const int2 what = queries[item / kJoinChunks];
    float o[8] = {}, l = 0.f, top = -INFINITY;
    bool complete = true;
    for (int k0 = 0; k0 < pieces; k0 += kJoinAhead) {
      float2 ml[kJoinAhead];
      float4 v[kJoinAhead][2];
      int done[kJoinAhead];
#pragma unroll
      for (int k = 0; k < kJoinAhead; ++k) {
        if (k0 + k < pieces) {
          const int64_t slot = k0 + k == 0 ? chain.y : 2 * busy[chain.z + k0 + k];
          done[k] = P.done[slot * 8 + warp];
          ml[k] = P.ml[slot * kRows + row];
          const float4* const s = P.sums + (slot * (kValue / 4) + 2 * c) * kRows + row;
          v[k][0] = s[0], v[k][1] = s[kRows];
        }
      }
#pragma unroll
      for (int k = 0; k < kJoinAhead; ++k) {
        if (k0 + k >= pieces) break;
        complete &= done[k] != 0;
        const float to = fmaxf(top, ml[k].x), off = to == -INFINITY ? 0.f : to;
        const float f = exp2f(ml[k].x - off), was = exp2f(top - off);
        // (a piece without a step for the query's tile holds no sums)
        const bool sums = ml[k].x > -INFINITY || ml[k].y != 0.f;
        const float e[8] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w, v[k][1].x, v[k][1].y, v[k][1].z, v[k][1].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = o[j] * was + (sums ? f * e[j] : 0.f);
        l = l * was + f * ml[k].y;
        top = to;
      }
    }
    if (!complete || row >= what.y) continue;  // a wait ran out; behind the item's last query
    const float inv = top > -INFINITY ? 1.f / l : 0.f;
    uint32_t v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = pack_bf16(o[2 * k] * inv, o[2 * k + 1] * inv);
    *reinterpret_cast<uint4*>(P.out + ((int64_t)(what.x + row) * P.H + chain.x) * kValue + 8 * c) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}
static_assert(kMaxRanges == kRows, "a thread looks at a range");

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

int most_ranges() { return std::min(kMaxRanges, num_sms()); }
size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace

cudaError_t latent_attention_error(int32_t** word) {
  return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_attention_err);
}

}  // namespace moe_fp4

using namespace moe_fp4;

extern "C" {

size_t moe_fp4_latent_attention_workspace_bytes(void) {
  const size_t slots = 2 * (size_t)most_ranges();
  return align256(kMaxRanges * sizeof(int4)) + align256(slots * 8 * sizeof(int32_t)) + slots * kRows * sizeof(float2) +
         slots * kRows * kValue * sizeof(float);
}

int moe_fp4_latent_attention(const moe_fp4_latent_attention_args* args, void* workspace, size_t workspace_bytes,
                             void* cuda_stream) {
  if (!args) return MOE_FP4_ERR_INVALID_ARG;
  const moe_fp4_latent_attention_args a = *args;
  if (a.B < 0 || a.H < 1 || a.H > MOE_FP4_LATENT_MAX_HEADS || a.Tq < 0 || a.Tk < 0 || !(a.scale > 0.f) || !finite_scale(a.scale) ||
      a.causal < 0 || a.causal > 1)
    return MOE_FP4_ERR_INVALID_ARG;
  // items and TMA coordinates are counted in 32 bits
  const int64_t tiles = a.Tq / (2 * kQ) + std::min<int64_t>(a.B, a.Tq);
  if (a.B > kMaxSequences || a.Tq > INT32_MAX - 4 * kQ || a.Tk > INT32_MAX - 2 * kK || tiles * a.H >= (1LL << 30) || (int64_t)a.B * a.H >= (1LL << 31)) return MOE_FP4_ERR_UNSUPPORTED;
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
  if (!workspace || ((uintptr_t)workspace & 255)) return MOE_FP4_ERR_INVALID_ARG;
  if (workspace_bytes < moe_fp4_latent_attention_workspace_bytes()) return MOE_FP4_ERR_WORKSPACE;
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
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  // Sequences of few queries and keys, where there may be many of them, or no others.  (The fault tests' long waits are
  // the other kernel's.)
  const bool only = few(a.Tq, a.Tk);
  P.others = (only || (a.Tq <= (int64_t)kFewQueries * a.B && (int64_t)a.B * a.H >= (int64_t)kFewItems * num_sms())) && !P.fault;
  if (P.others) {
    const FewParams F{P, static_cast<const uint16_t*>(a.q), static_cast<const uint16_t*>(a.kv), static_cast<const uint16_t*>(a.k_rope),
                      a.q_stride, a.q_head_stride, a.kv_stride, a.kv_head_stride, a.rope_stride, only};
    if (launch_early(latent_attention_few_kernel, dim3((unsigned)(a.B * ((a.H + kFewWarps - 1) / kFewWarps))), dim3(32 * kFewWarps), 0, st, F) != cudaSuccess)
      return MOE_FP4_ERR_CUDA;
    if (only) return MOE_FP4_OK;
  }
  if (ready() != cudaSuccess) return MOE_FP4_ERR_CUDA;
  // ranges for all SMs if items may be cut, else for the items that there may be
  const bool cut = a.Tk > kMinSplit * kK;
  P.ranges = cut ? most_ranges() : (int)std::min<int64_t>(most_ranges(), tiles * a.H);
  P.dealt = !cut && a.B <= 32 && tiles * a.H <= P.ranges;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const size_t slots = 2 * (size_t)most_ranges();
  P.info = reinterpret_cast<int4*>(ws);
  ws += align256(kMaxRanges * sizeof(int4));
  P.done = reinterpret_cast<int32_t*>(ws);
  ws += align256(slots * 8 * sizeof(int32_t));
  P.ml = reinterpret_cast<float2*>(ws);
  P.sums = reinterpret_cast<float4*>(ws + slots * kRows * sizeof(float2));
  if (launch_early(latent_attention_kernel, dim3(P.ranges), dim3(kThreads), kSmem, st, map_q, map_kv, map_rope, P) != cudaSuccess)
    return MOE_FP4_ERR_CUDA;
  if (!cut) return MOE_FP4_OK;
  // an item is cut for each range but the first, at most
  const int64_t items = std::min<int64_t>(P.ranges - 1, tiles * a.H) * kJoinChunks;
  if (items == 0) return MOE_FP4_OK;
  return launch_early(latent_attention_join_kernel, dim3((unsigned)std::min<int64_t>(items, 8 * num_sms())), dim3(kRows), 0, st,
                      P) == cudaSuccess
             ? MOE_FP4_OK
             : MOE_FP4_ERR_CUDA;
}

}  // extern "C"
