// Block tables and slots of a batch's new tokens in a paged cache, from the
// requests' lengths: the step between a scheduler's list and the kernels that write
// and read the cache, without a copy to the host.
//
// Request b owns the pages of its n[b] tokens and gets t[b] new ones; it needs
// ceil((n + t) / page) - ceil(n / page) pages more, taken from the free list in the
// requests' order.  Both need sums over all requests before b: every CTA makes them
// itself (a few loads a thread), so that one launch does, and then takes its share of
// the tokens, finding a token's request by bisection.  A page's first new token
// enters it in the table; entries that this call enters are read by nobody in it.
//
// Latency bounds it: 32 requests of a token each take 2.8 us, 256 of 131072 tokens
// together 5.7, 8192 requests 28.
#include <algorithm>

#include "moe_fp4_internal.cuh"
#include "mxfp4_ops.cuh"

namespace moe_fp4 {
namespace {

__device__ int32_t g_pages_err[4];

constexpr int kThreads = 256;
constexpr int kMaxRequests = 8192;

struct PageParams {
  moe_fp4_page_slots_args a;
};

// (of what a row of the table holds, less than 2^31: a division of 64 bits takes 0.3 us)
__device__ __forceinline__ int64_t ceil_div(int64_t a, int32_t b) { return ((uint32_t)a + (uint32_t)b - 1) / (uint32_t)b; }

// inclusive sum over the block of a pair of values; total: of all threads
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

__global__ void __launch_bounds__(kThreads) page_slots_kernel(const PageParams Q) {
  griddep_begin();
  const moe_fp4_page_slots_args& P = Q.a;
  extern __shared__ longlong2 before[];  // [B + 1]: new tokens and new pages of the requests before b
  __shared__ longlong2 scratch[kThreads / 32];
  const int64_t most = (int64_t)P.width * P.page;  // tokens that a row of the table holds
  const bool first_cta = blockIdx.x == 0;
  longlong2 sum = make_longlong2(0, 0);
  long long keys = 0;
  int bad = 0;
  int next_n = 0, next_t = 0;  // on their way while the sums before them are made
  if ((int)threadIdx.x < P.B) next_n = P.lengths[threadIdx.x], next_t = P.new_tokens[threadIdx.x];
  for (int b0 = 0; b0 < P.B; b0 += kThreads) {
    const int b = b0 + threadIdx.x;
    int64_t n = next_n, t = next_t, after = 0;
    if (b + kThreads < P.B) next_n = P.lengths[b + kThreads], next_t = P.new_tokens[b + kThreads];
    if (b < P.B) {
      if (n < 0 || t < 0 || n + t > most) bad = kErrBadExpertId;
      n = min(max(n, (int64_t)0), most), t = max(t, (int64_t)0);
      after = min(n + t, most);
    } else {
      n = t = 0;
    }
    longlong2 all;
    const longlong2 own = make_longlong2(t, ceil_div(after, P.page) - ceil_div(n, P.page));
    const longlong2 v = block_scan(own, scratch, &all);
    if (b < P.B) before[b] = make_longlong2(sum.x + v.x - own.x, sum.y + v.y - own.y);
    sum.x += all.x, sum.y += all.y;
    if (first_cta) {  // (the same for all threads of a CTA)
      longlong2 all_keys;
      const longlong2 k = block_scan(make_longlong2(after, 0), scratch, &all_keys);
      if (b < P.B) {
        P.out_lengths[b] = (int32_t)after;
        P.q_offsets[b] = (int32_t)min((long long)P.tokens, before[b].x);
        P.k_offsets[b] = (int32_t)min((long long)INT32_MAX, keys + k.x - after);
      }
      keys += all_keys.x;
    }
  }
  long long taken = sum.y;
  if (first_cta && (sum.x > P.tokens || sum.y > P.free_count)) {
    // Some have no place: again with what the first P.tokens new tokens' own pages and the free ones hold.  (Beside the
    // sums above it costs 8% where all have one, 8192 requests.)
    keys = taken = 0;
    for (int b0 = 0; b0 < P.B; b0 += kThreads) {
      const int b = b0 + threadIdx.x;
      int64_t after = 0, pages = 0;
      if (b < P.B) {
        const int64_t n = min(max((int64_t)P.lengths[b], (int64_t)0), most), t = max((int64_t)P.new_tokens[b], (int64_t)0);
        const int64_t room = P.tokens - before[b].x, left = P.free_count - before[b].y, owned = ceil_div(n, P.page);
        after = min(min(n + t, most), n + min(t, max(room, (int64_t)0)));
        after = min(after, max(n, (owned + max(left, (int64_t)0)) * P.page));
        pages = ceil_div(after, P.page) - owned;
      }
      longlong2 all;
      const longlong2 k = block_scan(make_longlong2(after, pages), scratch, &all);
      if (b < P.B) {
        P.out_lengths[b] = (int32_t)after;
        P.k_offsets[b] = (int32_t)min((long long)INT32_MAX, keys + k.x - after);
      }
      keys += all.x, taken += all.y;
    }
  }
  if (threadIdx.x == 0) {
    before[P.B] = sum;
    if (first_cta) {
      P.q_offsets[P.B] = (int32_t)min((long long)P.tokens, sum.x);
      P.k_offsets[P.B] = (int32_t)min((long long)INT32_MAX, keys);
      *P.taken = (int32_t)taken;
      if (sum.x > P.tokens || sum.y > P.free_count || keys > INT32_MAX) bad = kErrBadExpertId;
    }
  }
  if (!first_cta) bad = 0;  // (one CTA reports the requests)
  __syncthreads();
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < P.tokens; i += (int64_t)gridDim.x * kThreads) {
    int64_t slot = -1, position = 0;
    if (i < sum.x) {
      int lo = 0, hi = P.B;  // the last request that begins at or before i (and is not empty)
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before[mid].x <= i)
          lo = mid;
        else
          hi = mid;
      }
      const int64_t n = min(max((int64_t)P.lengths[lo], (int64_t)0), most);
      position = n + i - before[lo].x;
      if (position < most) {
        const uint32_t index = (uint32_t)position / (uint32_t)P.page, in_page = (uint32_t)position - index * (uint32_t)P.page;
        const int64_t owned = ceil_div(n, P.page);
        int32_t* const entry = P.table + lo * P.table_stride + index;
        int32_t page = -1;
        if (index < owned) {
          page = *entry;
        } else {
          const int64_t f = before[lo].y + index - owned;
          if (f < P.free_count) {
            page = P.free_pages[f];
            if (in_page == 0) *entry = page;
          }
        }
        if (page >= 0)
          slot = (int64_t)page * P.page + in_page;
        else
          bad = kErrBadExpertId;  // no page for it, or the row or the free list names none
      } else {
        position = 0;
      }
    }
    P.slots[i] = slot;
    P.positions[i] = (int32_t)position;
  }
  if (bad) atomicOr(&g_pages_err[0], bad);
}

struct Bytes {
  uintptr_t at, size;
};
Bytes bytes_at(const void* p, int64_t size) { return {(uintptr_t)p, (uintptr_t)size}; }
bool overlap(const Bytes& x, const Bytes& y) {
  return x.size > 0 && y.size > 0 && x.at < y.at + y.size && y.at < x.at + x.size;
}
// whether some of x is in a row of the table (not only between rows)
bool in_table(const moe_fp4_page_slots_args& a, const Bytes& x) {
  const uintptr_t base = (uintptr_t)a.table, row = 4 * (uintptr_t)a.width, stride = 4 * (uintptr_t)a.table_stride;
  if (a.B == 0 || !overlap(x, {base, (uintptr_t)(a.B - 1) * stride + row})) return false;
  if (x.at <= base) return true;  // it reaches the first row
  const uintptr_t in_row = (x.at - base) % stride;
  return in_row < row || in_row + x.size > stride;
}

}  // namespace

cudaError_t page_slots_error(int32_t** word) { return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_pages_err); }

}  // namespace moe_fp4

using namespace moe_fp4;

extern "C" int moe_fp4_page_slots(const moe_fp4_page_slots_args* args, void* cuda_stream) {
  if (!args) return MOE_FP4_ERR_INVALID_ARG;
  const moe_fp4_page_slots_args a = *args;
  if (a.B < 0 || a.B > kMaxRequests || a.page < 1 || a.width < 1 || a.tokens < 0 || a.tokens > INT32_MAX || a.free_count < 0 ||
      a.free_count > INT32_MAX || a.table_stride < a.width)
    return MOE_FP4_ERR_INVALID_ARG;
  if ((int64_t)a.width * a.page >= (1LL << 31)) return MOE_FP4_ERR_UNSUPPORTED;
  if (!a.q_offsets || !a.k_offsets || !a.taken || (a.tokens > 0 && (!a.slots || !a.positions)) ||
      (a.B > 0 && (!a.lengths || !a.new_tokens || !a.table || !a.out_lengths)) || (a.free_count > 0 && !a.free_pages))
    return MOE_FP4_ERR_INVALID_ARG;
  if (((uintptr_t)a.slots & 7) || ((uintptr_t)a.lengths & 3) || ((uintptr_t)a.new_tokens & 3) || ((uintptr_t)a.table & 3) ||
      ((uintptr_t)a.free_pages & 3) || ((uintptr_t)a.positions & 3) || ((uintptr_t)a.out_lengths & 3) ||
      ((uintptr_t)a.q_offsets & 3) || ((uintptr_t)a.k_offsets & 3) || ((uintptr_t)a.taken & 3))
    return MOE_FP4_ERR_INVALID_ARG;
  // what a CTA writes, others read or write meanwhile, if it is the same memory
  const Bytes in[] = {bytes_at(a.lengths, 4 * (int64_t)a.B), bytes_at(a.new_tokens, 4 * (int64_t)a.B), bytes_at(a.free_pages, 4 * a.free_count)};
  const Bytes out[] = {bytes_at(a.slots, 8 * a.tokens),         bytes_at(a.positions, 4 * a.tokens),
                       bytes_at(a.out_lengths, 4 * (int64_t)a.B), bytes_at(a.q_offsets, 4 * ((int64_t)a.B + 1)),
                       bytes_at(a.k_offsets, 4 * ((int64_t)a.B + 1)), bytes_at(a.taken, 4)};
  for (const Bytes& i : in)
    if (in_table(a, i)) return MOE_FP4_ERR_INVALID_ARG;
  for (const Bytes& o : out) {
    if (in_table(a, o)) return MOE_FP4_ERR_INVALID_ARG;
    for (const Bytes& i : in)  // (out_lengths, beside the requests' numbers, as of B + 1)
      if (overlap(&o == &out[2] && &i != &in[2] ? Bytes{o.at, o.size + 4} : o, i)) return MOE_FP4_ERR_INVALID_ARG;
    for (const Bytes* p = out; p != &o; ++p)
      if (overlap(o, *p)) return MOE_FP4_ERR_INVALID_ARG;
  }
  PageParams P{a};
  const int smem = (a.B + 1) * (int)sizeof(longlong2);
  if (smem > 48 * 1024 - 256 &&
      ensure_smem_optin(reinterpret_cast<const void*>(page_slots_kernel), (kMaxRequests + 1) * (int)sizeof(longlong2)) != cudaSuccess)
    return MOE_FP4_ERR_CUDA;
  const int64_t blocks = std::min<int64_t>(std::max<int64_t>((a.tokens + kThreads - 1) / kThreads, 1), num_sms());
  return launch_early(page_slots_kernel, dim3((unsigned)blocks), dim3(kThreads), smem, static_cast<cudaStream_t>(cuda_stream), P) ==
                 cudaSuccess
             ? MOE_FP4_OK
             : MOE_FP4_ERR_CUDA;
}
