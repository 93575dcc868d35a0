// The end of a block in one pass over its rows:
//
//   b = y + y2;  b *= rsqrt(mean b^2 + eps);  b *= post_weight;  b *= gate | sigmoid(gate)
//   out = residual + scale b;  normed = out rsqrt(mean out^2 + eps) next_weight
//
// Every operand is read once: a row stays in registers between its two sums of
// squares.  Sums are fp32: a thread's elements in order, then a tree over the
// CTA (a fixed order: the same bits on every call).
//
// Few rows: one CTA a row, bound by latency.  Many rows: bound by HBM, and with
// a CTA a row its loads stop while the sums are reduced and the row is written
// (16384 x 7168, fp32 + bf16 branch, bf16 residual: 298 us, 4.7 TB/s).  There
// persistent CTAs keep a ring of rows in shared memory that bulk copies fill
// ahead, and the weights in registers: 200 us, 7.1 TB/s, the rate of a copy.
#include <algorithm>

#include "moe_fp4_internal.cuh"
#include "mxfp4_ops.cuh"
#include "ptx_sm103.cuh"

namespace moe_fp4 {
namespace {

__device__ int32_t g_norm_err[4];

struct NormParams {
  moe_fp4_block_norm_args a;
  float k;  // d^-1/2: the squares of k v sum to the mean, which overflows only if the mean itself does
};

// Where element j of a thread's chunk c is.  V adjacent elements a load: 8 where
// rows start on 16 bytes and d is a multiple of 8; else a warp's 256 elements in
// turns of its 32 lanes, 2 (rows start on two elements, d is even) or 1 a lane, so
// that one address and one comparison serve the 8.
template <int V>
__device__ __forceinline__ int elem(int c, int j) {
  const int i = c * (int)blockDim.x + (int)threadIdx.x;
  return V == 8 ? i * 8 + j : (i & ~31) * 8 + (i & 31) * V + j / V * 32 * V + j % V;
}

// 8 values from p = the first on; `left` elements are there to the row's end
template <int V>
__device__ __forceinline__ void load8(const void* p, bool f32, int left, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; j += V) {
    const int at = V == 8 ? 0 : j * 32;
    const float* const pf = static_cast<const float*>(p) + at;
    const uint16_t* const ph = static_cast<const uint16_t*>(p) + at;
#pragma unroll
    for (int i = 0; i < V; ++i) v[j + i] = 0.f;
    if (at >= left) continue;
    if constexpr (V == 8) {
      if (f32) {
        const float4 x = reinterpret_cast<const float4*>(pf)[0], y = reinterpret_cast<const float4*>(pf)[1];
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
      } else {
        const uint4 x = *reinterpret_cast<const uint4*>(ph);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = __uint_as_float(w[i] << 16);
          v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
      }
    } else if constexpr (V == 2) {
      if (f32) {
        const float2 x = *reinterpret_cast<const float2*>(pf);
        v[j] = x.x, v[j + 1] = x.y;
      } else {
        const uint32_t x = *reinterpret_cast<const uint32_t*>(ph);
        v[j] = __uint_as_float(x << 16);
        v[j + 1] = __uint_as_float(x & 0xFFFF0000u);
      }
    } else {
      v[j] = f32 ? *pf : bf16_to_f32(*ph);
    }
  }
}

// chunk c of the row that starts at element row_at
template <int V>
__device__ __forceinline__ void load8(const void* base, int type, int64_t row_at, int c, int d, float (&v)[8]) {
  const int e = elem<V>(c, 0);
  if (type == MOE_FP4_TYPE_F32)
    load8<V>(static_cast<const float*>(base) + row_at + e, true, d - e, v);
  else
    load8<V>(static_cast<const uint16_t*>(base) + row_at + e, false, d - e, v);
}

template <int V>
__device__ __forceinline__ void store8(void* base, int type, int64_t row_at, int c, int d, const float (&v)[8]) {
  const int e = elem<V>(c, 0), left = d - e;
  auto bf2 = [](float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&p);
  };
  if (type == MOE_FP4_TYPE_F32) {
    float* const p = static_cast<float*>(base) + row_at + e;
#pragma unroll
    for (int j = 0; j < 8; j += V) {
      if ((V == 8 ? 0 : j * 32) >= left) continue;
      if constexpr (V == 8) {
        reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else if constexpr (V == 2) {
        *reinterpret_cast<float2*>(p + j * 32) = make_float2(v[j], v[j + 1]);
      } else {
        p[j * 32] = v[j];
      }
    }
  } else {
    uint16_t* const p = static_cast<uint16_t*>(base) + row_at + e;
#pragma unroll
    for (int j = 0; j < 8; j += V) {
      if ((V == 8 ? 0 : j * 32) >= left) continue;
      if constexpr (V == 8)
        *reinterpret_cast<uint4*>(p) =
            make_uint4(bf2(v[0], v[1]), bf2(v[2], v[3]), bf2(v[4], v[5]), bf2(v[6], v[7]));
      else if constexpr (V == 2)
        *reinterpret_cast<uint32_t*>(p + j * 32) = bf2(v[j], v[j + 1]);
      else
        p[j * 32] = f32_to_bf16_rn(v[j]);
    }
  }
}

// For results in bf16, many at a time: its error (2^-18 of the value at |g| = 80)
// is far below their rounding.  (A gate of every element, 16384 x 7168: 263 us,
// 286 with the other one.)
__device__ __forceinline__ float fast_sigmoid(float g) { return __fdividef(1.f, 1.f + __expf(-g)); }

// sum over the CTA, the same in every thread; `part` holds 32 floats.  What a
// thread wrote before it the others see behind it.
__device__ __forceinline__ float cta_sum(float s, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (warps == 1) {
    __syncwarp();
    return s;
  }
  if (lane == 0) part[warp] = s;
  __syncthreads();
  float t = lane < warps ? part[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
  return t;
}

// GATE: whether there is a gate of elements (of every one, or of channels in the
// form for few rows), and for which results: in bf16 its sigmoid is the fast one.
// (A kernel of its own for each: with both sigmoids in the loop, and none
// needed, 16384 x 7168 takes 204 us, 200 so.)
enum class Gate { none, bf16, f32 };

template <int NC, int V, Gate GATE>
__global__ void __launch_bounds__(1024, NC == 1 && V > 1 ? 2 : 1) block_norm_kernel(const NormParams P) {
  griddep_begin();
  __shared__ float part[2][32];
  const moe_fp4_block_norm_args& a = P.a;
  const int64_t t = blockIdx.x;
  const int d = a.d;
  float r[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c) load8<V>(a.residual, a.residual_type, t * a.residual_stride, c, d, r[c]);
  if (a.y) {
    float b[NC][8];
#pragma unroll
    for (int c = 0; c < NC; ++c) load8<V>(a.y, a.y_type, t * a.y_stride, c, d, b[c]);
    if (a.y2) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        float v[8];
        load8<V>(a.y2, a.y2_type, t * a.y2_stride, c, d, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) b[c][j] += v[j];
      }
    }
    float m = a.scale;
    if (GATE == Gate::none && a.gate_shape == MOE_FP4_GATE_TOKEN) {
      const float g = a.gate_type == MOE_FP4_TYPE_F32 ? static_cast<const float*>(a.gate)[t]
                                                      : bf16_to_f32(static_cast<const uint16_t*>(a.gate)[t]);
      m *= a.gate_sigmoid ? sigmoid(g) : g;
    }
    if (a.post_norm) {
      float s = 0.f;
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) s += (P.k * b[c][j]) * (P.k * b[c][j]);
      m *= rsqrtf(cta_sum(s, part[0]) + a.eps);
    }
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) b[c][j] *= m;
      if (a.post_weight) {
        load8<V>(a.post_weight, a.post_weight_type, 0, c, d, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) b[c][j] *= v[j];
      }
      if (GATE != Gate::none) {
        load8<V>(a.gate, a.gate_type, a.gate_shape == MOE_FP4_GATE_ELEMENT ? t * a.gate_stride : 0, c, d, v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          b[c][j] *= !a.gate_sigmoid ? v[j] : GATE == Gate::f32 ? sigmoid(v[j]) : fast_sigmoid(v[j]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) r[c][j] += b[c][j];
    }
  }
  if (a.out) {
#pragma unroll
    for (int c = 0; c < NC; ++c) store8<V>(a.out, a.residual_type, t * a.out_stride, c, d, r[c]);
  }
  if (!a.normed) return;
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) s += (P.k * r[c][j]) * (P.k * r[c][j]);
  const float n = rsqrtf(cta_sum(s, part[1]) + a.eps);
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[c][j] *= n;
    if (a.next_weight) {
      load8<V>(a.next_weight, a.next_weight_type, 0, c, d, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) r[c][j] *= v[j];
    }
    store8<V>(a.normed, MOE_FP4_TYPE_BF16, t * d, c, d, r[c]);
  }
}

// ---- many rows ----
// Two chunks of 8 elements a thread, placed as above.  A bulk copy starts on 16
// bytes and has a multiple of them: a row that does not is copied with its
// neighbours' ends (up to 15 bytes on both sides) and read at its offset; the
// first and the last row, beside which memory may be another's, are read where
// they are.
constexpr int kRingThreads = 512;      // with the weights in registers; 1024 read them again for every row
constexpr int kRingSmThreads = 640;    // on an SM, in CTAs of up to 512: 5 warps of each of its quarters, 96 registers a thread
constexpr int kRingMaxSlots = 8;
constexpr int kRingSmem = 200 * 1024;

struct RingParams {
  NormParams n;
  int slots, slot_bytes;                    // rows in the ring
  int y_bytes, y2_bytes, r_bytes, g_bytes;  // of a row in its slot; 0: not there
  int fault;                                // CTA 0 never loads its first row
  uint64_t wait_ns;
};

// The row weights from element `at` on, or `to` where there are none.
template <int V>
__device__ __forceinline__ void weight8(const void* w, int type, int at, int d, float to, float (&v)[8]) {
  if (w) {
    const bool f = type == MOE_FP4_TYPE_F32;
    load8<V>(static_cast<const uint8_t*>(w) + (size_t)at * (f ? 4 : 2), f, d - at, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 1.f;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= to;
}

template <bool KEEP, int V, Gate GATE>
__global__ void __launch_bounds__(KEEP ? kRingSmThreads : 2 * kRingThreads, 1)
block_norm_ring_kernel(const RingParams R) {
  griddep_begin();
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float part[2][2][32];
  __shared__ uint64_t full[kRingMaxSlots];
  __shared__ int abort_word;
  const moe_fp4_block_norm_args& a = R.n.a;
  volatile int* abort_flag = &abort_word;
  const int d = a.d, tid = threadIdx.x;
  const int64_t T = a.T, step = gridDim.x;
  const bool yf = a.y_type == MOE_FP4_TYPE_F32, y2f = a.y2_type == MOE_FP4_TYPE_F32,
             rf = a.residual_type == MOE_FP4_TYPE_F32, gf = a.gate_type == MOE_FP4_TYPE_F32;
  if (tid == 0) {
    for (int s = 0; s < R.slots; ++s) mbar_init(&full[s], 1);
    abort_word = 0;
    mbar_fence_init();
  }
  // where row t of an operand is, and whether it is read there
  auto row = [&](const void* base, bool f, int64_t stride, int64_t t) {
    return static_cast<const uint8_t*>(base) + t * stride * (f ? 4 : 2);
  };
  auto edge = [&](int64_t t) { return V == 1 && (t == 0 || t == T - 1); };
  // one thread: the operands of row t to slot s
  auto fill = [&](int64_t t, int s) {
    if (edge(t)) {
      mbar_arrive(&full[s]);
      return;
    }
    uint8_t* p = ring + (size_t)s * R.slot_bytes;
    const uint8_t* from[4] = {row(a.residual, rf, a.residual_stride, t), row(a.y, yf, a.y_stride, t),
                              row(a.y2, y2f, a.y2_stride, t), row(a.gate, gf, a.gate_stride, t)};
    const int room[4] = {R.r_bytes, R.y_bytes, R.y2_bytes, R.g_bytes};
    const bool wide[4] = {rf, yf, y2f, gf};
    uint32_t bytes[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bytes[i] = room[i];
      if (V == 1 && room[i]) {
        const uint32_t skip = (uint32_t)(uintptr_t)from[i] & 15;
        from[i] -= skip;
        bytes[i] = (skip + d * (wide[i] ? 4 : 2) + 15) & ~15u;
      }
      sum += bytes[i];
    }
    mbar_expect_tx(&full[s], sum);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (room[i]) bulk_load(p, from[i], bytes[i], &full[s]);
      p += room[i];
    }
  };
  int fills = 0;  // of thread 0
  if (tid == 0)
    for (; fills < R.slots && blockIdx.x + fills * step < T; ++fills)
      if (!(R.fault && blockIdx.x == 0 && fills == 0)) fill(blockIdx.x + fills * step, fills);
  // what multiplies the branch (its weight, a channel gate, the scale), and the next norm's weight
  const int at[2] = {elem<V>(0, 0), elem<V>(1, 0)};
  auto branch_weights = [&](int c, float (&w)[8]) {
    weight8<V>(a.post_weight, a.post_weight_type, at[c], d, a.scale, w);
    if (GATE != Gate::none || a.gate_shape != MOE_FP4_GATE_CHANNEL) return;
    float g[8];
    load8<V>(static_cast<const uint8_t*>(a.gate) + (size_t)at[c] * (gf ? 4 : 2), gf, d - at[c], g);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] *= a.gate_sigmoid ? sigmoid(g[j]) : g[j];
  };
  float bw[KEEP ? 2 : 1][8], nw[KEEP ? 2 : 1][8];
#pragma unroll
  for (int c = 0; c < (KEEP ? 2 : 1); ++c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) bw[c][j] = nw[c][j] = 0.f;
    if (!KEEP || at[c] >= d) continue;
    branch_weights(c, bw[c]);
    weight8<V>(a.next_weight, a.next_weight_type, at[c], d, 1.f, nw[c]);
  }
  __syncthreads();
  // Once a wait has run out the CTA stores nothing any more: the slots are not filled again, and a barrier that is a
  // phase behind would let later rows pass.  A thread knows it of its own waits, and behind a sum (of this row or an
  // earlier one) of those of all the threads that were in it, which raised the flag before its barrier; every thread
  // goes on through the sums' barriers.
  bool ok = true;
  int s = 0, i = 0;
  uint32_t phase = 0;
  for (int64_t t = blockIdx.x; t < T; t += step, ++i) {
    float m = 1.f;
    if (GATE == Gate::none && a.gate_shape == MOE_FP4_GATE_TOKEN) {
      m = gf ? static_cast<const float*>(a.gate)[t] : bf16_to_f32(static_cast<const uint16_t*>(a.gate)[t]);
      if (a.gate_sigmoid) m = sigmoid(m);
    }
    ok &= mbar_wait(&full[s], phase, abort_flag, &g_norm_err[0], kErrWaitTimeout, R.wait_ns);
    const uint8_t* pr = ring + (size_t)s * R.slot_bytes;
    const uint8_t* py = pr + R.r_bytes;
    const uint8_t* py2 = py + R.y_bytes;
    const uint8_t* pg = py2 + R.y2_bytes;
    if (V == 1) {
      auto at_row = [&](const uint8_t*& p, const uint8_t* g) { p = edge(t) ? g : p + ((uintptr_t)g & 15); };
      at_row(pr, row(a.residual, rf, a.residual_stride, t));
      at_row(py, row(a.y, yf, a.y_stride, t));
      at_row(py2, row(a.y2, y2f, a.y2_stride, t));
      at_row(pg, row(a.gate, gf, a.gate_stride, t));
    }
    float r[2][8];
    if (a.y) {
      float b[2][8];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (at[c] >= d) {
#pragma unroll
          for (int j = 0; j < 8; ++j) b[c][j] = 0.f;
          continue;
        }
        load8<V>(py + at[c] * (yf ? 4 : 2), yf, d - at[c], b[c]);
        if (R.y2_bytes) {
          float v[8];
          load8<V>(py2 + at[c] * (y2f ? 4 : 2), y2f, d - at[c], v);
#pragma unroll
          for (int j = 0; j < 8; ++j) b[c][j] += v[j];
        }
      }
      if (a.post_norm) {
        float q = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) q += (R.n.k * b[c][j]) * (R.n.k * b[c][j]);
        m *= rsqrtf(cta_sum(q, part[i & 1][0]) + a.eps);
        ok &= !*abort_flag;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float v[8];
        if (!KEEP && at[c] < d) branch_weights(c, bw[0]);
#pragma unroll
        for (int j = 0; j < 8; ++j) b[c][j] *= m * bw[KEEP ? c : 0][j];
        if (GATE != Gate::none && at[c] < d) {
          load8<V>(pg + at[c] * (gf ? 4 : 2), gf, d - at[c], v);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            b[c][j] *= !a.gate_sigmoid ? v[j] : GATE == Gate::f32 ? sigmoid(v[j]) : fast_sigmoid(v[j]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) r[c][j] = 0.f;
        if (at[c] < d) load8<V>(pr + at[c] * (rf ? 4 : 2), rf, d - at[c], r[c]);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[c][j] += b[c][j];
      }
    } else {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int j = 0; j < 8; ++j) r[c][j] = 0.f;
        if (at[c] < d) load8<V>(pr + at[c] * (rf ? 4 : 2), rf, d - at[c], r[c]);
      }
    }
    if (a.out && ok) {
#pragma unroll
      for (int c = 0; c < 2; ++c) store8<V>(a.out, a.residual_type, t * a.out_stride, c, d, r[c]);
    }
    float n = 0.f;
    if (a.normed) {
      float q = 0.f;
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) q += (R.n.k * r[c][j]) * (R.n.k * r[c][j]);
      n = rsqrtf(cta_sum(q, part[i & 1][1]) + a.eps);
      ok &= !*abort_flag;
      if (blockDim.x == 32) __syncthreads();
    } else {
      __syncthreads();
    }
    // (a barrier has passed since the last read of the slot, and since the sums of row i - 1 were read)
    if (tid == 0 && t + (int64_t)R.slots * step < T && !*abort_flag) {
      fill(t + (int64_t)R.slots * step, s);
      ++fills;
    }
    if (a.normed && ok) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (!KEEP && at[c] < d) weight8<V>(a.next_weight, a.next_weight_type, at[c], d, 1.f, nw[0]);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[c][j] *= n * nw[KEEP ? c : 0][j];
        store8<V>(a.normed, MOE_FP4_TYPE_BF16, t * d, c, d, r[c]);
      }
    }
    if (++s == R.slots) {
      s = 0;
      phase ^= 1;
    }
  }
  // every row that was filled has been waited for, unless a wait ran out: then no copy may outlive the CTA
  __syncthreads();
  if (tid == 0 && *abort_flag)
    for (int q = std::max(fills - R.slots, 0); q < fills; ++q)
      mbar_wait_drain(&full[q % R.slots], (q / R.slots) & 1, &g_norm_err[0], kErrWaitTimeout, R.wait_ns);
  __syncthreads();
}

// The ring's layout and grid; false where the plain kernel is used: few rows, or
// too wide ones.
template <int V>
bool ring_layout(const NormParams& P, RingParams* R, int* threads, int* ctas) {
  const moe_fp4_block_norm_args& a = P.a;
  const int chunks = (a.d + 7) / 8;
  *threads = std::max(32, ((chunks + 1) / 2 + 31) / 32 * 32);
  if (*threads > 2 * kRingThreads) return false;
  // rows read element by element are bound by instructions: the ring's fewer
  // threads an SM pay for wide ones alone (bf16: 8192 x 3001 64 us, plain 64; x 4097
  // 89 and 116; 4096 x 7167 81 and 122), and not at all by pairs (8192 x 5122 114
  // and 91; 4096 x 7166 72 and 72)
  if (V == 1 && a.d <= 4096) return false;
  auto bytes = [&](const void* p, int type) {
    const int n = a.d * (type == MOE_FP4_TYPE_F32 ? 4 : 2);
    return p ? V == 8 ? n : (n + 30) / 16 * 16 : 0;
  };
  R->n = P;
  R->y_bytes = bytes(a.y, a.y_type);
  R->y2_bytes = bytes(a.y2, a.y2_type);
  R->r_bytes = bytes(a.residual, a.residual_type);
  R->g_bytes = a.gate_shape == MOE_FP4_GATE_ELEMENT ? bytes(a.gate, a.gate_type) : 0;
  R->slot_bytes = (R->y_bytes + R->y2_bytes + R->r_bytes + R->g_bytes + 127) / 128 * 128;
  // as many CTAs an SM as run there (4096 x 5120, bf16: two of 320 threads 33 us,
  // one 50) with 2 rows in the ring (two are enough, 8192 x 3584, fp32: two CTAs of
  // 2 rows 95 us, one of 4 154)
  int per_sm = std::max(1, kRingSmThreads / *threads);
  while (per_sm > 1 && kRingSmem / per_sm / R->slot_bytes < 2) --per_sm;
  *ctas = per_sm * num_sms();
  if (a.T < 4 * (int64_t)*ctas) return false;
  R->slots = std::min(kRingMaxSlots, kRingSmem / per_sm / R->slot_bytes);
  R->fault = fault_site() == MOE_FP4_FAULT_TC_TOKEN_TILE;
  R->wait_ns = wait_limit_ns();
  return R->slots >= 2;
}

template <int V, Gate GATE>
cudaError_t launch_ring(const RingParams& R, int threads, int ctas, cudaStream_t st) {
  auto* k = threads <= kRingThreads ? block_norm_ring_kernel<true, V, GATE> : block_norm_ring_kernel<false, V, GATE>;
  const cudaError_t e = ensure_smem_optin(reinterpret_cast<const void*>(k), kRingSmem);
  if (e != cudaSuccess) return e;
  return launch_early(k, dim3(ctas), dim3(threads), R.slots * R.slot_bytes, st, R);
}

template <int V, Gate GATE>
cudaError_t launch_rows(const NormParams& P, cudaStream_t st) {
  // a CTA a row: one chunk of 8 elements a thread up to 1024 threads (few rows are bound by latency), else two
  const int chunks = (P.a.d + 7) / 8, nc = chunks <= 1024 ? 1 : 2;
  const int threads = ((chunks + nc - 1) / nc + 31) / 32 * 32;
  return launch_spread(nc == 1 ? block_norm_kernel<1, V, GATE> : block_norm_kernel<2, V, GATE>, (unsigned)P.a.T,
                       (unsigned)threads, st, P);
}

template <int V>
cudaError_t launch_norm(const NormParams& P, cudaStream_t st) {
  const bool f32 = P.a.residual_type == MOE_FP4_TYPE_F32;
  RingParams R;
  int threads, ctas;
  if constexpr (V != 2)
    if (ring_layout<V>(P, &R, &threads, &ctas))
      return P.a.gate_shape != MOE_FP4_GATE_ELEMENT ? launch_ring<V, Gate::none>(R, threads, ctas, st)
             : f32                                  ? launch_ring<V, Gate::f32>(R, threads, ctas, st)
                                                    : launch_ring<V, Gate::bf16>(R, threads, ctas, st);
  return P.a.gate_shape < MOE_FP4_GATE_CHANNEL ? launch_rows<V, Gate::none>(P, st)
         : f32                                 ? launch_rows<V, Gate::f32>(P, st)
                                               : launch_rows<V, Gate::bf16>(P, st);
}

bool is_type(int t) { return t == MOE_FP4_TYPE_BF16 || t == MOE_FP4_TYPE_F32; }
int64_t type_size(int t) { return t == MOE_FP4_TYPE_F32 ? 4 : 2; }
// an operand of whole elements; *v goes down to what its rows' starts allow
bool operand_ok(const void* p, int type, int64_t stride, int64_t rows, int d, int* v) {
  if (!is_type(type) || ((uintptr_t)p & (uintptr_t)(type_size(type) - 1))) return false;
  if (rows > 1 && (stride < d || stride >= (1LL << 32))) return false;
  const uintptr_t starts = (uintptr_t)p | (rows > 1 ? (uintptr_t)(stride * type_size(type)) : 0);
  *v = std::min(*v, starts % 16 == 0 ? 8 : starts % (2 * type_size(type)) == 0 ? 2 : 1);
  return true;
}

}  // namespace

cudaError_t ops_norm_error(int32_t** word) { return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_norm_err); }

}  // namespace moe_fp4

extern "C" int moe_fp4_block_norm(const moe_fp4_block_norm_args* args, void* cuda_stream) {
  using namespace moe_fp4;
  if (!args) return MOE_FP4_ERR_INVALID_ARG;
  const moe_fp4_block_norm_args& a = *args;
  if (a.T < 0 || a.T >= (1LL << 31) || a.d < 1 || a.d > 16384) return MOE_FP4_ERR_INVALID_ARG;
  if (!(a.eps >= 0.f) || a.gate_shape < MOE_FP4_GATE_NONE || a.gate_shape > MOE_FP4_GATE_ELEMENT)
    return MOE_FP4_ERR_INVALID_ARG;
  if (a.T == 0) return MOE_FP4_OK;
  if (!a.residual || (!a.out && !a.normed) || (a.y && !a.out)) return MOE_FP4_ERR_INVALID_ARG;
  if (!a.y && (a.y2 || a.post_norm || a.post_weight || a.gate_shape != MOE_FP4_GATE_NONE))
    return MOE_FP4_ERR_INVALID_ARG;
  if ((a.gate_shape != MOE_FP4_GATE_NONE) != (a.gate != nullptr) || (!a.normed && a.next_weight))
    return MOE_FP4_ERR_INVALID_ARG;
  int v = a.d % 8 == 0 ? 8 : a.d % 2 == 0 ? 2 : 1;
  if (!operand_ok(a.residual, a.residual_type, a.residual_stride, a.T, a.d, &v)) return MOE_FP4_ERR_INVALID_ARG;
  if (a.y && !operand_ok(a.y, a.y_type, a.y_stride, a.T, a.d, &v)) return MOE_FP4_ERR_INVALID_ARG;
  if (a.y2 && !operand_ok(a.y2, a.y2_type, a.y2_stride, a.T, a.d, &v)) return MOE_FP4_ERR_INVALID_ARG;
  if (a.post_weight && !operand_ok(a.post_weight, a.post_weight_type, a.d, 1, a.d, &v))
    return MOE_FP4_ERR_INVALID_ARG;
  if (a.next_weight && !operand_ok(a.next_weight, a.next_weight_type, a.d, 1, a.d, &v))
    return MOE_FP4_ERR_INVALID_ARG;
  int any = 8;  // a [T] gate is read one element a row
  if (a.gate && !operand_ok(a.gate, a.gate_type, a.gate_stride, a.gate_shape == MOE_FP4_GATE_ELEMENT ? a.T : 1, a.d,
                            a.gate_shape == MOE_FP4_GATE_TOKEN ? &any : &v))
    return MOE_FP4_ERR_INVALID_ARG;
  if (a.out && !operand_ok(a.out, a.residual_type, a.out_stride, a.T, a.d, &v)) return MOE_FP4_ERR_INVALID_ARG;
  if (a.normed && !operand_ok(a.normed, MOE_FP4_TYPE_BF16, a.d, a.T, a.d, &v)) return MOE_FP4_ERR_INVALID_ARG;
  const NormParams P{a, 1.0f / sqrtf((float)a.d)};
  cudaStream_t st = static_cast<cudaStream_t>(cuda_stream);
  const cudaError_t e = v == 8 ? launch_norm<8>(P, st) : v == 2 ? launch_norm<2>(P, st) : launch_norm<1>(P, st);
  return e == cudaSuccess ? MOE_FP4_OK : MOE_FP4_ERR_CUDA;
}
